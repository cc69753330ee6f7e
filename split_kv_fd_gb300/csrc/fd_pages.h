// fd_pages.h -- parameter blocks and launchers of the page bookkeeping and
// the cache append (fd_pages.cu, fd_append.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fd {

struct ResizeParams {
    int32_t *seqlens;        // [B] in, out
    const int32_t *target;   // [B]
    int B;
    int32_t *table;          // [B, max_pages] in, out
    int max_pages, page_size;
    int32_t *free_pages;     // [num_pages] stack, in, out
    int32_t *free_count;     // [1] in, out
    int num_pages;
    int32_t *slots;          // [max_tokens] or null
    int32_t *positions;      // [max_tokens] or null
    int max_tokens;
    int32_t *cu;             // [B + 1] or null
    unsigned *status;
};

cudaError_t launch_resize(const ResizeParams &p, cudaStream_t s);

struct AppendParams {
    const void *k, *v;       // [T, H, d], token strides in elements
    long long k_stride, v_stride;
    int T, H, d, dtype;
    int step;                // tokens side by side in a CTA
    const int32_t *slots;    // [T]
    void *k_pages, *v_pages; // [num_pages, H, page_size, d]
    int page_size;
    long long num_slots;     // num_pages * page_size
    // E4M3 pages: one scale per (sequence, head) and the rows' sequences
    int f8, B;
    const int32_t *cu;       // [B + 1]
    const float *k_scale, *v_scale;   // [B, H]
    unsigned *status;
};

cudaError_t launch_append(const AppendParams &p, cudaStream_t s);

}  // namespace fd
