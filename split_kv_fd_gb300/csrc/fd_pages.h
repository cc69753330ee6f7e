// fd_pages.h -- parameter blocks and launchers of the page bookkeeping and
// the cache append, with the rotation and without (fd_pages.cu,
// fd_append.cu, fd_rope.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fd {

// Status bit (beside those of fd_device.cuh): a position without a row in the
// rotation's table, or a parent that is no beam.
constexpr unsigned STATUS_BAD_INDEX = 8u;

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

// An append with the rotation: K's (and q's) first `rot` elements of a head
// turned by the token's position on the way.
struct RopeParams {
    const void *q;           // [T, Hq, d], null with Hq = 0
    const void *k, *v;       // [T, H, d]
    void *q_out;             // [T, Hq, d]
    long long q_stride, q_out_stride, k_stride, v_stride;
    const int32_t *positions;   // [T]
    const float *table;         // [max_position, rot]: rot/2 cosines, rot/2 sines
    int max_position, rot, pairs;
    int T, Hq, H, d, dtype;
    const int32_t *slots;    // [T]
    void *k_pages, *v_pages; // [num_pages, H, page_size, d]
    int page_size;
    long long num_slots;
    int f8, B;
    const int32_t *cu;       // [B + 1]
    const float *k_scale, *v_scale;   // [B, H]
    int sms;                 // of the device
    unsigned *status;
};

cudaError_t launch_rope(const RopeParams &p, cudaStream_t s);

}  // namespace fd
