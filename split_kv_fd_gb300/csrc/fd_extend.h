// fd_extend.h -- parameter block and launcher of attention with several new
// tokens a sequence (fd_extend.cuh): over a paged cache, or over packed
// prompts.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fd {

struct ExtendParams {
    const void *q;           // [total_q, Hq, d], q_stride elements between tokens
    long long q_stride;
    const void *k, *v;       // packed [total_k, Hkv, d] with strides, or pages [num_pages, Hkv, page_size, d]
    long long k_stride, v_stride;
    int paged;
    const int32_t *table;    // [B, max_pages]
    int page_size, max_pages;
    long long num_pages;
    const int32_t *cu_q;     // [B + 1] rows of q
    const int32_t *cu_k;     // [B + 1] rows of k, v (packed)
    const int32_t *seqlens;  // [B] tokens in the cache, the new ones among them (paged)
    int B, total_q, total_k, Hq, Hkv, d;
    int causal;
    float scale_log2;        // scale * log2(e): scores are kept in base 2
    int f8;                  // E4M3 K/V
    const float *k_scale, *v_scale;   // [B, Hkv]
    int dtype;               // of q, and of K/V unless f8
    void *out;               // [total_q, Hq, d]
    int out_dtype;
    float *lse;              // [total_q, Hq] or null
    unsigned *status;
};

cudaError_t launch_extend(const ExtendParams &p, cudaStream_t s);

}  // namespace fd
