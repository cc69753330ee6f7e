// fd_append.cu -- new K and V rows into a paged KV cache: row t of head h to
// row slot % page_size of (page slot / page_size, head h), as they are or
// rounded to E4M3 with the sequence's scale.
#include "fd_device.cuh"
#include "fd_pages.h"

namespace fd {
namespace {

// One CTA a token; a thread moves one element.
template <typename T, bool F8> __global__ void append_kernel(const AppendParams p)
{
    const int t = blockIdx.x;
    const int slot = p.slots[t];
    if (slot < 0)
        return;
    if (slot >= p.num_slots) {
        if (threadIdx.x == 0)
            atomicOr(p.status, STATUS_BAD_PAGE);
        return;
    }
    int b = 0;
    if (F8) {
        if (t < p.cu[0] || t >= p.cu[p.B])
            return;
        while (b < p.B - 1 && p.cu[b + 1] <= t)
            ++b;
    }
    const long long page = slot / p.page_size;
    const int row = slot % p.page_size;
    for (int i = threadIdx.x; i < p.H * p.d; i += blockDim.x) {
        const int h = i / p.d, e = i % p.d;
        const long long dst = ((page * p.H + h) * p.page_size + row) * p.d + e;
        const T k = static_cast<const T *>(p.k)[t * p.k_stride + i];
        const T v = static_cast<const T *>(p.v)[t * p.v_stride + i];
        if (F8) {
            static_cast<__nv_fp8_e4m3 *>(p.k_pages)[dst] =
                __nv_fp8_e4m3(__fdiv_rn((float)k, p.k_scale[(long long)b * p.H + h]));
            static_cast<__nv_fp8_e4m3 *>(p.v_pages)[dst] =
                __nv_fp8_e4m3(__fdiv_rn((float)v, p.v_scale[(long long)b * p.H + h]));
        } else {
            static_cast<T *>(p.k_pages)[dst] = k;
            static_cast<T *>(p.v_pages)[dst] = v;
        }
    }
}

template <typename T> cudaError_t launch_t(const AppendParams &p, cudaStream_t s)
{
    if (p.f8)
        append_kernel<T, true><<<p.T, 256, 0, s>>>(p);
    else
        append_kernel<T, false><<<p.T, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, cudaStream_t s)
{
    return p.dtype == 0   ? launch_t<float>(p, s)
           : p.dtype == 1 ? launch_t<__half>(p, s)
                          : launch_t<__nv_bfloat16>(p, s);
}

}  // namespace fd
