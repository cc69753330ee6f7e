// fd_append.cu -- new K and V rows into a paged KV cache: row t of head h to
// row slot % page_size of (page slot / page_size, head h), as they are or
// rounded to E4M3 with the sequence's scale.
//
// The rows are only moved, so memory bounds it: each K and V element is read
// once and written once.  A thread moves 16 bytes of the result a token (32
// of a 16-bit source, 64 of a float32 one, where the result is E4M3), the
// same piece of a CTA's TOKENS tokens, all loads ahead of the stores.
#include "fd_device.cuh"
#include "fd_pages.h"

namespace fd {
namespace {

constexpr int AT = 256;   // threads of a CTA

__device__ __forceinline__ uint4 ldg_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Two floats to two E4M3 bytes (the first in the lower), to nearest, ties to
// even, saturated; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// T: of the rows.  A thread's 16 bytes are SRC 16-byte vectors of the source.
template <typename T, bool F8, int TOKENS> __global__ void __launch_bounds__(AT) append_kernel(const AppendParams p)
{
    constexpr int SRC = F8 ? (int)sizeof(T) : 1;
    constexpr int EL = F8 ? 16 : 16 / (int)sizeof(T);   // elements of a piece
    const int t0 = blockIdx.x * TOKENS;
    const int per = p.H * p.d / EL;                     // pieces of a token's K
    const int cpr = p.d / EL;                           // pieces of a head's row: a power of two
    const int shift = __ffs(cpr) - 1;

    // the slots, and for E4M3 the sequence of the CTA's first token: the
    // offsets at or below it, counted by the whole block
    int slot[TOKENS], seq[TOKENS];
#pragma unroll
    for (int u = 0; u < TOKENS; ++u) {
        slot[u] = t0 + u < p.T ? __ldg(p.slots + t0 + u) : -1;
        if (slot[u] >= p.num_slots) {
            if (threadIdx.x == 0)
                atomicOr(p.status, STATUS_BAD_PAGE);
            slot[u] = -1;
        }
        seq[u] = 0;
    }
    if (F8) {
        int n = 0;
        for (int b0 = 0; b0 <= p.B; b0 += AT) {
            const int b = b0 + (int)threadIdx.x;
            n += __syncthreads_count(b <= p.B && p.cu[min(b, p.B)] <= t0);
        }
        int b = n - 1;   // -1: before the first sequence
#pragma unroll
        for (int u = 0; u < TOKENS; ++u) {
            while (b < p.B && p.cu[b + 1] <= t0 + u)
                ++b;
            if (b < 0 || b >= p.B)
                slot[u] = -1;
            seq[u] = min(max(b, 0), p.B - 1);
        }
    }

    for (int c = threadIdx.x; c < 2 * per; c += AT) {
        const bool isv = c >= per;
        const int i = isv ? c - per : c;
        const int h = i >> shift, e = (i & (cpr - 1)) * EL;
        const T *src = static_cast<const T *>(isv ? p.v : p.k) + (long long)i * EL;
        const long long stride = isv ? p.v_stride : p.k_stride;
        char *pages = static_cast<char *>(isv ? p.v_pages : p.k_pages);
        uint4 x[TOKENS][SRC];
        float sc[TOKENS];
#pragma unroll
        for (int u = 0; u < TOKENS; ++u) {
            if (slot[u] < 0)
                continue;
#pragma unroll
            for (int k = 0; k < SRC; ++k)
                x[u][k] = ldg_stream(reinterpret_cast<const uint4 *>(src + (t0 + u) * stride) + k);
            if (F8)
                sc[u] = __ldg((isv ? p.v_scale : p.k_scale) + (long long)seq[u] * p.H + h);
        }
#pragma unroll
        for (int u = 0; u < TOKENS; ++u) {
            if (slot[u] < 0)
                continue;
            const long long row = ((long long)(slot[u] / p.page_size) * p.H + h) * p.page_size + slot[u] % p.page_size;
            uint4 y = x[u][0];
            if (F8) {
                float f[16];
#pragma unroll
                for (int k = 0; k < SRC; ++k)
                    Elem<T>::widen(x[u][k], f + k * Elem<T>::VEC);
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = e4m3x2(__fdiv_rn(f[4 * k], sc[u]), __fdiv_rn(f[4 * k + 1], sc[u])) |
                           e4m3x2(__fdiv_rn(f[4 * k + 2], sc[u]), __fdiv_rn(f[4 * k + 3], sc[u])) << 16;
                y = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *reinterpret_cast<uint4 *>(pages + (row * p.d + e) * (F8 ? 1 : (int)sizeof(T))) = y;
        }
    }
}

template <typename T, bool F8> cudaError_t launch_t(const AppendParams &p, cudaStream_t s)
{
    // several tokens a CTA once there are CTAs for every SM without
    if (p.T >= 4096)
        append_kernel<T, F8, 4><<<(p.T + 3) / 4, AT, 0, s>>>(p);
    else
        append_kernel<T, F8, 1><<<p.T, AT, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, cudaStream_t s)
{
    if (p.f8)
        return p.dtype == 0   ? launch_t<float, true>(p, s)
               : p.dtype == 1 ? launch_t<__half, true>(p, s)
                              : launch_t<__nv_bfloat16, true>(p, s);
    return p.dtype == 0 ? launch_t<float, false>(p, s) : launch_t<__half, false>(p, s);   // 16 bits are 16 bits
}

}  // namespace fd
