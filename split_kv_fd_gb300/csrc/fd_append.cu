// fd_append.cu -- new K and V rows into a paged KV cache: row t of head h to
// row slot % page_size of (page slot / page_size, head h), as they are or
// rounded to E4M3 with the sequence's scale.
//
// The rows are only moved, so memory bounds it: each K and V element is read
// once and written once.  A thread moves 16 bytes of the result a token (32
// of a 16-bit source, 64 of a float32 one, where the result is E4M3), the
// same piece of TOKENS tokens, all loads ahead of the stores.  16K tokens of
// 8 heads of 128, bf16 (views of a fused projection): 17-18 us where part of
// the rows is still in L2, 24 from memory, 5.3 TB/s; into E4M3 pages 20 us
// (59 with 4 tokens and an IEEE division an element).  256 tokens: 1.9 and
// 3.1 us, a launch and two or three dependent loads.
#include "fd_device.cuh"
#include "fd_e4m3.cuh"
#include "fd_pages.h"

namespace fd {
namespace {


__device__ __forceinline__ uint4 ldg_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Threads of a CTA: 8 heads of 128 are 256 pieces in 16 bits, 128 in E4M3
// (256 threads, half of them idle: 16K tokens 27 us against 20).
constexpr int threads(bool f8) { return f8 ? 128 : 256; }

// T: of the rows.  A thread's 16 bytes are SRC 16-byte vectors of the source.
template <typename T, bool F8, int TOKENS, bool SIDE, int AT>
__global__ void __launch_bounds__(AT) append_kernel(const AppendParams p)
{
    constexpr int EL = F8 ? 16 : 16 / (int)sizeof(T);   // elements of a piece
    constexpr int SRC = EL * (int)sizeof(T) / 16;       // its vectors of the source
    const int per = p.H * p.d / EL;                     // pieces of a token's K
    const int cpr = p.d / EL;                           // pieces of a head's row: a power of two
    const int shift = __ffs(cpr) - 1;
    // SIDE: `step` tokens side by side; this thread takes piece c0 of tokens
    // t0, t0 + step, ...
    const int step = SIDE ? p.step : 1;
    const int u0 = SIDE ? threadIdx.x / (2 * per) : 0;
    const int c0 = threadIdx.x - u0 * 2 * per;
    const int first = blockIdx.x * step * TOKENS, t0 = first + u0;

    // the slots, and for E4M3 the sequence of the CTA's first token: the
    // offsets at or below it, counted by the whole block
    int slot[TOKENS], seq[TOKENS];
#pragma unroll
    for (int u = 0; u < TOKENS; ++u) {
        const int t = t0 + u * step;
        slot[u] = u0 < step && t < p.T ? __ldg(p.slots + t) : -1;
        if (slot[u] >= p.num_slots) {
            if (c0 == 0)
                atomicOr(p.status, STATUS_BAD_PAGE);
            slot[u] = -1;
        }
        seq[u] = 0;
    }
    if (F8) {
        int n = 0;
        for (int b0 = 0; b0 <= p.B; b0 += AT) {
            const int b = b0 + (int)threadIdx.x;
            n += __syncthreads_count(b <= p.B && p.cu[min(b, p.B)] <= first);
        }
        int b = n - 1;   // -1: before the first sequence
#pragma unroll
        for (int u = 0; u < TOKENS; ++u) {
            while (b < p.B && p.cu[b + 1] <= t0 + u * step)
                ++b;
            if (b < 0 || b >= p.B)
                slot[u] = -1;
            seq[u] = min(max(b, 0), p.B - 1);
        }
    }

    for (int c = c0; c < 2 * per; c += AT) {
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
                x[u][k] = ldg_stream(reinterpret_cast<const uint4 *>(src + (t0 + u * step) * stride) + k);
            if (F8)
                sc[u] = __ldg((isv ? p.v_scale : p.k_scale) + (long long)seq[u] * p.H + h);
        }
#pragma unroll
        for (int u = 0; u < TOKENS; ++u) {
            if (slot[u] < 0)
                continue;
            const long long row = ((long long)(slot[u] / p.page_size) * p.H + h) * p.page_size + slot[u] % p.page_size;
            char *to = pages + (row * p.d + e) * (F8 ? 1 : (int)sizeof(T));
            if constexpr (F8) {
                float f[EL];
#pragma unroll
                for (int k = 0; k < SRC; ++k)
                    Elem<T>::widen(x[u][k], f + k * Elem<T>::VEC);
                uint32_t w[EL / 4];
                e4m3_quotients<EL>(f, sc[u], w);
                *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                *reinterpret_cast<uint4 *>(to) = x[u][0];
            }
        }
    }
}

template <typename T, bool F8, int TOKENS, bool SIDE> cudaError_t launch_n(const AppendParams &p, cudaStream_t s)
{
    constexpr int AT = threads(F8);
    const long long each = (long long)p.step * TOKENS;
    append_kernel<T, F8, TOKENS, SIDE, AT><<<(unsigned)((p.T + each - 1) / each), AT, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, bool F8> cudaError_t launch_t(AppendParams p, cudaStream_t s)
{
    // Tokens side by side where one does not fill a CTA (16K tokens of one
    // head of 64: bf16 2.8 us against 6.7, E4M3 3.1 against 11), several
    // each behind the other once there are CTAs for every SM without: of 8
    // heads of 128 in bf16, 16K tokens 18 us against 22, 2048 alike, 256
    // 1.7 against 2.2.  Not for E4M3, whose arithmetic wants more warps
    // (16K tokens 20 us either way, 256 2.8 against 3.8).
    constexpr int MANY = F8 ? 1 : 4;
    const long long pieces = 2LL * p.H * p.d * (int)(F8 ? 1 : sizeof(T)) / 16;   // of a token
    p.step = 2 * pieces <= threads(F8) ? (int)(threads(F8) / pieces) : 1;
    if (p.T / p.step >= 2048)
        return p.step > 1 ? launch_n<T, F8, MANY, true>(p, s) : launch_n<T, F8, MANY, false>(p, s);
    return p.step > 1 ? launch_n<T, F8, 1, true>(p, s) : launch_n<T, F8, 1, false>(p, s);
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
