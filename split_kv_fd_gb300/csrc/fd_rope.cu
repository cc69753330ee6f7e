// fd_rope.cu -- new K and V rows into a paged KV cache with the position
// rotation applied to K on the way, and q rotated beside them.
//
// A head's first `rot` elements are rot/2 pairs (x, y), turned by the angle
// that the table gives the token's position: x cos - y sin and y cos + x sin.
// A pair is elements i and i + rot/2, or 2i and 2i + 1 (`pairs`).  Products
// and sum are float32, each rounded to nearest (no fused operation: what an
// element-by-element program computes, bit for bit), and the result is rounded
// once more, to the rows' type, or divided by the scale and rounded to E4M3.
//
// Memory bounds it: every element is read once and written once, and the
// arithmetic is some 3 operations an element.  A thread takes 8 + 8 elements
// of a head, such that both halves of a pair are its own, and the same ones of
// every `hs`-th head, so that its cosines and sines are loaded once a token.
// 16K tokens of 64 query heads and 8 K/V heads of 128, bf16 (637 MB): 100 us,
// 6.3 TB/s.  (More rows a thread at a time, or more tokens a CTA, cost registers
// and so CTAs on an SM: 105-130 us.)  Into E4M3 pages 108, 0.83 of the copy
// bandwidth: 70 registers against 48 leave 7 CTAs on an SM.  A decode step of
// 256 such tokens into E4M3 pages: 5 us, a launch and the loads slot, table and
// offsets wait for.  A CTA takes one token however few its heads are: 16K tokens
// of 8 + 1 heads of 64 take 17 us, three times their bytes' time.
#include "fd_device.cuh"
#include "fd_e4m3.cuh"
#include "fd_pages.h"

namespace fd {
namespace {

constexpr int RT = 128;   // threads of a CTA

// Not through the read-only path: q may be rotated in place.
__device__ __forceinline__ uint4 load_once(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t round2(float a, float b, const float *)
{
    (void)b;
    return __float_as_uint(a);
}
__device__ __forceinline__ uint32_t round2(float a, float b, const __half *)
{
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
}
__device__ __forceinline__ uint32_t round2(float a, float b, const __nv_bfloat16 *)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
}

// 8 elements as they lie in memory.
template <typename T> struct Eight {
    static constexpr int VECS = 8 * (int)sizeof(T) / 16;
    uint4 x[VECS];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < VECS; ++i)
            x[i] = load_once(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void store(T *p) const
    {
#pragma unroll
        for (int i = 0; i < VECS; ++i)
            reinterpret_cast<uint4 *>(p)[i] = x[i];
    }
    __device__ __forceinline__ void widen(float *f) const
    {
#pragma unroll
        for (int i = 0; i < VECS; ++i)
            Elem<T>::widen(x[i], f + i * Elem<T>::VEC);
    }
    __device__ __forceinline__ void round(const float *f)
    {
        uint32_t w[VECS * 4];
#pragma unroll
        for (int i = 0; i < VECS * 4; ++i)
            w[i] = sizeof(T) == 4 ? round2(f[i], 0.f, (const T *)nullptr)
                                  : round2(f[2 * i % 8], f[(2 * i + 1) % 8], (const T *)nullptr);
#pragma unroll
        for (int i = 0; i < VECS; ++i)
            x[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
};

__device__ __forceinline__ void turn(float &x, float &y, float c, float s)
{
    const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = a;
}

// The sequence whose rows cu[b] .. cu[b+1]-1 hold t, or -1: how many of the
// offsets are at or below t, by whole warps, 32 * TESTS of them at a time (a
// bisection would wait for eight loads, one behind the other, of 256 sequences).
__device__ __forceinline__ int sequence_of(const int32_t *cu, int B, int t)
{
    constexpr int TESTS = 16;
    const int lane = threadIdx.x & 31;
    long long lo = 0, n = (long long)B + 1;   // those before lo are, those from lo + n on are not
    for (;;) {
        const long long stride = (n + 32 * TESTS - 1) / (32 * TESTS);
        int below = 0;
#pragma unroll
        for (int k = 0; k < TESTS; ++k) {
            const long long i = (k * 32 + lane + 1) * stride - 1;   // the last of its stretch
            below += i < n && __ldg(cu + lo + i) <= t;
        }
        const long long skip = __reduce_add_sync(FULL_MASK, below) * stride;
        lo += skip;
        if (stride == 1)
            break;
        n = min(n - skip, stride - 1);
        if (n <= 0)
            break;
    }
    return lo >= 1 && lo <= B ? (int)lo - 1 : -1;
}

// A CTA a token, or, with gridDim.y > 1, a share of its heads.
template <typename T, bool F8, bool PAIRS>
__global__ void __launch_bounds__(RT) rope_kernel(const RopeParams p)
{
    const int t = blockIdx.x;
    const int per = p.d / 16;                  // threads of a head: a power of two
    const int j = threadIdx.x & (per - 1), half = p.rot / 2;
    // this thread's elements, e0 and e1 and the 7 behind each, and whether they turn
    int e0 = 16 * j, e1 = 16 * j + 8;
    const bool turns = 16 * j < p.rot;
    if (!PAIRS && turns) {
        e0 = 8 * j;
        e1 = half + 8 * j;
    }
    const int heads = p.Hq + 2 * p.H, hs = RT / per, first = threadIdx.x / per + blockIdx.y * hs;
    Eight<T> x, y;
    auto load = [&](int h) {
        const bool isq = h < p.Hq, isv = h >= p.Hq + p.H;
        const int hk = isq ? h : h - p.Hq - (isv ? p.H : 0);
        const T *from = static_cast<const T *>(isq ? p.q : isv ? p.v : p.k) +
                        t * (isq ? p.q_stride : isv ? p.v_stride : p.k_stride) + (long long)hk * p.d;
        x.load(from + e0);
        y.load(from + e1);
    };
    if (first < heads)
        load(first);   // (before it is known whether and where to it goes)

    const int slot = __ldg(p.slots + t), pos = __ldg(p.positions + t);
    const int b = F8 ? sequence_of(p.cu, p.B, t) : 0;
    if (slot < 0 || b < 0)
        return;
    const bool out = slot >= p.num_slots, off = pos < 0 || pos >= p.max_position;
    if (out || off) {
        if (threadIdx.x == 0 && blockIdx.y == 0)
            atomicOr(p.status, (out ? STATUS_BAD_PAGE : 0u) | (off ? STATUS_BAD_INDEX : 0u));
        return;
    }
    float c[8], s[8];
    if (turns) {
        const float4 *row = reinterpret_cast<const float4 *>(p.table + (long long)pos * p.rot + 8 * j);
        const float4 *sin = reinterpret_cast<const float4 *>(p.table + (long long)pos * p.rot + half + 8 * j);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 a = __ldg(row + i), e = __ldg(sin + i);
            c[4 * i] = a.x, c[4 * i + 1] = a.y, c[4 * i + 2] = a.z, c[4 * i + 3] = a.w;
            s[4 * i] = e.x, s[4 * i + 1] = e.y, s[4 * i + 2] = e.z, s[4 * i + 3] = e.w;
        }
    }
    const long long page = slot / p.page_size, at = slot % p.page_size;
    for (int h = first; h < heads; h += hs * gridDim.y) {
        const bool isq = h < p.Hq, isv = h >= p.Hq + p.H;
        const int hk = isq ? h : h - p.Hq - (isv ? p.H : 0);
        if (h != first)
            load(h);
        const bool turn_it = turns && !isv;
        float f[16];
        if (turn_it || (F8 && !isq)) {
            x.widen(f);
            y.widen(f + 8);
        }
        if (turn_it) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (PAIRS)
                    turn(f[2 * i], f[2 * i + 1], c[i], s[i]);
                else
                    turn(f[i], f[8 + i], c[i], s[i]);
            }
        }
        if (F8 && !isq) {
            uint32_t w[4];
            e4m3_quotients<16>(f, __ldg((isv ? p.v_scale : p.k_scale) + (long long)b * p.H + hk), w);
            uint8_t *to = static_cast<uint8_t *>(isv ? p.v_pages : p.k_pages) +
                          ((page * p.H + hk) * p.page_size + at) * p.d;
            *reinterpret_cast<uint2 *>(to + e0) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2 *>(to + e1) = make_uint2(w[2], w[3]);
            continue;
        }
        if (turn_it) {
            x.round(f);
            y.round(f + 8);
        }
        T *to = isq ? static_cast<T *>(p.q_out) + t * p.q_out_stride + (long long)hk * p.d
                    : static_cast<T *>(isv ? p.v_pages : p.k_pages) + ((page * p.H + hk) * p.page_size + at) * p.d;
        x.store(to + e0);
        y.store(to + e1);
    }
}

template <typename T, bool F8> cudaError_t launch_t(const RopeParams &p, cudaStream_t s)
{
    // Passes of a CTA over a token's heads; shared between CTAs where a CTA a
    // token leaves SMs with fewer than four (one token of 32 + 8 heads 2.9 ->
    // 2.1 us, 256 of 64 + 8 into E4M3 pages 5.2, with twice as many 5.8, with
    // none 7.7).  16K tokens gain nothing (129 us in five shares, 100 in one:
    // each reads the table's row).
    const int passes = (int)((((long long)p.Hq + 2LL * p.H) * (p.d / 16) + RT - 1) / RT);
    const int ctas = 4 * p.sms, share = p.T < ctas ? (ctas + p.T - 1) / p.T : 1;
    const dim3 grid(p.T, passes < share ? passes : share);
    if (p.pairs)
        rope_kernel<T, F8, true><<<grid, RT, 0, s>>>(p);
    else
        rope_kernel<T, F8, false><<<grid, RT, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, cudaStream_t s)
{
    if (p.f8)
        return p.dtype == 0   ? launch_t<float, true>(p, s)
               : p.dtype == 1 ? launch_t<__half, true>(p, s)
                              : launch_t<__nv_bfloat16, true>(p, s);
    return p.dtype == 0   ? launch_t<float, false>(p, s)
           : p.dtype == 1 ? launch_t<__half, false>(p, s)
                          : launch_t<__nv_bfloat16, false>(p, s);
}

}  // namespace fd
