// fd_beam_select.cu -- beam search's selection: of the W * V continuations of
// a request's W beams the K with the largest log probability
//     score_w + x_wv - ln sum_v exp(x_wv),
// ties to the lowest w * V + v.
//
// Memory bounds it: the logits are read once.  Two kernels.
//
// 1. Rows: a warp reads a segment of 2 KB at a time, and keeps the running
//    maximum m and sum s of exp(x - m) of its segments, and each segment's
//    maximum.  No candidate is looked for.
// 2. Top: a CTA a request joins the parts' (m, s) and with them brings the
//    segments' maxima of all its beams to one scale.  The K segments with the
//    largest of them hold the K best continuations: one outside has K others
//    before it, each of which has an element at least as large (or as large,
//    and of a lower index).  Only these K segments are read again.
//
// Across beams the order is decided by sums in two float32 parts, close to 48
// bits, so that only the sum of exponentials is rounded to less: neighbours
// nearer than some 1e-7 may change places, those of one beam never do.
#include "fd_beam.h"
#include "fd_device.cuh"

#include <float.h>
#include <limits.h>

namespace fd {
namespace {

constexpr int ST = SEL_THREADS;
constexpr int SW = ST / 32;
constexpr int SEG_VECS = SEG_BYTES / 16;   // 16-byte vectors of a segment
constexpr int U = SEG_VECS / 32;           // of a lane
constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float minus_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A logit as the definition takes it: NaN is no candidate (-inf), and +inf
// the largest finite value.
__device__ __forceinline__ float sane(float x) { return fminf(fmaxf(x, minus_inf()), FLT_MAX); }

template <typename T> struct Row;
template <> struct Row<float> {
    static constexpr int VE = 4;
    static constexpr uint32_t NONE = 0xff800000u;   // -inf
    __device__ __forceinline__ static uint32_t bits(const float *p) { return __float_as_uint(__ldg(p)); }
};
template <> struct Row<__half> {
    static constexpr int VE = 8;
    static constexpr uint32_t NONE = 0xfc00u;
    __device__ __forceinline__ static uint32_t bits(const __half *p)
    {
        return __ldg(reinterpret_cast<const uint16_t *>(p));
    }
};
template <> struct Row<__nv_bfloat16> {
    static constexpr int VE = 8;
    static constexpr uint32_t NONE = 0xff80u;
    __device__ __forceinline__ static uint32_t bits(const __nv_bfloat16 *p)
    {
        return __ldg(reinterpret_cast<const uint16_t *>(p));
    }
};

// The vector of elements i .. i + VE - 1 of a row, of which only those in
// [first, end) are the row's: the others are -inf and are not read.
template <typename T> __device__ __forceinline__ uint4 load_part(const T *base, long long i, int first, int end)
{
    constexpr int VE = Row<T>::VE;
    uint4 x;
    if (i >= first && i + VE <= end) {
        const uint4 *p = reinterpret_cast<const uint4 *>(base + i);
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "l"(p));
        return x;
    }
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t e[4 / sizeof(T)];
#pragma unroll
        for (int j = 0; j < (int)(4 / sizeof(T)); ++j) {
            const long long at = i + k * (int)(4 / sizeof(T)) + j;
            e[j] = at >= first && at < end ? Row<T>::bits(base + at) : Row<T>::NONE;
        }
        w[k] = sizeof(T) == 4 ? e[0] : e[0] | e[4 / sizeof(T) - 1] << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        x = fmaxf(x, __shfl_xor_sync(FULL_MASK, x, o));
    return x;
}

// A row of logits: its address rounded down to 16 bytes, and where its
// elements lie from there.
template <typename T> struct Place {
    const T *base;
    int first, end;
    __device__ __forceinline__ Place(const SelectParams &p, int r, int w)
    {
        const T *x = static_cast<const T *>(p.logits) + r * p.r_stride + w * p.w_stride;
        first = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
        end = first + p.V;
        base = x - first;
    }
};

__device__ __forceinline__ bool is_live(const SelectParams &p, int row)
{
    return isfinite(p.scores[row]) && !(p.finished && p.finished[row]);
}

template <typename T> __global__ void __launch_bounds__(ST) rows_kernel(const SelectParams p)
{
    constexpr int VE = Row<T>::VE, SEG = SEG_VECS * VE;
    const int row = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!is_live(p, row))
        return;
    const Place<T> at(p, row / p.W, row % p.W);
    float m = minus_inf(), s = 0.f;
    const int s1 = min((part + 1) * p.per_part, p.segs);
    for (int g = part * p.per_part + warp; g < s1; g += SW) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            x[u] = load_part(at.base, (long long)g * SEG + (u * 32 + lane) * VE, at.first, at.end);
        float top = minus_inf();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[VE];
            Elem<T>::widen(x[u], f);
#pragma unroll
            for (int i = 0; i < VE; ++i)
                top = fmaxf(top, f[i]);   // (of a NaN and a number, the number)
        }
        top = fminf(warp_max(top), FLT_MAX);
        if (lane == 0)
            p.seg_max[(long long)row * p.segs + g] = top;
        if (top == minus_inf())
            continue;
        if (top > m) {
            s *= exp2_fast((m - top) * LOG2E);
            m = top;
        }
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[VE];
            Elem<T>::widen(x[u], f);
#pragma unroll
            for (int i = 0; i < VE; ++i)
                sum += exp2_fast((f[i] - m) * LOG2E);
        }
        // a NaN or +inf among them: once more, as the definition takes them
        if (!(sum <= FLT_MAX)) {
            sum = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[VE];
                Elem<T>::widen(x[u], f);
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    sum += exp2_fast((sane(f[i]) - m) * LOG2E);
            }
        }
        s += sum;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        s += __shfl_xor_sync(FULL_MASK, s, o);
    __shared__ float2 warps[SW];
    if (lane == 0)
        warps[warp] = make_float2(m, s);
    __syncthreads();
    if (warp == 0) {
        const float2 v = lane < SW ? warps[lane] : make_float2(minus_inf(), 0.f);
        m = warp_max(v.x);
        s = v.y > 0.f ? v.y * exp2_fast((v.x - m) * LOG2E) : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            s += __shfl_xor_sync(FULL_MASK, s, o);
        if (lane == 0)
            p.part[blockIdx.x] = make_float2(m, s);
    }
}

// ------------------------------------------------------------------ top
// What is compared: a sum of two float32 parts, the larger first, as whole
// numbers in their order, then the lower index.
struct Cand {
    uint64_t key;
    int idx;
    __device__ __forceinline__ bool before(uint64_t k, int i) const { return key > k || (key == k && idx < i); }
};

__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x + 0.f);   // (-0 is 0)
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float unordered(uint32_t b)
{
    return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}

__device__ __forceinline__ uint64_t key_of(float hi, float lo) { return (uint64_t)ordered(hi) << 32 | ordered(lo); }

// A beam's scale: its maximum, and score - ln(sum) in two parts.
struct Base {
    float m, hi, lo;
};

// The key of logit v of a beam, 0 (below every key) where it is no candidate.
__device__ __forceinline__ uint64_t value_key(const Base &b, float v)
{
    // v - m and then the sum with `hi`, each with what its rounding cut off
    const float d = __fsub_rn(v, b.m), t = __fsub_rn(d, v);
    const float dl = __fsub_rn(__fsub_rn(v, __fsub_rn(d, t)), __fadd_rn(b.m, t));
    const float s = __fadd_rn(b.hi, d), z = __fsub_rn(s, b.hi);
    const float sl = __fadd_rn(__fsub_rn(b.hi, __fsub_rn(s, z)), __fsub_rn(d, z));
    const float l = __fadd_rn(sl, __fadd_rn(dl, b.lo));
    const float hi = __fadd_rn(s, l), lo = __fsub_rn(l, __fsub_rn(hi, s));
    return hi >= -FLT_MAX ? key_of(hi, lo) : 0;
}

constexpr int CHUNK = 8 * ST;               // keys that are offered between two looks at the list
constexpr int ROOM = CHUNK + BEAM_MAX_K;

struct Lists {
    Cand a[ROOM];
    Cand b[BEAM_MAX_K * ((ROOM + ST - 1) / ST)];   // a thread's share of `a`, of K threads
    Cand best[ST];
    Cand edge;      // nothing behind it is wanted
    int n, nb;
};

// Adds this thread's candidate to the list (every thread of the warp calls).
__device__ __forceinline__ void offer(Lists &l, uint64_t key, int idx, const Cand &edge)
{
    const bool want = key != 0 && !edge.before(key, idx);
    const unsigned who = __ballot_sync(FULL_MASK, want);
    if (who == 0)
        return;
    const int lane = threadIdx.x & 31;
    int at = 0;
    if (lane == 0)
        at = atomicAdd(&l.n, __popc(who));
    at = __shfl_sync(FULL_MASK, at, 0) + __popc(who & ((1u << lane) - 1));
    if (want)
        l.a[at] = Cand{key, idx};
}

// The first K of the list, in order, and `edge` at the K-th of them (every
// thread of the block calls, the list complete).
__device__ __forceinline__ void prune(Lists &l, int K)
{
    __syncthreads();
    const int n = l.n, tid = threadIdx.x;
    Cand *from = l.a, *to = l.b;
    int have = n;
    if (n > ST) {
        // the K-th of the threads' first ones has K before it or is it
        Cand best = from[tid];
        for (int i = tid + ST; i < n; i += ST)
            if (from[i].before(best.key, best.idx))
                best = from[i];
        l.best[tid] = best;
        if (tid == 0)
            l.nb = 0;
        __syncthreads();
        int rank = 0;
        for (int i = 0; i < ST; ++i)
            rank += l.best[i].before(best.key, best.idx);
        if (rank == K - 1)
            l.edge = best;
        __syncthreads();
        const Cand edge = l.edge;
        for (int i = tid; i < n; i += ST)
            if (!edge.before(from[i].key, from[i].idx))
                to[atomicAdd(&l.nb, 1)] = from[i];
        __syncthreads();
        have = l.nb;
        from = l.b;
        to = l.a;
    }
    for (int i = tid; i < have; i += ST) {
        const Cand c = from[i];
        int rank = 0;
        for (int j = 0; j < have; ++j)
            rank += from[j].before(c.key, c.idx);
        if (rank < K)
            to[rank] = c;
        if (rank == K - 1)
            l.edge = c;
    }
    __syncthreads();
    if (to != l.a && tid < min(have, K))
        l.a[tid] = to[tid];
    if (tid == 0)
        l.n = min(have, K);
    __syncthreads();
}

template <typename T> __global__ void __launch_bounds__(ST) top_kernel(const SelectParams p)
{
    constexpr int VE = Row<T>::VE, SEG = SEG_VECS * VE;
    __shared__ Lists l;
    __shared__ Base base[BEAM_MAX_W];
    __shared__ bool live[BEAM_MAX_W];
    __shared__ int seg[BEAM_MAX_K];   // w * segs + segment
    __shared__ int nsegs;
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row0 = r * p.W;

    // the beams' scales, a warp a beam
    for (int w = warp; w < p.W; w += SW) {
        const int row = row0 + w;
        bool ok = is_live(p, row);
        float m = minus_inf();
        double s = 0.0;
        if (ok) {
            const float2 *part = p.part + (long long)row * p.parts;
            for (int i = lane; i < p.parts; i += 32)
                m = fmaxf(m, part[i].x);
            m = warp_max(m);
            for (int i = lane; i < p.parts; i += 32) {
                const float2 v = part[i];
                if (v.y > 0.f)
                    s += (double)(v.y * expf(v.x - m));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1)
                s += __shfl_xor_sync(FULL_MASK, s, o);
            ok = m > minus_inf();
        }
        if (lane == 0) {
            live[w] = ok;
            if (ok) {
                const double b = (double)p.scores[row] - log(s);
                base[w].m = m;
                base[w].hi = (float)b;
                base[w].lo = (float)(b - (double)base[w].hi);
            }
        }
    }
    if (tid == 0) {
        l.n = 0;
        l.edge = Cand{0, INT_MAX};
    }
    __syncthreads();

    // the K segments with the largest maxima (a segment's index: its first element's)
    const int all = p.W * p.segs;
    for (int g0 = 0; g0 < all; g0 += CHUNK) {
        const Cand edge = l.edge;
#pragma unroll
        for (int u = 0; u < CHUNK / ST; ++u) {
            const int g = g0 + u * ST + tid;
            uint64_t key = 0;
            if (g < all) {
                const int w = g / p.segs;
                if (live[w]) {
                    const float v = p.seg_max[(long long)row0 * p.segs + g];
                    key = v > minus_inf() ? value_key(base[w], v) : 0;
                }
            }
            offer(l, key, g, edge);
        }
        prune(l, p.K);
    }
    const int found = l.n;
    if (tid < found)
        seg[tid] = l.a[tid].idx;
    __syncthreads();
    if (tid == 0) {
        nsegs = found;
        l.n = 0;
        // no element behind the K-th segment's largest is among the first K
        l.edge = Cand{found == p.K ? l.a[p.K - 1].key : 0, INT_MAX};
    }
    __syncthreads();

    // a finished beam continues in one way, at no cost
    if (warp == 0) {
        const bool over = lane < p.W && p.finished && p.finished[row0 + lane];
        const float score = lane < p.W ? p.scores[row0 + lane] : 0.f;
        offer(l, over && isfinite(score) ? key_of(score, 0.f) : 0, lane * p.V + p.eos, Cand{0, INT_MAX});
    }
    const int vecs = nsegs * SEG_VECS;
    for (int v0 = 0; v0 < vecs; v0 += ST) {
        // (as long as the list has room for a vector of every thread)
        __syncthreads();
        if (l.n > ROOM - CHUNK)
            prune(l, p.K);
        const Cand edge = l.edge;
        const int v = v0 + tid;
        float f[VE];
        int first = 0, w = 0;
        if (v < vecs) {
            const int g = seg[v / SEG_VECS];
            w = g / p.segs;
            const Place<T> at(p, r, w);
            const int i = (g - w * p.segs) * SEG + v % SEG_VECS * VE;
            Elem<T>::widen(load_part(at.base, i, at.first, at.end), f);
            first = w * p.V + i - at.first;
        }
        __syncthreads();   // every thread has looked at the list's length
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const float x = v < vecs ? sane(f[i]) : minus_inf();
            offer(l, x > minus_inf() ? value_key(base[w], x) : 0, first + i, edge);
        }
    }
    prune(l, p.K);

    for (int k = tid; k < p.K; k += ST) {
        const bool some = k < l.n;
        const int idx = some ? l.a[k].idx : -1;
        const int parent = some ? idx / p.V : -1, token = some ? idx % p.V : -1;
        const long long to = (long long)r * p.K + k;
        p.out_scores[to] = some ? unordered((uint32_t)(l.a[k].key >> 32)) : minus_inf();
        p.out_parents[to] = parent;
        p.out_tokens[to] = token;
        if (p.out_finished)
            p.out_finished[to] = !some || token == p.eos || (p.finished && p.finished[row0 + parent]);
    }
}

template <typename T> cudaError_t launch_t(const SelectParams &p, cudaStream_t s)
{
    rows_kernel<T><<<(unsigned)(p.R * p.W * p.parts), ST, 0, s>>>(p);
    top_kernel<T><<<p.R, ST, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_select(const SelectParams &p, cudaStream_t s)
{
    return p.dtype == 0   ? launch_t<float>(p, s)
           : p.dtype == 1 ? launch_t<__half>(p, s)
                          : launch_t<__nv_bfloat16>(p, s);
}

}  // namespace fd
