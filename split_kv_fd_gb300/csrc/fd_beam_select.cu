// fd_beam_select.cu -- beam search's selection: of the W * V continuations of
// a request's W beams the K with the largest log probability
//     score_w + x_wv - ln sum_v exp(x_wv),
// ties to the lowest w * V + v.
//
// Memory bounds it: the logits are read once.  Two kernels.
//
// 1. Rows: a warp reads 2 KB of a row at a time, and keeps the running maximum
//    m and sum s of exp(x - m), and the maximum of each segment of 512 bytes.
//    No candidate is looked for.
// 2. Top: a CTA a request joins the parts' (m, s) and with them brings the
//    segments' maxima of all its beams to one scale.  The K segments with the
//    largest of them hold the K best continuations: one outside has K others
//    before it, each of which has an element at least as large (or as large,
//    and of a lower index).  Only some K segments are read again, and the K-th
//    largest maximum is a bound that few of their elements reach.
//
// Sums of exponentials and their logarithm are float32, the parts' sums joined
// with what rounding cuts off: off by less than (90 + 2.25 ln V) 2^-24 together
// (derived beside the tests), 2e-7 on ordinary rows and 1e-6 at most measured.
// More would cost the rows' kernel instructions, of which it has none to spare.
// That error is a beam's as a whole: what its candidates add to it are sums in
// two float32 parts, close to 48 bits, so neighbours of two beams nearer than
// twice the error may change places, those of one beam do not.
//
// 64 requests of 8 beams over 131072 tokens, bf16, a tenth of them finished (121
// MB): 30 us, of which the rows take some 23 (a bare read of as many bytes
// 20.5) and the top 7; 32 of 4 over 128000 in float32 (66 MB) 17.7, 12.6 and 5;
// one of 4 over 32000 6, where both are chains of dependent steps.  Constant
// rows, which pass the bound whole, take the slower way: 4 x 32000 22 us.
#include "fd_beam.h"
#include "fd_device.cuh"

#include <float.h>
#include <limits.h>

namespace fd {
namespace {

constexpr int ST = SEL_THREADS;
constexpr int SW = ST / 32;
constexpr int SEG_VECS = SEG_BYTES / 16;   // 16-byte vectors of a segment, one a lane
static_assert(SEG_VECS == 32, "a warp reads a segment with one load");
constexpr int U = SEL_SEGS;                // segments that a warp reads at a time
constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float minus_inf() { return __int_as_float(0xff800000); }

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

__device__ __forceinline__ uint4 load_vec(const uint4 *p)
{
    uint4 x;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "l"(p));
    return x;
}

// The vector of elements i .. i + VE - 1 of a row, of which only those in
// [first, end) are the row's: the others are -inf and are not read.
template <typename T> __device__ __forceinline__ uint4 load_part(const T *base, int i, int first, int end)
{
    constexpr int VE = Row<T>::VE;
    if (i >= first && i + VE <= end)
        return load_vec(reinterpret_cast<const uint4 *>(base + i));
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t e[4 / sizeof(T)];
#pragma unroll
        for (int j = 0; j < (int)(4 / sizeof(T)); ++j) {
            const int at = i + k * (int)(4 / sizeof(T)) + j;
            e[j] = at >= first && at < end ? Row<T>::bits(base + at) : Row<T>::NONE;
        }
        w[k] = sizeof(T) == 4 ? e[0] : e[0] | e[4 / sizeof(T) - 1] << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float warp_max(float x)
{
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// The largest element of a vector (of a NaN and a number, the number).
__device__ __forceinline__ float vec_max(const uint4 &x, const float *)
{
    return fmaxf(fmaxf(__uint_as_float(x.x), __uint_as_float(x.y)), fmaxf(__uint_as_float(x.z), __uint_as_float(x.w)));
}
template <typename T2> __device__ __forceinline__ T2 max2(uint32_t a, uint32_t b)
{
    T2 x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    return __hmax2(x, y);
}
__device__ __forceinline__ float vec_max(const uint4 &x, const __half *)
{
    const float2 f = __half22float2(__hmax2(max2<__half2>(x.x, x.y), max2<__half2>(x.z, x.w)));
    return fmaxf(f.x, f.y);
}
__device__ __forceinline__ float vec_max(const uint4 &x, const __nv_bfloat16 *)
{
    const float2 f = __bfloat1622float2(__hmax2(max2<__nv_bfloat162>(x.x, x.y), max2<__nv_bfloat162>(x.z, x.w)));
    return fmaxf(f.x, f.y);
}

// Element e of a vector (chosen, not indexed: it lies in registers).
__device__ __forceinline__ uint32_t word_of(const uint4 &x, int i)
{
    return i < 2 ? (i == 0 ? x.x : x.y) : i == 2 ? x.z : x.w;
}
__device__ __forceinline__ float element(const uint4 &x, int e, const float *)
{
    return __uint_as_float(word_of(x, e));
}
__device__ __forceinline__ float element(const uint4 &x, int e, const __half *)
{
    return __half2float(__ushort_as_half((unsigned short)(word_of(x, e >> 1) >> (e & 1) * 16)));
}
__device__ __forceinline__ float element(const uint4 &x, int e, const __nv_bfloat16 *)
{
    const uint32_t w = word_of(x, e >> 1);
    return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
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

// 16 bytes of a row to this thread's own place in shared memory.
__device__ __forceinline__ void copy_ahead(uint4 *to, const uint4 *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All copies but those of the last N groups have landed.
template <int N> __device__ __forceinline__ void copies_landed()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp a part of a row, U segments at a time.  Those that lie within the row
// are copied AHEAD of their turn, each 16 bytes by the thread that takes
// them: no thread waits for another, and what is under way costs no register.
template <typename T> __global__ void __launch_bounds__(ST, SEL_CTAS) rows_kernel(const SelectParams p)
{
    constexpr int VE = Row<T>::VE, SEG = SEG_VECS * VE, STAGES = SEL_STAGES, AHEAD = STAGES - 1;
    extern __shared__ uint4 stages[];   // [warp][stage][U][lane]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned me = blockIdx.x * SW + warp, row = me / p.parts, r = row / p.W;
    const int part = (int)(me - row * p.parts);
    if (row >= (unsigned)p.R * p.W)
        return;
    const Place<T> at(p, (int)r, (int)(row - r * p.W));
    float *seg_max = p.seg_max + (long long)row * p.segs;
    uint4 *mine = stages + warp * STAGES * U * 32 + lane;
    const uint4 *from = reinterpret_cast<const uint4 *>(at.base) + lane;
    const int g0 = (part * p.reads + min(part, p.longer)) * U;
    const int g1 = min(g0 + (p.reads + (part < p.longer)) * U, p.segs);
    auto within = [&](int g) { return g < g1 && g * SEG >= at.first && (g + U) * SEG <= at.end; };
    auto ahead = [&](int g, int stage) {
        if (within(g)) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                copy_ahead(mine + (stage * U + u) * 32, from + (g + u) * SEG_VECS);
        }
        copies_issued();
    };
    // A beam that has ended is not read, so its flag is waited for (one request
    // of 4 beams 6.0 us, 5.9 with the first reads ahead of it); the score is not,
    // rows without one may be read.
    const float score = p.scores[row];
    if (p.finished && p.finished[row])
        return;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        ahead(g0 + i * U, i);
    if (!isfinite(score)) {
        copies_landed<0>();
        return;
    }

    float m = minus_inf(), s = 0.f;
    int stage = 0;
    for (int g = g0; g < g1; g += U) {
        const int next = stage == 0 ? AHEAD : stage - 1;   // the stage that was taken last
        ahead(g + AHEAD * U, next);
        copies_landed<AHEAD>();
        uint4 x[U];
        if (within(g)) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                x[u] = mine[(stage * U + u) * 32];
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                x[u] = load_part(at.base, (g + u) * SEG + lane * VE, at.first, at.end);
        }
        stage = stage == AHEAD ? 0 : stage + 1;
        float top = minus_inf(), seg = top;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float t = warp_max(vec_max(x[u], (const T *)nullptr));
            seg = lane == u ? t : seg;
            top = fmaxf(top, t);
        }
        if (lane < U && g + lane < p.segs)
            seg_max[g + lane] = sane(seg);
        top = fminf(top, FLT_MAX);
        if (top == minus_inf())
            continue;
        if (top > m) {
            s *= ex2((m - top) * LOG2E);
            m = top;
        }
        // exp(x - m), two at a time
        const uint64_t minus_m = pack2(-m, -m), scale = pack2(LOG2E, LOG2E);
        uint64_t sum2 = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[VE];
            Elem<T>::widen(x[u], f);
#pragma unroll
            for (int i = 0; i < VE; i += 2) {
                float a, b;
                unpack2(mul2(add2(pack2(f[i], f[i + 1]), minus_m), scale), a, b);
                sum2 = add2(sum2, pack2(ex2(a), ex2(b)));
            }
        }
        float a, b;
        unpack2(sum2, a, b);
        float sum = a + b;
        if (!(sum <= FLT_MAX)) {   // a NaN or +inf among them: once more, as the definition takes them
            sum = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[VE];
                Elem<T>::widen(x[u], f);
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    sum += ex2((sane(f[i]) - m) * LOG2E);
            }
        }
        s += sum;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        s += __shfl_xor_sync(FULL_MASK, s, o);
    if (lane == 0)
        p.part[me] = make_float2(m, s);
}

// ------------------------------------------------------------------ top
// What is compared: a sum of two float32 parts, the larger first, as whole
// numbers in their order, then the lower index.
struct Cand {
    uint64_t key;
    int idx;
    // (no branch: loops of it keep their loads on the way)
    __device__ __forceinline__ bool before(uint64_t k, int i) const { return (key > k) | ((key == k) & (idx < i)); }
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
constexpr int MAX_SEGS = 1024;              // segments that are looked through without a second thought

struct Lists {
    Cand a[ROOM];
    Cand b[BEAM_MAX_K * ((ROOM + ST - 1) / ST)];   // a thread's share of `a`, of K threads
    Cand best[ST];
    Cand edge;      // nothing behind it is wanted
    int n, nb;
};
static_assert(sizeof(Cand[BEAM_MAX_K * ((ROOM + ST - 1) / ST)]) >= MAX_SEGS * sizeof(int), "the segments lie in `b`");

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
#pragma unroll 8
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
#pragma unroll 8
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

// ln(s + e) in two parts, e what rounding cut off s: s = 2^k f with f in
// [0.75, 1.5), k ln 2 by two parts of ln 2, of which the first has so few bits
// that its product is exact (Cody and Waite), and ln f, whose half step is
// 2^-26 there.
__device__ __forceinline__ void log2parts(float s, float e, float &hi, float &lo)
{
    const int k = (__float_as_int(s) - 0x3f400000) >> 23;
    const float f = __int_as_float(__float_as_int(s) - (k << 23));
    constexpr float LN2_HI = 0x1.62e4p-1f, LN2_LO = (float)(0.693147180559945309417 - 0x1.62e4p-1);
    const float a = (float)k * LN2_HI, b = logf(f);
    hi = a + b;
    const float z = hi - a;
    lo = (a - (hi - z)) + (b - z) + ((float)k * LN2_LO + __fdividef(e, s));
}

// The K best where the bound leaves too many: the list is pruned whenever it
// is full.  (Every thread of the block calls.)
template <typename T>
__device__ __noinline__ void top_of_many(const SelectParams &p, Lists &l, const Base *base, int *seg)
{
    constexpr int VE = Row<T>::VE, SEG = SEG_VECS * VE;
    const int r = blockIdx.x, tid = threadIdx.x;
    const long long row0 = (long long)r * p.W;
    __syncthreads();
    if (tid == 0) {
        l.n = 0;
        l.edge = Cand{0, INT_MAX};
    }
    __syncthreads();
    // the K segments with the largest maxima (a segment's index stands for its first element's)
    const int all = p.W * p.segs;
    for (int g0 = 0; g0 < all; g0 += CHUNK) {
        const Cand edge = l.edge;
#pragma unroll 1
        for (int u = 0; u < CHUNK / ST; ++u) {
            const int g = g0 + u * ST + tid;
            uint64_t key = 0;
            if (g < all) {
                const int w = g / p.segs;
                if (isfinite(base[w].m)) {
                    const float v = p.seg_max[row0 * p.segs + g];
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
        l.n = 0;
        // no element behind the K-th segment's largest is among the first K
        l.edge = Cand{found == p.K ? l.a[p.K - 1].key : 0, INT_MAX};
    }
    __syncthreads();
    const int vecs = found * SEG_VECS;
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
}

// A request's k-th continuation: c, or none.  `ended`: the finished beams.
__device__ __forceinline__ void emit(const SelectParams &p, int k, bool some, const Cand &c, unsigned ended)
{
    const long long to = (long long)blockIdx.x * p.K + k;
    const int parent = some ? c.idx / p.V : -1, token = some ? c.idx - parent * p.V : -1;
    p.out_scores[to] = some ? unordered((uint32_t)(c.key >> 32)) : minus_inf();
    p.out_parents[to] = parent;
    p.out_tokens[to] = token;
    if (p.out_finished)
        p.out_finished[to] = !some || token == p.eos || (ended >> parent & 1);
}

template <typename T> __global__ void __launch_bounds__(ST) top_kernel(const SelectParams p)
{
    constexpr int VE = Row<T>::VE, SEG = SEG_VECS * VE;
    constexpr int HELD = 16;          // maxima that a thread holds
    __shared__ __align__(16) Lists l;
    __shared__ Base base[BEAM_MAX_W];
    __shared__ __align__(16) float tops[ST];
    __shared__ int seg[BEAM_MAX_K];   // w * segs + segment
    __shared__ int nsegs;
    __shared__ unsigned bound, spread;
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row0 = (long long)r * p.W;
    Cand *few = l.best;               // the candidates, where the bound leaves no more than FEW
    constexpr int FEW = ST;
    // (scores and flags are older than the rows' kernel)
    bool over = false;
    float score = 0.f;
    if (lane < p.W) {
        score = p.scores[row0 + lane];
        over = p.finished && p.finished[row0 + lane];
    }
    const bool ends = over && isfinite(score);
    const unsigned ended = __ballot_sync(FULL_MASK, over);
    // a finished beam continues in one way, at no cost
    const unsigned ending = __ballot_sync(FULL_MASK, ends);
    if (warp == 0 && ends)
        few[__popc(ending & ((1u << lane) - 1))] = Cand{key_of(score, 0.f), lane * p.V + p.eos};
    if (tid == 0) {
        l.n = __popc(ending);
        nsegs = 0;
        bound = ~0u;
        spread = 0;
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // The scales, a warp a beam; the segments' maxima are on their way
    // meanwhile.
    const int all = p.W * p.segs;
    const float *seg_max = p.seg_max + row0 * p.segs;
    float v[HELD];
    auto load_maxima = [&] {
#pragma unroll
        for (int u = 0; u < HELD; ++u)
            v[u] = u * ST + tid < all ? seg_max[u * ST + tid] : minus_inf();
    };
    if (warp >= p.W)
        load_maxima();
    for (int w = warp; w < p.W; w += SW) {
        const float sc = __shfl_sync(FULL_MASK, score, w);
        const bool done = __shfl_sync(FULL_MASK, (int)over, w);
        float m = minus_inf(), s = 0.f, e = 0.f;
        const bool counts = isfinite(sc) && !done;
        const float2 *part = p.part + (row0 + w) * p.parts;
        float2 x[4];   // (as many as most rows have, loaded at once)
#pragma unroll
        for (int u = 0; u < 4; ++u)
            x[u] = counts && u * 32 + lane < p.parts ? part[u * 32 + lane] : make_float2(minus_inf(), 0.f);
        if (w == warp)
            load_maxima();
        if (counts) {
            float mine = fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x));
            for (int i = 128 + lane; i < p.parts; i += 32)
                mine = fmaxf(mine, part[i].x);
            m = warp_max(mine);
            // the sum with what its roundings cut off: a row of 2^29 has 2048
            // parts a lane, which a plain one may leave 3e-5 off
            auto plus = [&](float x) {
                const float t = s + x, z = t - s;
                e += (s - (t - z)) + (x - z);
                s = t;
            };
#pragma unroll
            for (int u = 0; u < 4; ++u)
                plus(x[u].y > 0.f ? __fmul_rn(x[u].y, expf(x[u].x - m)) : 0.f);
            for (int i = 128 + lane; i < p.parts; i += 32) {
                const float2 y = part[i];
                plus(y.y > 0.f ? __fmul_rn(y.y, expf(y.x - m)) : 0.f);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const float x = __shfl_xor_sync(FULL_MASK, s, o);
                e += __shfl_xor_sync(FULL_MASK, e, o);
                plus(x);
            }
        }
        if (lane == 0) {
            Base b = {__int_as_float(0x7f800000), 0.f, 0.f};   // m = inf: no element is a candidate
            if (m > minus_inf()) {
                float hi, lo;
                log2parts(s, e, hi, lo);
                b.m = m;
                b.hi = sc - hi;
                const float z = b.hi - sc;
                b.lo = ((sc - (b.hi - z)) + (-hi - z)) - lo;
                atomicMax(&spread, __float_as_uint(fabsf(b.hi) * 0.5f + fabsf(m) * 0.5f));
            }
            base[w] = b;
        }
    }
    __syncthreads();

    // All maxima on one scale, roughly.  (What no beam wrote gives -inf or
    // NaN, and is not taken.)
    const int dw = ST / p.segs, di = ST - dw * p.segs;   // a thread's step through beams and segments
    int w = tid / p.segs, i = tid - w * p.segs;
    float top = minus_inf();
#pragma unroll
    for (int u = 0; u < HELD; ++u) {
        if (u * ST + tid < all) {
            v[u] = (v[u] - base[w].m) + base[w].hi;
            top = fmaxf(top, v[u]);
            w += dw;
            if ((i += di) >= p.segs)
                i -= p.segs, ++w;
        }
    }
    const int w1 = w, i1 = i;
    for (int g = HELD * ST + tid; g < all; g += ST) {
        top = fmaxf(top, (seg_max[g] - base[w].m) + base[w].hi);
        w += dw;
        if ((i += di) >= p.segs)
            i -= p.segs, ++w;
    }
    // The K-th largest of the largest ones of groups of four threads: K
    // segments, and so K elements, reach it.  (Of single threads where K is
    // more than half of the groups, whose last ones lie far down.)
    const bool four = p.K <= ST / 8;
    if (four) {
        top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 1));
        top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 2));
    }
    if (!four || (lane & 3) == 0)
        tops[four ? tid / 4 : tid] = top;
    __syncthreads();
    {
        int larger[4] = {0, 0, 0, 0};
        const float4 *t4 = reinterpret_cast<const float4 *>(tops);
        const int n = four ? ST / 16 : ST / 4;
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float4 t = t4[i];
            larger[0] += t.x > top;
            larger[1] += t.y > top;
            larger[2] += t.z > top;
            larger[3] += t.w > top;
        }
        const bool in = (larger[0] + larger[1]) + (larger[2] + larger[3]) < p.K;
        const unsigned lowest = __reduce_min_sync(FULL_MASK, in ? ordered(top) : ~0u);
        if (lane == 0 && lowest != ~0u)
            atomicMin(&bound, lowest);
    }
    __syncthreads();
    // ... less what these sums may be off, some steps of each of their terms
    const float kth = unordered(bound), size = __uint_as_float(spread);
    const float thr = (kth - 0x1p-19f * fabsf(kth)) - 0x1p-18f * size;
    int *list = reinterpret_cast<int *>(l.b);
    unsigned wanted = 0;
#pragma unroll
    for (int u = 0; u < HELD; ++u)
        wanted |= (v[u] >= thr && v[u] > minus_inf()) << u;
    auto add = [&](int g) {
        const int to = atomicAdd(&nsegs, 1);
        const int w = g / p.segs;
        if (to < MAX_SEGS)
            list[to] = w << 24 | (g - w * p.segs);
    };
    for (; wanted; wanted &= wanted - 1)
        add((__ffs(wanted) - 1) * ST + tid);
    if (all > HELD * ST) {
        w = w1, i = i1;
        for (int g = HELD * ST + tid; g < all; g += ST) {
            const float x = (seg_max[g] - base[w].m) + base[w].hi;
            if (x >= thr && x > minus_inf())
                add(g);
            w += dw;
            if ((i += di) >= p.segs)
                i -= p.segs, ++w;
        }
    }
    __syncthreads();
    const int found = nsegs;
    if (found <= MAX_SEGS) {
        // A batch of segments' vectors, each to its thread's own place, all of
        // them on their way before the first is looked at.
        uint4 *stage = reinterpret_cast<uint4 *>(l.a);
        constexpr int BATCH = sizeof(l.a) / (ST * 16) * ST;
        const int vecs = found * SEG_VECS;
        auto place = [&](int k, int &w, int &i) {
            const int g = list[k / SEG_VECS];
            w = g >> 24;
            i = (g & 0xffffff) * SEG + k % SEG_VECS * VE;
            return Place<T>(p, r, w);
        };
        for (int k0 = 0; k0 < vecs; k0 += BATCH) {
            const int end = min(vecs, k0 + BATCH);
            int w, i;
#pragma unroll 1
            for (int k = k0 + tid; k < end; k += ST) {
                const Place<T> at = place(k, w, i);
                if (i >= at.first && i + VE <= at.end)
                    copy_ahead(stage + (k - k0), reinterpret_cast<const uint4 *>(at.base + i));
                else
                    stage[k - k0] = load_part(at.base, i, at.first, at.end);
            }
            copies_issued();
            copies_landed<0>();
#pragma unroll 1
            for (int k = k0 + tid; k < end; k += ST) {
                if (*(volatile int *)&l.n > FEW)
                    break;   // it is the slower way
                const Place<T> at = place(k, w, i);
                const uint4 x = stage[k - k0];
                const Base b = base[w];
                const float need = thr - b.hi;
                const float limit = (b.m + need) - (0x1p-20f * fabsf(b.m) + 0x1p-20f * fabsf(need));
                unsigned some = 0;
                float f[VE];
                Elem<T>::widen(x, f);
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    some |= (f[e] >= limit && f[e] > minus_inf()) << e;
                for (; some && *(volatile int *)&l.n <= FEW; some &= some - 1) {
                    const int e = __ffs(some) - 1;
                    const uint64_t key = value_key(b, sane(element(x, e, (const T *)nullptr)));
                    const int to = key ? atomicAdd(&l.n, 1) : FEW;
                    if (to < FEW)
                        few[to] = Cand{key, w * p.V + i + e - at.first};
                }
            }
        }
    }
    __syncthreads();
    const int n = l.n;
    if (found <= MAX_SEGS && n <= FEW) {
        // eight threads a candidate: how many are before it
        for (int i0 = 0; i0 < n; i0 += ST / 8) {
            const int i = i0 + tid / 8;
            const Cand c = few[min(i, n - 1)];
            int rank = 0;
#pragma unroll 4
            for (int j = tid & 7; j < n; j += 8)
                rank += few[j].before(c.key, c.idx);
#pragma unroll
            for (int o = 4; o; o >>= 1)
                rank += __shfl_xor_sync(FULL_MASK, rank, o);
            if ((tid & 7) == 0 && i < n && rank < p.K)
                emit(p, rank, true, c, ended);
        }
        if (tid >= n && tid < p.K)
            emit(p, tid, false, Cand{0, 0}, ended);
        return;
    }
    top_of_many<T>(p, l, base, seg);
    if (warp == 0)   // the finished beams, behind the others
        offer(l, ends ? key_of(score, 0.f) : 0, lane * p.V + p.eos, Cand{0, INT_MAX});
    prune(l, p.K);
    if (tid < p.K)
        emit(p, tid, tid < l.n, l.a[tid], ended);
}

template <typename T> cudaError_t launch_t(const SelectParams &p, cudaStream_t s)
{
    const long long warps = (long long)p.R * p.W * p.parts;
    constexpr int smem = ST * SEL_STAGES * U * 16;
    static_assert(smem <= 48 * 1024, "no attribute is set");
    rows_kernel<T><<<(unsigned)((warps + SW - 1) / SW), ST, smem, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    // its CTAs start while the rows' last ones end
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.R);
    cfg.blockDim = dim3(ST);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, top_kernel<T>, p);
}

}  // namespace

cudaError_t launch_select(const SelectParams &p, cudaStream_t s)
{
    return p.dtype == 0   ? launch_t<float>(p, s)
           : p.dtype == 1 ? launch_t<__half>(p, s)
                          : launch_t<__nv_bfloat16>(p, s);
}

}  // namespace fd
