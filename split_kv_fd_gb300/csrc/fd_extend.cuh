// fd_extend.cuh -- attention with several new tokens a sequence on the
// fifth-generation tensor cores: token i of a sequence's n new ones over m
// keys sees the keys below m - n + i + 1 (causal) or all m,
//     out = softmax(scale q K^T) V,   lse = ln sum exp(scale q K^T).
//
// The MMA rows of a sub-tile are 128 (token, query head) pairs of one K/V
// head, so every K/V block serves the whole group of query heads; a tile is
// two sub-tiles.  For each block of 128 keys and sub-tile
//     S [128 x 128] = Q [128 x d] . K^T      (both in shared memory)
//     O [128 x d]  += P [128 x 128] . V      (P in tensor memory)
// with the online softmax between them in float32 registers, one thread a
// row: the reference maximum of a row moves only when a block's maximum
// passes it by more than TAU (base 2), and only then are its sum and its O
// row rescaled; P may reach 2^TAU meanwhile, and the quotient is the same.
// P is rounded to the inputs' 16-bit type for the product with V (half a
// step of each weight), sums of weights stay float32 and unrounded.
//
// Two engines, each with a warpgroup of softmax and S, P and O of its own in
// tensor memory, keep the tensor cores busy by turns: engine x takes
// sub-tile x, both on the same K/V blocks.  Where a tile has only one
// sub-tile (a few drafted tokens), the engines share it instead: engine x
// takes every other block and the two results are joined at the end, so
// that the time of a block is half that of the chain S, softmax, P.V.
//
// Sums over more than EXT_LINK blocks are taken in links, each a segment of
// its own, joined in the CTA's two slots of the workspace (ext_join).
//
// P lies in the columns of its S, and S of an engine's next block follows
// P.V of the one before, so S's commit also says that P.V is done.  (At
// d = 64 there is room for P beside S; with S of the next block issued as
// soon as the softmax had read this one, both engines fell into step on the
// special-function units: 373 us against 325 for 8192 tokens of 32 heads.)
//
// Warp roles (384 threads, 512 for E4M3 K/V, one CTA per SM):
//  - warps 0-3, 4-7: softmax and results of engines 0 and 1;
//  - warp 8: K and V by tensor-map TMA into one ring;
//  - warp 9: allocates TMEM, issues every MMA, engine 0's and engine 1's by
//    turns (a warp for each engine let them fall into step on the
//    special-function units: 3050 us against 2590 for 16384 tokens of 64
//    heads);
//  - warp 10: Q by TMA, as soon as a sub-tile's last S is done;
//  - warp 11: walks the CTA's share of the plan, segments into a small ring;
//  - E4M3 only, warps 12-15: widen the blocks that warp 8 copied as they are
//    to f16 (exact: E4M3 has 4 significant bits and exponents from -9 to 8)
//    for the same products.  A bf16 Q becomes f16 too, each row brought to
//    a maximum in [2^8, 2^9) by a power of two that its scores undo: exact
//    but for elements 2^22 times smaller than that.  The K scale is part of
//    the score's, the V scale of the result's.
// Every hand-off is an mbarrier, and every wait is bounded (ext_wait_ns): on
// expiry a role records FD_ERR_DEVICE_TIMEOUT, stops, waits for the copies it
// issued, and the CTA frees its TMEM.  A role that waits by parity waits for
// every phase of its barrier, or one that it cannot fall two behind of.
//
// What bounds it, and what it measured (one GB300, device times; cuBLAS and
// a copy reach 1889 TFLOP/s and 6794 GB/s):
//  - long prompts and chunks at d = 128: the tensor cores; 16001 tokens of
//    64 heads on 8, bf16: 2236-2270 us, 1850-1880 TFLOP/s; f16 chunks of 2048
//    tokens over 16K-30K keys 1790-1840.  In a loop the power cap holds it to
//    1640 and 1560, 0.97 and 0.92 of the sustained cuBLAS rate;
//  - d = 64: the chain of a block, S, maximum, 128 exponentials a row, P.V
//    (2475 cycles a pair of blocks): 8192 tokens of 32 heads 281-286 us,
//    962-978; over an E4M3 cache 773 (2 x 2048 tokens over 4096);
//  - few new tokens over a long 16-bit cache: memory; 32 sequences of 8
//    tokens over 4K-32K keys, 64 heads on 8: 322-327 us, 6.6 TB/s;
//  - E4M3 caches: shared memory, 224 KB a block of 128 keys in some 2400
//    cycles: 16 sequences of 5 tokens 139 us, 3545 GB/s; 2 x 2048 tokens
//    over 4096 539 us, 1275 TFLOP/s;
//  - short and packed prompts: the ends of items.  A CTA's last block, the
//    drain of P.V and the result take some 9000 cycles beside the next
//    item's start: 20K tokens in 9 prompts 382-407 us, 1345-1430 TFLOP/s.
#pragma once

#include "fd_extend.h"
#include "fd_extend_ops.cuh"

namespace fd {

// T: the type of the MMAs (f16 for E4M3 K/V).
template <typename T, int D, bool F8> struct ExtCfg {
    static constexpr int M = EXT_M, CT = EXT_CT;
    static constexpr int PLANES = D / 64;                // 128-byte planes of a row
    static constexpr int PLANE = CT * 128;               // one plane of a block, or of a sub-tile's Q
    static constexpr int BLOCK_BYTES = PLANES * PLANE;   // K or V of one block
    static constexpr int Q_BYTES = PLANES * PLANE;       // one sub-tile
    // 16-bit K and V: 160 KB of copies in flight.  E4M3: the copies land in
    // a ring of raw blocks of 64 KB, all that three stages of widened ones
    // leave (two or four stages are slower at long or at few queries).
    static constexpr int STAGES = (F8 ? 3 : 5) * (128 / D);
    static constexpr int RAW_BYTES = CT * D;             // an E4M3 block
    static constexpr int RAWS = F8 ? 4 * (128 / D) : 0;
    static constexpr int SEGS = 3;                       // segments the scheduler runs ahead
    static constexpr int KV_WARP = 8, MMA_WARP = 9, Q_WARP = 10, SCHED_WARP = 11, CVT_WARP = 12;
    static constexpr int CVT_WARPS = 4;
    static constexpr int THREADS = F8 ? 384 + 32 * CVT_WARPS : 384;
    // registers a thread: the softmax warpgroups hold a row of S each; the
    // shares fit the launch's (168 x 384 and 128 x 512)
    static constexpr int REGS_SOFTMAX = F8 ? 184 : 208, REGS_OTHER = F8 ? 72 : 88;
    static_assert(2 * REGS_SOFTMAX + (THREADS / 128 - 2) * REGS_OTHER <= (F8 ? 4 * 128 : 3 * 168), "register shares");
    // TMEM columns: S and O of both engines, P in the first half of its S
    static constexpr int TM_O = 2 * CT;
    __host__ __device__ static constexpr int tm_s(int x) { return x * CT; }
    __host__ __device__ static constexpr int tm_o(int x) { return TM_O + x * D; }
    __host__ __device__ static constexpr int tm_p(int x) { return x * CT; }
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr float TAU = 8.f;
    // f16 weights carry a factor 2^7 (the sum does too): below 2^-14 an f16
    // loses bits, above 2^16 it overflows, and 2^(TAU + 7) stays below that.
    // bf16 has float32's range and needs none.
    static constexpr float SHIFT = std::is_same<T, __half>::value ? 7.f : 0.f;
    static constexpr uint32_t SLEEP_NS = 100000;
    // P is handed over in two parts, so that the product of the first with V
    // runs while the softmax computes the second (measured for 16384 tokens
    // of 64 heads: 64 + 64 keys 2340 us, 32 + 96 2385, 96 + 32 2420; all 128
    // at once 2424).
    static constexpr int PART = 64;
    // barriers: ring full/empty; S full, both parts of P, O, Q
    // full, Q empty, Q widened of each engine or sub-tile; the engines'
    // meeting, the last commit; segments full/empty; raw ring full/empty
    static constexpr int NBAR = 2 * STAGES + 14 + 2 + 2 * SEGS + 2 * RAWS;
    static constexpr int XCH_BYTES = 2 * M * 8;          // (reference, sum) of both engines' rows
    static constexpr int QEXP_BYTES = F8 ? 2 * 2 * M : 0;   // exponents of Q's rows, two in flight
    static constexpr int SMEM = STAGES * BLOCK_BYTES + RAWS * RAW_BYTES + 2 * Q_BYTES + NBAR * 8 + 16 + SEGS * 56 +
                                XCH_BYTES + QEXP_BYTES;
    static_assert(SMEM <= 232448, "shared memory");
};

// What the roles of a CTA need to know of a segment: a range of K/V blocks
// of one item.
struct ExtSeg {
    int valid;
    int row0, ntok;      // the tile's first row of q and out, its tokens
    int h, slice, b;
    int m, lim, k0;
    int blk0, end0, end1;   // blocks [blk0, end x) of sub-tile x
    int flags;           // see below
    int slot;            // partial result, or -1: the whole item
    __device__ __forceinline__ int end(int x) const { return x ? end1 : end0; }
    // one sub-tile, its blocks dealt to both engines
    __device__ __forceinline__ bool twin() const { return flags & 1; }
    // a link of a chain (the first, one between, the last), or none of one
    enum { ALONE, FIRST, INNER, LAST };
    __device__ __forceinline__ int link() const { return (flags >> 1) & 3; }
    // where the chain's result goes, as `slot`
    __device__ __forceinline__ int target() const { return flags >> 3; }
};

__device__ __forceinline__ int ext_blocks(const ExtSeg &g) { return max(g.end0, g.end1) - g.blk0; }

// The order of a segment's n blocks in the ring: K(0), V(0), K(1), V(1), ...,
// or with K one block ahead (S of the next block is wanted before P.V of
// this one) K(0), K(1), V(0), K(2), V(1), ..., V(n-1).
struct ExtOrder {
    bool ahead;
    int n;
    // Item t of 2n is V (or K) of block i.
    __device__ __forceinline__ bool item(int t, int &i) const
    {
        if (!ahead || t == 0 || t == 2 * n - 1) {
            i = t >> 1;
            return t & 1;
        }
        i = (t & 1) ? (t + 1) >> 1 : (t >> 1) - 1;
        return !(t & 1);
    }
};

// 32 bytes at a 32-byte aligned address in one store.
__device__ __forceinline__ void stg256(void *ptr, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(ptr), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 32 consecutive outputs from index idx (a multiple of 32) of a
// 16-byte aligned tensor.  A thread writes its own row, so a store touches
// as many lines as the warp has rows whatever its width: 32-byte stores (a
// whole sector each) where the tensor allows them.
__device__ __forceinline__ void store_out32(void *out, long long idx, int out_dtype, const float *x)
{
    char *at = static_cast<char *>(out) + idx * (out_dtype == 0 ? 4 : 2);
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    const int step = out_dtype == 0 ? 8 : 16;   // elements of 32 bytes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i * step >= 32)
            break;
        uint32_t w[8];
        if (out_dtype == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = __float_as_uint(x[8 * i + e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = x[(16 * i + 2 * e) & 31], b = x[(16 * i + 2 * e + 1) & 31];
                w[e] = out_dtype == 1 ? Mma<__half>::pack(a, b) : Mma<__nv_bfloat16>::pack(a, b);
            }
        }
        if (wide) {
            stg256(at + 32 * i, w);
        } else {
            uint4 *o = reinterpret_cast<uint4 *>(at + 32 * i);
            o[0] = make_uint4(w[0], w[1], w[2], w[3]);
            o[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

// 16 E4M3 values as f16, exactly: two 16-byte vectors.
__device__ __forceinline__ void e4m3_widen16(const uint4 &u, uint4 &lo, uint4 &hi)
{
    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(r[2 * i]), "=r"(r[2 * i + 1])
            : "r"(in[i]));
    }
    lo = make_uint4(r[0], r[1], r[2], r[3]);
    hi = make_uint4(r[4], r[5], r[6], r[7]);
}

__device__ __forceinline__ void sts128(uint32_t a, const uint4 &v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

template <int R> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// The CTA's shared memory, and a segment ring cursor per warp.
template <typename T, int D, bool F8> struct ExtCta {
    using C = ExtCfg<T, D, F8>;
    const ExtendParams &p;
    uint32_t ring, raw, qbuf, bar0;
    volatile ExtSeg *segs;
    volatile float *xch;    // [2][M] pairs
    volatile signed char *qexp;   // [2 in flight][2][M]
    int lane;
    int sg = 0;             // segments taken so far
    bool dead = false;

    __device__ __forceinline__ explicit ExtCta(const ExtendParams &params) : p(params) {}

    __device__ __forceinline__ uint32_t bar(int i) const { return bar0 + 8u * (uint32_t)i; }
    __device__ __forceinline__ uint32_t full(int s) const { return bar(s); }
    __device__ __forceinline__ uint32_t empty(int s) const { return bar(C::STAGES + s); }
    static constexpr int B0 = 2 * C::STAGES;
    __device__ __forceinline__ uint32_t s_full(int x) const { return bar(B0 + x); }
    __device__ __forceinline__ uint32_t p_full(int x, int part) const { return bar(B0 + 2 + 2 * x + part); }
    __device__ __forceinline__ uint32_t o_full(int x) const { return bar(B0 + 6 + x); }
    __device__ __forceinline__ uint32_t q_full(int x) const { return bar(B0 + 8 + x); }
    __device__ __forceinline__ uint32_t q_empty(int x) const { return bar(B0 + 10 + x); }
    __device__ __forceinline__ uint32_t q_wide(int x) const { return bar(B0 + 12 + x); }
    __device__ __forceinline__ uint32_t meet() const { return bar(B0 + 14); }
    __device__ __forceinline__ uint32_t fin() const { return bar(B0 + 15); }
    static constexpr int B1 = B0 + 16;
    __device__ __forceinline__ uint32_t g_full(int s) const { return bar(B1 + s); }
    __device__ __forceinline__ uint32_t g_empty(int s) const { return bar(B1 + C::SEGS + s); }
    static constexpr int B2 = B1 + 2 * C::SEGS;
    __device__ __forceinline__ uint32_t r_full(int s) const { return bar(B2 + s); }
    __device__ __forceinline__ uint32_t r_empty(int s) const { return bar(B2 + C::RAWS + s); }
    static_assert(B2 + 2 * C::RAWS == C::NBAR, "barrier count");

    __device__ __forceinline__ void init()
    {
        for (int s = 0; s < C::STAGES; ++s) {
            // the producer's arrival plus the copy's bytes, or the widening warps
            mbar_init(full(s), F8 ? C::CVT_WARPS : 1);
            mbar_init(empty(s), 1);           // commit behind the block's last MMA
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full(x), 1);          // commit behind S
            mbar_init(p_full(x, 0), 4);       // the engine's warps: S read, O rescaled, a part of P written
            mbar_init(p_full(x, 1), 4);
            mbar_init(o_full(x), 1);          // commit behind the segment's last P.V
            mbar_init(q_full(x), 1);
            mbar_init(q_empty(x), 1);         // commit behind the segment's last S
            mbar_init(q_wide(x), C::CVT_WARPS);   // the widening warps
        }
        mbar_init(meet(), 8);                 // the softmax warps of both engines
        mbar_init(fin(), 1);
        for (int s = 0; s < C::SEGS; ++s) {
            mbar_init(g_full(s), 1);
            mbar_init(g_empty(s), F8 ? 11 + C::CVT_WARPS : 11);   // every warp but the scheduler
        }
        for (int s = 0; s < C::RAWS; ++s) {
            mbar_init(r_full(s), 1);
            mbar_init(r_empty(s), C::CVT_WARPS);
        }
    }

    // Wait of a whole warp for the n-th (from 0) completion of a barrier.
    __device__ __forceinline__ bool wait(uint32_t b, int n)
    {
        if (!dead && !mbar_wait_bounded_soon(b, (uint32_t)(n & 1), C::SLEEP_NS, p.wait_ns))
            dead = true;
        return !dead;
    }

    __device__ __forceinline__ void arrive(uint32_t b)
    {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(b);
    }

    // The next segment, by a whole warp; false at the end (or on expiry).
    __device__ __forceinline__ bool next(ExtSeg &g)
    {
        const int s = sg % C::SEGS;
        if (!wait(g_full(s), sg / C::SEGS))
            return false;
        const volatile ExtSeg &x = segs[s];
        g.valid = x.valid;
        g.row0 = x.row0;
        g.ntok = x.ntok;
        g.h = x.h;
        g.slice = x.slice;
        g.b = x.b;
        g.m = x.m;
        g.lim = x.lim;
        g.k0 = x.k0;
        g.blk0 = x.blk0;
        g.end0 = x.end0;
        g.end1 = x.end1;
        g.flags = x.flags;
        g.slot = x.slot;
        arrive(g_empty(s));
        ++sg;
        return g.valid != 0;
    }
};

// ---------------------------------------------------------------- scheduler
// One lane: the CTA's cut pieces first, then its whole items.
template <typename T, int D, bool F8>
__device__ __forceinline__ void ext_schedule(const ExtendParams &p, ExtCta<T, D, F8> &cta)
{
    using C = ExtCfg<T, D, F8>;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int G = p.grid, c = blockIdx.x, Hv = p.Hkv * p.NG;
    const ExtPlanHeader hd = *p.header;
    const ExtCut a = p.cuts[c], e = p.cuts[c + 1];
    int sg = 0;
    // a segment of item `it`, blocks [blk0, blk1)
    auto push = [&](int it, const ExtTile &t, int blk0, int blk1, int slot, int link, int target) {
        const int s = sg % C::SEGS;
        if (sg >= C::SEGS &&
            !mbar_wait_bounded_sleep_thread(cta.g_empty(s), (uint32_t)(((sg / C::SEGS) - 1) & 1), C::SLEEP_NS,
                                            p.wait_ns)) {
            cta.dead = true;
            return;
        }
        volatile ExtSeg &g = cta.segs[s];
        const int vh = it < 0 ? 0 : it % Hv;
        g.valid = it >= 0;
        g.row0 = t.row0;
        g.ntok = t.ntok;
        g.h = vh / p.NG;
        g.slice = vh % p.NG;
        g.b = t.b;
        g.m = t.m;
        g.lim = t.lim;
        g.k0 = t.k0;
        g.blk0 = blk0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int n = min(t.ntok - x * p.tps, p.tps);   // the sub-tile's tokens
            const int see = n <= 0 ? 0 : p.causal ? min(t.m, t.lim + x * p.tps + n - 1) : t.m;
            const int end = see > 0 ? (see + C::CT - 1) / C::CT : 0;
            (x ? g.end1 : g.end0) = max(blk0, min(blk1, end));
        }
        g.flags = (t.ntok <= p.tps && blk1 - blk0 > 1 ? 1 : 0) | link << 1 | target * 8;
        g.slot = slot;
        mbar_arrive(cta.g_full(s));
        ++sg;
    };
    // the same, as a chain where the range is long: links of like lengths (so
    // all of them are twins or none is), the first one's result in the CTA's
    // first slot, the others' in its second
    auto pieces = [&](int it, const ExtTile &t, int blk0, int blk1, int slot) {
        const int n = blk1 - blk0;
        if (n <= EXT_LINK) {
            push(it, t, blk0, blk1, slot, ExtSeg::ALONE, 0);
            return;
        }
        const int links = (n + EXT_LINK - 1) / EXT_LINK, own = 2 * (G + 1) + 2 * c;
        for (int k = 0, b = blk0; k < links && !cta.dead; ++k) {
            const int e = b + (blk1 - b + links - k - 1) / (links - k);
            push(it, t, b, e, k ? own + 1 : own, k == 0 ? ExtSeg::FIRST : k + 1 < links ? ExtSeg::INNER : ExtSeg::LAST, slot);
            b = e;
        }
    };
    for (int it = a.item; it < hd.n_items && !cta.dead; ++it) {
        const bool last = it == e.item;
        if (it > e.item || (last && e.off == 0))
            break;
        const ExtTile t = p.tiles[it / Hv];
        const bool fresh = it > a.item || a.off == 0;
        const int b0 = it > a.item ? 0 : a.blk, b1 = last ? e.blk : t.nblk;
        if (t.nblk == 0 ? !fresh : b1 <= b0)
            continue;
        const bool whole = b0 == 0 && b1 == t.nblk;
        pieces(it, t, b0, b1, whole ? -1 : b0 > 0 ? 2 * c + 1 : 2 * (c + 1));
    }
    for (int x = 0; x < hd.waves && !cta.dead; ++x) {
        const int it = x * G + ((x & 1) ? G - 1 - c : c);
        const ExtTile t = p.tiles[it / Hv];
        pieces(it, t, 0, t.nblk, -1);
    }
    if (!cta.dead) {
        const ExtTile none = {};
        push(-1, none, 0, 0, -1, ExtSeg::ALONE, 0);
    }
}

// ---------------------------------------------------------------- K and V
// Each lane one box of a block (row group, plane), so the rows of a block
// may come from several pages.
template <typename T, int D, bool F8>
__device__ __forceinline__ void ext_load_kv(const ExtendParams &p, ExtCta<T, D, F8> &cta)
{
    using C = ExtCfg<T, D, F8>;
    constexpr int NS = F8 ? C::RAWS : C::STAGES;
    const int R = p.paged ? p.box_rows : C::CT;
    const int ng = C::CT / R;   // row groups (at most 8)
    const int grp = cta.lane % ng, plane = cta.lane / ng;
    // (one box holds all planes where a block is one row group)
    const bool mine = plane < (F8 || ng == 1 ? 1 : C::PLANES);
    const uint32_t box = (uint32_t)(R * (F8 ? D : ng == 1 ? 128 * C::PLANES : 128));
    const uint32_t at = (uint32_t)(F8 ? grp * R * D : plane * C::PLANE + grp * R * 128);   // in the stage
    // a block's rows, in pages and rows of a page (no division in the loop:
    // this warp's time an item bounds how fast a cache can stream)
    const int ps = p.paged ? p.page_size : 1;
    const int pstep = C::CT / ps, rstep = C::CT % ps;
    int slot = 0, lap = 0;      // the ring: next stage, times round
    ExtSeg g;
    while (cta.next(g)) {
        const int nb = ext_blocks(g);
        const ExtOrder order = {g.twin(), nb};
        int tok = g.blk0 * C::CT + grp * R;   // this lane's first row of the next K
        int pidx = tok / ps, row = tok % ps;
        const int32_t *table = p.table + (long long)g.b * p.max_pages;
        auto page_at = [&]() { return (p.paged && mine && tok < g.m) ? __ldg(table + pidx) : 0; };
        int page = page_at();   // read a block ahead
        // where this lane's rows of K(ki) and of K(ki - 1) are: row in the
        // page (or of all), page and head (or head); x < 0: behind the
        // sequence's keys
        int ki = 0, kx = -1, ky = 0, bx = -1, by = 0;
        for (int t = 0; t < 2 * nb && !cta.dead; ++t) {
            int i;
            const bool isv = order.item(t, i);
            if (!isv) {
                bx = kx;
                by = ky;
                ki = i;
                kx = -1;
                if (mine && tok < g.m) {
                    if (!p.paged) {
                        kx = g.k0 + tok;
                        ky = g.h;
                    } else {
                        if (page < 0 || page >= p.num_pages) {
                            atomicOr(p.status, STATUS_BAD_PAGE);
                            page = 0;
                        }
                        kx = row;
                        ky = page * p.Hkv + g.h;
                    }
                }
                tok += C::CT;
                pidx += pstep;
                row += rstep;
                if (row >= ps) {
                    row -= ps;
                    ++pidx;
                }
                page = i + 1 < nb ? page_at() : 0;
            }
            const int x = i == ki ? kx : bx, y = i == ki ? ky : by;
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(FULL_MASK, x >= 0)) * box;
            const uint32_t full = F8 ? cta.r_full(slot) : cta.full(slot);
            if (lap > 0 && !cta.wait(F8 ? cta.r_empty(slot) : cta.empty(slot), lap - 1))
                break;
            if (cta.lane == 0)
                mbar_arrive_expect_tx(full, bytes);
            __syncwarp();
            const CUtensorMap *tm = isv ? &p.tmv : &p.tmk;
            if (F8 && x >= 0)
                tma_load_3d(cta.raw + (uint32_t)(slot * C::RAW_BYTES) + at, tm, 0, x, y, full);
            else if (x >= 0)
                tma_load_4d(cta.ring + (uint32_t)(slot * C::BLOCK_BYTES) + at, tm, 0, x, y, plane, full);
            if (++slot == NS) {
                slot = 0;
                ++lap;
            }
        }
    }
    // no copy may be in flight when the CTA ends: the last fill of each stage
    for (int i = 0; i < NS; ++i) {
        const int n = i < slot ? lap : lap - 1;   // its last lap
        if (n >= 0)
            mbar_wait_bounded_soon(F8 ? cta.r_full(i) : cta.full(i), (uint32_t)(n & 1), C::SLEEP_NS, p.wait_ns);
    }
}

// ---------------------------------------------------------------- Q
// A sub-tile's rows: tps tokens of Gs heads each, plane by plane.  Rows
// behind the sequence's are other sequences' (or zeros): they are computed
// and not written out.
template <typename T, int D, bool F8>
__device__ __forceinline__ void ext_load_q(const ExtendParams &p, ExtCta<T, D, F8> &cta)
{
    using C = ExtCfg<T, D, F8>;
    int n[2] = {0, 0};
    ExtSeg g;
    while (cta.next(g)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (g.end(x) <= g.blk0)
                continue;
            if (n[x] > 0 && !cta.wait(cta.q_empty(x), n[x] - 1))
                break;
            if (cta.lane == 0) {
                mbar_arrive_expect_tx(cta.q_full(x), (uint32_t)(C::PLANES * p.tps * p.Gs * 128));
                for (int pl = 0; pl < C::PLANES; ++pl)
                    tma_load_4d(cta.qbuf + (uint32_t)(x * C::Q_BYTES + pl * C::PLANE), &p.tmq, 0,
                                g.h * p.G + g.slice * p.Gs, g.row0 + x * p.tps, pl, cta.q_full(x));
            }
            ++n[x];
        }
    }
    for (int x = 0; x < 2; ++x)
        if (n[x] > 0)
            mbar_wait_bounded_soon(cta.q_full(x), (uint32_t)((n[x] - 1) & 1), C::SLEEP_NS, p.wait_ns);
}

// ---------------------------------------------------------------- E4M3 to f16
template <typename T, int D, bool F8>
__device__ __forceinline__ void ext_widen(const ExtendParams &p, ExtCta<T, D, F8> &cta)
{
    using C = ExtCfg<T, D, F8>;
    constexpr int NR = F8 ? C::RAWS : 1, ST = C::STAGES;
    // A thread widens 16 values of a row at a time into the swizzled planes
    // that the MMAs read; the raw rows are swizzled too (by the copy: 128
    // bytes at d = 128, 64 at d = 64).  Eight lanes take the same piece of
    // eight rows in a row, which the swizzles put into eight different
    // banks on both sides, and a thread's rows are a multiple of 8 apart, so
    // its offsets are constants.
    constexpr int CPR = D / 16;             // 16-value pieces of a row
    constexpr int BATCH = C::CT * CPR / 128;
    const int ct = (int)threadIdx.x - C::CVT_WARP * 32;
    const int r8 = ct & 7, c = (ct >> 3) % CPR;
    const int r0 = r8 + 8 * ((ct >> 3) / CPR);
    const uint32_t src0 = (uint32_t)(r0 * D + ((D == 128 ? c ^ r8 : c ^ (r8 >> 1)) << 4));
    const uint32_t dst0 = (uint32_t)((c >> 2) * C::PLANE + r0 * 128 + (((2 * (c & 3)) ^ r8) << 4));
    const uint32_t dst1 = dst0 ^ 16u;
    int rs = 0, rlap = 0, s = 0, lap = 0;   // both rings: next stage, times round
    int nq[2] = {0, 0};
    ExtSeg g;
    while (cta.next(g)) {
        const int nb = ext_blocks(g);
        // Q of the segment, a thread a row, in place
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (g.end(x) <= g.blk0)
                continue;
            if (!cta.wait(cta.q_full(x), nq[x]))
                break;
            int sh = 0;
            if (p.dtype == 2) {
                const uint32_t row = cta.qbuf + (uint32_t)(x * C::Q_BYTES + ct * 128);
                uint32_t top = 0;   // the largest magnitude's bits
#pragma unroll
                for (int i = 0; i < C::PLANES * 8; ++i) {
                    const uint4 u = lds128(row + (uint32_t)((i >> 3) * C::PLANE + (((i & 7) ^ (ct & 7)) << 4)));
                    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top = max(top, max((v[e] << 16) & 0x7fff0000u, v[e] & 0x7fff0000u));
                }
                if (top)
                    sh = min(max(8 + 127 - (int)(top >> 23), -120), 120);
                const float f = __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
                for (int i = 0; i < C::PLANES * 8; ++i) {
                    const uint32_t a = row + (uint32_t)((i >> 3) * C::PLANE + (((i & 7) ^ (ct & 7)) << 4));
                    float y[8];
                    Elem<__nv_bfloat16>::widen(lds128(a), y);
                    sts128(a, make_uint4(Mma<__half>::pack(y[0] * f, y[1] * f), Mma<__half>::pack(y[2] * f, y[3] * f),
                                         Mma<__half>::pack(y[4] * f, y[5] * f), Mma<__half>::pack(y[6] * f, y[7] * f)));
                }
                fence_proxy_async_smem();
            }
            cta.qexp[((nq[x] & 1) * 2 + x) * C::M + ct] = (signed char)sh;
            cta.arrive(cta.q_wide(x));
            ++nq[x];
        }
        const ExtOrder order = {g.twin(), nb};
        for (int t = 0; t < 2 * nb && !cta.dead; ++t) {
            int i;
            order.item(t, i);
            const int left = g.m - (g.blk0 + i) * C::CT;
            if (!cta.wait(cta.r_full(rs), rlap) || (lap > 0 && !cta.wait(cta.empty(s), lap - 1)))
                break;
            const uint32_t src = cta.raw + (uint32_t)(rs * C::RAW_BYTES) + src0;
            const uint32_t dst = cta.ring + (uint32_t)(s * C::BLOCK_BYTES);
            constexpr int STEP = 128 / CPR;   // rows between a thread's pieces
            uint4 v[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                v[k] = lds128(src + (uint32_t)(k * STEP * D));
            if (left < C::CT) {
                // rows behind the sequence's last key may hold anything, and
                // 0 * NaN is NaN
#pragma unroll
                for (int k = 0; k < BATCH; ++k)
                    if (r0 + k * STEP >= left)
                        v[k] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                uint4 lo, hi;
                e4m3_widen16(v[k], lo, hi);
                sts128(dst + dst0 + (uint32_t)(k * STEP * 128), lo);
                sts128(dst + dst1 + (uint32_t)(k * STEP * 128), hi);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (cta.lane == 0) {
                mbar_arrive(cta.full(s));
                mbar_arrive(cta.r_empty(rs));
            }
            if (++rs == NR) {
                rs = 0;
                ++rlap;
            }
            if (++s == ST) {
                s = 0;
                ++lap;
            }
        }
    }
}

// ---------------------------------------------------------------- MMA issue
// The whole warp runs it; the instructions are predicated on one lane.
template <typename T, int D, bool F8>
__device__ __forceinline__ void ext_mma(const ExtendParams &p, ExtCta<T, D, F8> &cta, uint32_t tmem)
{
    using C = ExtCfg<T, D, F8>;
    constexpr int ST = C::STAGES;
    constexpr int BF = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    constexpr uint32_t ID_S = idesc_f16(BF, 0, 0, C::M, C::CT);   // Q K-major, K K-major
    constexpr uint32_t ID_O = idesc_f16(BF, 0, 1, C::M, D);       // P (TMEM) K-major, V MN-major
    // Descriptors: a base, plus offsets in its units of 16 bytes (an address
    // fits the field, so no carry leaves it).
    const uint64_t qdesc = smem_desc_sw128(cta.qbuf, 16, 1024), kdesc = smem_desc_sw128(cta.ring, 16, 1024);
    const uint64_t vdesc = smem_desc_sw128(cta.ring, (uint32_t)C::PLANE, 1024);
    const uint32_t one = elect_one();
    int np0 = 0, np1 = 0;   // P taken from each engine
    int nq0 = 0, nq1 = 0;   // Q of each sub-tile taken
    // the ring is used in the order it is filled
    struct Cursor {
        int slot, phase;
        __device__ __forceinline__ void step()
        {
            if (++slot == ST) {
                slot = 0;
                phase ^= 1;
            }
        }
    } cur = {0, 0};
    auto landed = [&](const Cursor &c) { return cta.wait(cta.full(c.slot), c.phase); };
    // S of engine x, from Q of sub-tile q and K in stage st
    auto issue_s = [&](int x, int q, int st) {
        const uint64_t a = qdesc + (uint64_t)(q * (C::Q_BYTES >> 4)), b = kdesc + (uint64_t)(st * (C::BLOCK_BYTES >> 4));
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            // 16 elements = 32 bytes of each 128-byte row of plane ks / 4
            const uint64_t o = (uint64_t)(((ks >> 2) * C::PLANE + (ks & 3) * 32) >> 4);
            tc_mma_ss_if(one, tmem + (uint32_t)C::tm_s(x), a + o, b + o, ID_S, ks > 0 ? 1u : 0u);
        }
        tc_commit_if(one, cta.s_full(x));
    };
    // P.V of engine x, part by part as P arrives, V in stage st
    auto issue_pv = [&](int x, int st, bool first, int &np) {
        const uint64_t b = vdesc + (uint64_t)(st * (C::BLOCK_BYTES >> 4));
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            if (!cta.wait(cta.p_full(x, part), np))
                return;
            tc_fence_after();
#pragma unroll
            for (int ks = part ? C::PART / 16 : 0; ks < (part ? C::CT : C::PART) / 16; ++ks)
                tc_mma_ts_if(one, tmem + (uint32_t)C::tm_o(x), tmem + (uint32_t)(C::tm_p(x) + ks * 8),
                             b + (uint64_t)(ks * (2048 >> 4)), ID_O, (!first || ks > 0) ? 1u : 0u);
        }
        ++np;
    };
    // The same for a sequence's last block: of the 16-key steps only the
    // first `steps` hold keys
    auto issue_pv_tail = [&](int x, int st, bool first, int &np, int steps) {
        const uint64_t b = vdesc + (uint64_t)(st * (C::BLOCK_BYTES >> 4));
        if (!cta.wait(cta.p_full(x, 0), np) || !cta.wait(cta.p_full(x, 1), np))
            return;
        tc_fence_after();
#pragma unroll 1
        for (int ks = 0; ks < steps; ++ks)
            tc_mma_ts_if(one, tmem + (uint32_t)C::tm_o(x), tmem + (uint32_t)(C::tm_p(x) + ks * 8),
                         b + (uint64_t)(ks * (2048 >> 4)), ID_O, (!first || ks > 0) ? 1u : 0u);
        ++np;
    };
    ExtSeg g;
    while (cta.next(g)) {
        const int nb = ext_blocks(g);
        if (nb == 0)
            continue;
        const bool twin = g.twin();
        // engine x's blocks: its own sub-tile's, or every other one
        const int ahead = twin ? 2 : 1;   // S runs so many blocks ahead of P.V
        const int len0 = twin ? nb : g.end0 - g.blk0, len1 = twin ? nb : g.end1 - g.blk0;
        auto has = [&](int x, int i) { return i >= 0 && i < (x ? len1 : len0) && (!twin || (i & 1) == x); };
        // Both engines have this block and the two behind it: straight
        // through.  A stage is given back as soon as its last MMA is issued
        // (both at the end cost 5%: the ring is just deep enough).  The
        // general loop below has one copy of each product for the rest: code
        // that runs once a call comes from L2 line by line.
        const int plain = twin ? 0 : min(len0, len1) - 2;
#pragma unroll 1
        for (int i = -ahead; i < nb && !cta.dead; ++i) {
            if (i == 0 && plain > 1) {
#pragma unroll 1
                for (; i < plain && !cta.dead; ++i) {
                    const Cursor vc = cur;
                    cur.step();
                    // (a wait costs some 150 cycles even when it is over: K's
                    // too is off the way from P to S)
                    if (!landed(vc) || !landed(cur))
                        break;
                    issue_pv(0, vc.slot, i == 0, np0);
                    issue_s(0, 0, cur.slot);
                    issue_pv(1, vc.slot, i == 0, np1);
                    tc_commit_if(one, cta.empty(vc.slot));
                    issue_s(1, 1, cur.slot);
                    tc_commit_if(one, cta.empty(cur.slot));
                    cur.step();
                }
                if (cta.dead)
                    break;
            }
            if (i == 0 && twin) {
                // the engines' blocks by turns, all but the last two
#pragma unroll 1
                for (; i + 2 < nb; ++i) {
                    const int x = i & 1;
                    const Cursor vc = cur;
                    cur.step();
                    if (!landed(vc))
                        break;
                    int np = x ? np1 : np0;
                    issue_pv(x, vc.slot, i < 2, np);
                    (x ? np1 : np0) = np;
                    tc_commit_if(one, cta.empty(vc.slot));
                    if (!landed(cur))
                        break;
                    issue_s(x, 0, cur.slot);
                    tc_commit_if(one, cta.empty(cur.slot));
                    if (i + 3 == nb)
                        tc_commit_if(one, cta.q_empty(0));
                    cur.step();
                }
                if (cta.dead)
                    break;
            }
            const int k = i + ahead;
            const bool more = k < nb;
            Cursor vc = cur;
            int steps = C::CT / 16;
            if (i >= 0) {
                cur.step();
                if (!landed(vc))
                    break;
                const int left = g.m - (g.blk0 + i) * C::CT;
                if (left < C::CT) {
                    steps = (left + 15) / 16;
                    if (!F8) {
                        // V's rows behind the sequence's last key may hold
                        // anything, and 0 * NaN is NaN: zeros instead, in the
                        // last step that is computed
                        const uint32_t vb = cta.ring + (uint32_t)(vc.slot * C::BLOCK_BYTES + left * 128);
                        for (int e = cta.lane; e < (steps * 16 - left) * 8; e += 32)
#pragma unroll
                            for (int pl = 0; pl < C::PLANES; ++pl)
                                sts128(vb + (uint32_t)(pl * C::PLANE + e * 16), make_uint4(0, 0, 0, 0));
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
            }
            const int last = has(1, i) ? 1 : 0;   // the engine that is done with V last
            bool kready = false;
#pragma unroll 1
            for (int x = 0; x < 2 && !cta.dead; ++x) {
                if (has(x, i)) {
                    int np = x ? np1 : np0;
                    if (steps == C::CT / 16)
                        issue_pv(x, vc.slot, i < ahead, np);
                    else
                        issue_pv_tail(x, vc.slot, i < ahead, np, steps);
                    (x ? np1 : np0) = np;
                    if (!has(x, k))
                        tc_commit_if(one, cta.o_full(x));
                    if (x == last)
                        tc_commit_if(one, cta.empty(vc.slot));
                }
                if (has(x, k)) {
                    const int q = twin ? 0 : x;
                    if (k == 0) {
                        int nq = q ? nq1 : nq0;
                        cta.wait(F8 ? cta.q_wide(q) : cta.q_full(q), nq);
                        (q ? nq1 : nq0) = nq + 1;
                    }
                    if (!kready && !landed(cur))
                        break;
                    kready = true;
                    issue_s(x, q, cur.slot);
                    if (k == (x && !twin ? len1 : len0) - 1)
                        tc_commit_if(one, cta.q_empty(q));   // the last S that reads this Q
                }
            }
            if (more && !cta.dead) {
                tc_commit_if(one, cta.empty(cur.slot));
                cur.step();
            }
        }
    }
    // every MMA issued here has completed before TMEM is freed
    __syncwarp();
    tc_commit_if(one, cta.fin());
    if (!mbar_wait_bounded_soon(cta.fin(), 0, C::SLEEP_NS, p.wait_ns))
        cta.dead = true;
}

// ---------------------------------------------------------------- chains
// A thread's row (columns [c0, c1) of it) of a link whose result stands in the
// CTA's slots, with the reference m and the sum l: the first link's is kept,
// the others' is joined with what stands there, and the last one's written
// where the chain's goes.  A thread reads only what it wrote itself (the
// engines of a twin keep a copy of (m, l) each).
template <typename T, int D, bool F8>
__device__ __forceinline__ void ext_join(const ExtendParams &p, const ExtSeg &g, int x, int sub, int row,
                                         long long qrow, int c0, int c1, float m, float l, float vscale)
{
    using C = ExtCfg<T, D, F8>;
    const long long own = 2 * ((long long)p.grid + 1 + blockIdx.x);   // the CTA's first slot
    float2 *ml = p.part_ml + (own * 2 + x) * C::M + row;
    if (g.link() == ExtSeg::FIRST) {
        *ml = make_float2(m, l);
        return;
    }
    float *before = p.part_o + ((own * 2 + sub) * C::M + row) * D;
    const float *now = before + 2LL * C::M * D;
    const float2 b = *ml;
    const float top = fmaxf(b.x, m);
    float fb = b.x == -INFINITY ? 0.f : ex2(b.x - top), fn = m == -INFINITY ? 0.f : ex2(m - top);
    l = fb * b.y + fn * l;
    const bool any = !(l <= 0.f);       // NaN counts: it is the result then
    m = any ? top : -INFINITY;
    const bool last = g.link() == ExtSeg::LAST;
    const int target = g.target();
    const bool result = last && target < 0;
    if (result) {
        const float inv = any ? vscale / l : 0.f;
        fb *= inv;
        fn *= inv;
    }
    const long long to = last && target >= 0 ? ((long long)target * 2 + sub) * C::M + row : (own * 2 + sub) * C::M + row;
    // (8 columns at a time: unrolled further, the code that most calls do not
    // run cost prompts of a link or less up to 2%)
#pragma unroll 1
    for (int c = c0; c < c1; c += 8) {
        float4 u[2], v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            u[i] = *reinterpret_cast<const float4 *>(before + c + 4 * i);
            v[i] = *reinterpret_cast<const float4 *>(now + c + 4 * i);
        }
        float o[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // (an empty row is 0)
            o[4 * i] = any ? fmaf(u[i].x, fb, v[i].x * fn) : 0.f;
            o[4 * i + 1] = any ? fmaf(u[i].y, fb, v[i].y * fn) : 0.f;
            o[4 * i + 2] = any ? fmaf(u[i].z, fb, v[i].z * fn) : 0.f;
            o[4 * i + 3] = any ? fmaf(u[i].w, fb, v[i].w * fn) : 0.f;
        }
        const long long at = (result ? qrow : to) * D + c;
        if (!result || p.out_dtype == 0) {
            float4 *w = reinterpret_cast<float4 *>((result ? static_cast<float *>(p.out) : p.part_o) + at);
            w[0] = make_float4(o[0], o[1], o[2], o[3]);
            w[1] = make_float4(o[4], o[5], o[6], o[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = p.out_dtype == 1 ? Mma<__half>::pack(o[2 * i], o[2 * i + 1])
                                        : Mma<__nv_bfloat16>::pack(o[2 * i], o[2 * i + 1]);
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    if (!last)
        *ml = make_float2(m, l);
    else if (c0 == 0 && !result)
        p.part_ml[to] = make_float2(m, l);
    else if (c0 == 0 && p.lse)
        p.lse[qrow] = any ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// ---------------------------------------------------------------- softmax
template <typename T, int D, bool F8>
__device__ __forceinline__ void ext_softmax(const ExtendParams &p, ExtCta<T, D, F8> &cta, uint32_t tmem)
{
    using C = ExtCfg<T, D, F8>;
    const int w = threadIdx.x >> 5;
    const int x = w >> 2;                      // engine
    const int row = (int)(threadIdx.x & 127);  // row of the sub-tile = TMEM lane
    const uint32_t tl = tmem + ((uint32_t)((w & 3) * 32) << 16);
    const int rtok = row / p.Gs, rg = row % p.Gs;
    int ns = 0, no = 0, meets = 0;
    int nq0 = 0, nq1 = 0;   // E4M3: loads of each sub-tile's Q
    ExtSeg g;
    while (cta.next(g)) {
        const bool twin = g.twin();
        const int sub = twin ? 0 : x;          // whose rows
        const int tok = sub * p.tps + rtok;    // token within the tile
        const int gv = min(p.Gs, p.G - g.slice * p.Gs);
        const bool live = rtok < p.tps && tok < g.ntok && rg < gv;
        // keys this row sees; a row that is not written takes those of the
        // last one, so that its warp masks no block for its sake
        const int lim = p.causal ? min(g.m, g.lim + min(tok, g.ntok - 1)) : g.m;
        float sc = p.scale_log2;
        float vscale = 1.f;
        if (F8) {
            sc *= __ldg(p.k_scale + (long long)g.b * p.Hkv + g.h);
            vscale = __ldg(p.v_scale + (long long)g.b * p.Hkv + g.h);
        }
        // the exponents of this segment's Q: of its sub-tile's n-th load
        int qn = 0;
        if (F8) {
            qn = (sub ? nq1 : nq0) & 1;
            nq0 += g.end0 > g.blk0;
            nq1 += g.end1 > g.blk0;
        }
        float mref = -INFINITY, l = 0.f;
        const int begin = g.blk0 + (twin ? x : 0), end = g.end(sub), step = twin ? 2 : 1;
        // blocks below this one hide nothing from any row of the warp
        const int whole = __reduce_min_sync(FULL_MASK, max(lim, 0)) / C::CT;
#pragma unroll 1
        for (int j = begin; j < end; j += step) {
            if (!cta.wait(cta.s_full(x), ns))
                break;
            ++ns;
            tc_fence_after();
            if (F8 && j == begin) {
                // S was issued behind the wait for Q's widening, which wrote
                // them (waiting for that again here could miss a phase: an
                // engine without blocks falls behind by several segments)
                const int sh = cta.qexp[(qn * 2 + sub) * C::M + row];
                sc *= __uint_as_float((uint32_t)(127 - sh) << 23);
            }
            float s[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                tmem_ld32(tl + (uint32_t)(C::tm_s(x) + 32 * i), s[i]);
            tmem_wait_ld();
            float sx = sc;
            if (F8 && !(sc > 0.f)) {   // a K scale that is not positive
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    s[i >> 5][i & 31] *= sc;
                sx = 1.f;
            }
            if (j >= whole) {
                const int see = lim - j * C::CT;
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    s[i >> 5][i & 31] = i < see ? s[i >> 5][i & 31] : -INFINITY;
            }
            // four chains of three-input maxima
            float mx[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mx[i] = fmaxf(s[i][0], s[i][1]);
#pragma unroll
            for (int e = 2; e < 32; e += 2)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mx[i] = fmaxf(mx[i], fmaxf(s[i][e], s[i][e + 1]));
            const float mc = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sx;
            const bool grow = mc > mref + C::TAU;
            float a = 1.f;
            if (grow) {
                a = ex2(mref - mc);   // 0 on the row's first keys
                l *= a;
                mref = mc;
            }
            // the tcgen05 loads and stores are warp-wide, so the whole warp
            // runs them when any of its rows grew (a = 1 for others)
            if (j > begin && __any_sync(FULL_MASK, grow)) {
#pragma unroll 1
                for (int q = 0; q < D / 16; ++q) {
                    float o[16];
                    tmem_ld16(tl + (uint32_t)(C::tm_o(x) + 16 * q), o);
                    tmem_wait_ld();
                    uint32_t u[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        u[e] = __float_as_uint(o[e] * a);
                    tmem_st16u(tl + (uint32_t)(C::tm_o(x) + 16 * q), u);
                }
            }
            const float nm = mref == -INFINITY ? 0.f : C::SHIFT - mref;
            const uint64_t sc2 = pack2(sx, sx), nm2 = pack2(nm, nm);
            uint64_t ls[4] = {0, 0, 0, 0};   // pairs of zeros
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t ph[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float x0, x1;
                    unpack2(fma2(pack2(s[i][2 * e], s[i][2 * e + 1]), sc2, nm2), x0, x1);
                    const float p0 = ex2(x0), p1 = ex2(x1);
                    ls[e & 3] = add2(ls[e & 3], pack2(p0, p1));
                    ph[e] = Mma<T>::pack(p0, p1);
                }
                tmem_st16u(tl + (uint32_t)(C::tm_p(x) + 16 * i), ph);
                if (i == C::PART / 32 - 1 || i == 3) {
                    // a part of P: its product with V may start
                    tmem_wait_st();
                    tc_fence_before();
                    cta.arrive(cta.p_full(x, i == 3));
                    // keep the rest's exponentials behind this hand-over (the
                    // compiler had computed them all first)
#pragma unroll
                    for (int k = i + 1; k < 4; ++k)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            asm volatile("" : "+f"(s[k][e]));
                }
            }
            float la, lb;
            unpack2(add2(add2(ls[0], ls[1]), add2(ls[2], ls[3])), la, lb);
            l += la + lb;
        }
        // ---- the segment's result ----
        const bool some = end > begin;
        if (some && !cta.dead && cta.wait(cta.o_full(x), no)) {
            ++no;
            tc_fence_after();
        }
        if (cta.dead)
            break;
        const long long qrow = (long long)(g.row0 + tok) * p.Hq + g.h * p.G + g.slice * p.Gs + rg;
        const long long prow = ((long long)g.slot * 2 + sub) * C::M + row;
        float M = mref, L = l;             // of the row; f0, f1: the factors of both O
        float f0 = 1.f, f1 = 0.f;
        int ta = C::tm_o(x), tb = ta;      // columns of this engine's O, and of a second one to add
        int c0 = 0, c1 = D;                // columns this engine writes
        if (twin) {
            // both engines hold the same rows: they swap (reference, sum),
            // and each joins and writes half of the columns
            cta.xch[2 * (x * C::M + row)] = mref;
            cta.xch[2 * (x * C::M + row) + 1] = l;
            tc_fence_before();
            cta.arrive(cta.meet());
            if (!cta.wait(cta.meet(), meets++))
                break;
            tc_fence_after();
            const float2 a0 = make_float2(cta.xch[2 * row], cta.xch[2 * row + 1]);
            const float2 a1 = make_float2(cta.xch[2 * (C::M + row)], cta.xch[2 * (C::M + row) + 1]);
            M = fmaxf(a0.x, a1.x);
            f0 = a0.x == -INFINITY ? 0.f : ex2(a0.x - M);
            f1 = a1.x == -INFINITY ? 0.f : ex2(a1.x - M);
            L = f0 * a0.y + f1 * a1.y;
            c0 = x * (D / 2);
            c1 = c0 + D / 2;
            ta = C::tm_o(0);
            tb = C::tm_o(1);
        }
        const bool any = !(L <= 0.f);      // NaN counts: it is the result then
        if (g.slot < 0) {
            const float inv = any ? vscale / L : 0.f;
            f0 *= inv;
            f1 *= inv;
        }
        void *dst = g.slot >= 0 ? (void *)p.part_o : p.out;
        const long long at = (g.slot >= 0 ? prow : qrow) * D;
        const int kind = g.slot >= 0 ? 0 : p.out_dtype;
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
            float o[32];
            if (some || twin) {
                tmem_ld32(tl + (uint32_t)(ta + c), o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    o[e] *= f0;
            }
            if (twin) {
                float v[32];
                tmem_ld32(tl + (uint32_t)(tb + c), v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    o[e] = fmaf(v[e], f1, o[e]);
            }
            if (!any) {   // an empty row is 0 whatever O holds
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    o[e] = 0.f;
            }
            if (live)
                store_out32(dst, at + c, kind, o);
            __syncwarp();
        }
        tc_fence_before();   // the next segment's P.V overwrites O behind this warp's next P
        if (live && (!twin || x == 0)) {
            if (g.slot >= 0)
                p.part_ml[prow] = make_float2(any ? M - C::SHIFT : -INFINITY, L);
            else if (p.lse)
                p.lse[qrow] = any ? (M - C::SHIFT + log2f(L)) * 0.6931471805599453f : -INFINITY;
        }
        if (twin) {
            // neither engine writes its next P before both have read both O
            cta.arrive(cta.meet());
            if (!cta.wait(cta.meet(), meets++))
                break;
        }
        if (g.link() != ExtSeg::ALONE && live)
            ext_join<T, D, F8>(p, g, x, sub, row, qrow, c0, c1, any ? M - C::SHIFT : -INFINITY, L, vscale);
    }
}

template <typename T, int D, bool F8>
__global__ void __launch_bounds__(ExtCfg<T, D, F8>::THREADS, 1) extend_kernel(const __grid_constant__ ExtendParams p)
{
    using C = ExtCfg<T, D, F8>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the merge waits for this grid's end
    extern __shared__ __align__(1024) unsigned char smem[];           // the swizzle's atoms are 1024 bytes
    const int w = threadIdx.x >> 5;
    ExtCta<T, D, F8> cta(p);
    cta.lane = threadIdx.x & 31;
    cta.ring = smem_addr(smem);
    cta.raw = cta.ring + C::STAGES * C::BLOCK_BYTES;
    cta.qbuf = cta.raw + C::RAWS * C::RAW_BYTES;
    unsigned char *rest = smem + (cta.qbuf + 2 * C::Q_BYTES - cta.ring);
    cta.bar0 = smem_addr(rest);
    rest += C::NBAR * 8;
    cta.xch = reinterpret_cast<volatile float *>(rest);
    rest += C::XCH_BYTES;
    cta.segs = reinterpret_cast<volatile ExtSeg *>(rest);
    static_assert(sizeof(ExtSeg) == 56, "segment slots");
    rest += C::SEGS * 56;
    uint32_t *misc = reinterpret_cast<uint32_t *>(rest);
    cta.qexp = reinterpret_cast<volatile signed char *>(rest + 16);
    if (threadIdx.x == 0) {
        cta.init();
        prefetch_tmap(&p.tmq);
        prefetch_tmap(&p.tmk);
        prefetch_tmap(&p.tmv);
    }
    if (w == C::MMA_WARP) {
        tmem_alloc(smem_addr(misc), C::TMEM_COLS);
        tmem_relinquish();
    }
    fence_mbar_init();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];

    // a warpgroup changes its share of the registers as a whole
    if (w < 8) {
        regs_inc<C::REGS_SOFTMAX>();
        ext_softmax<T, D, F8>(p, cta, tmem);
    } else {
        regs_dec<C::REGS_OTHER>();
        if (w == C::SCHED_WARP) {
            if (cta.lane == 0)
                ext_schedule<T, D, F8>(p, cta);
            __syncwarp();
        } else if (w == C::KV_WARP) {
            ext_load_kv<T, D, F8>(p, cta);
        } else if (w == C::Q_WARP) {
            ext_load_q<T, D, F8>(p, cta);
        } else if (w == C::MMA_WARP) {
            ext_mma<T, D, F8>(p, cta, tmem);
        } else if (F8) {
            ext_widen<T, D, F8>(p, cta);
        }
    }

    if (cta.dead && cta.lane == 0)
        atomicOr(p.status, STATUS_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == C::MMA_WARP)
        tmem_dealloc(tmem, C::TMEM_COLS);
}

template <typename T, int D, bool F8> static cudaError_t launch_extend_t(const ExtendParams &p, cudaStream_t s)
{
    using C = ExtCfg<T, D, F8>;
    auto kern = extend_kernel<T, D, F8>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace fd
