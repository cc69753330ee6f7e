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
// While one sub-tile's softmax runs, the tensor cores work on the other's
// products.  S of a sub-tile's next block is issued behind P.V of the one
// before, so that S's commit also says that P.V is done: a row's rescale
// needs no wait of its own.
//
// Warp roles (384 threads, 512 for E4M3 K/V, one CTA per SM):
//  - warps 0-3, 4-7: softmax and results of sub-tile A, B;
//  - warp 8: K and V by tensor-map TMA, in turn, into one ring;
//  - warp 9: allocates TMEM, issues every MMA;
//  - warp 10: Q by TMA, as soon as a sub-tile's last S is done;
//  - warp 11: walks the CTA's share of the plan, segments into a small ring;
//  - E4M3 only, warps 12-15: widen the blocks that warp 8 copied as they are
//    to the 16-bit type (exact: E4M3 has 4 significant bits and exponents
//    from -9 to 8) for the same products.  The K scale is part of the
//    score's, the V scale of the result's.
// Every hand-off is an mbarrier, and every wait is bounded: on expiry a role
// records FD_ERR_DEVICE_TIMEOUT, stops, waits for the copies it issued, and
// the CTA frees its TMEM.
#pragma once

#include "fd_device.cuh"
#include "fd_extend.h"
#include "fd_tc.cuh"

namespace fd {

template <typename T, int D, bool F8> struct ExtCfg {
    static constexpr int M = EXT_M, CT = EXT_CT;
    static constexpr int PLANES = D / 64;                // 128-byte planes of a row
    static constexpr int PLANE = CT * 128;               // one plane of a block, or of a sub-tile's Q
    static constexpr int BLOCK_BYTES = PLANES * PLANE;   // K or V of one block
    static constexpr int Q_BYTES = PLANES * PLANE;       // one sub-tile
    // 16-bit K and V: 160 KB of copies in flight.  E4M3: the copies land in
    // a ring of raw blocks, and two 16-bit stages (one K, one V) suffice.
    static constexpr int STAGES = F8 ? (D == 128 ? 2 : 4) : (D == 128 ? 5 : 10);
    static constexpr int RAW_BYTES = CT * D;             // an E4M3 block
    static constexpr int RAWS = F8 ? (D == 128 ? 6 : 12) : 0;
    static constexpr int SEGS = 4;                       // segments the scheduler runs ahead
    static constexpr int KV_WARP = 8, MMA_WARP = 9, Q_WARP = 10, SCHED_WARP = 11, CVT_WARP = 12;
    static constexpr int THREADS = F8 ? 512 : 384;
    // registers a thread: the softmax warpgroups hold a row of S each; the
    // shares add up to the launch's (168 x 384 and 128 x 512)
    static constexpr int REGS_SOFTMAX = F8 ? 200 : 208, REGS_OTHER = F8 ? 56 : 88;
    static_assert(2 * REGS_SOFTMAX + (THREADS / 128 - 2) * REGS_OTHER == (F8 ? 4 * 128 : 3 * 168), "register shares");
    // TMEM columns: S of A and B, O of A and B; P takes the first half of
    // its S (D = 128), or columns of its own where there are some (D = 64)
    static constexpr int TM_O = 2 * CT;
    __host__ __device__ static constexpr int tm_s(int x) { return x * CT; }
    __host__ __device__ static constexpr int tm_o(int x) { return TM_O + x * D; }
    __host__ __device__ static constexpr int tm_p(int x) { return D == 128 ? x * CT : TM_O + 2 * D + x * (CT / 2); }
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr float TAU = 8.f;
    // f16 weights carry a factor 2^7 (the sum does too): below 2^-14 an f16
    // loses bits, above 2^16 it overflows, and 2^(TAU + 7) stays below that.
    // bf16 has float32's range and needs none.
    static constexpr float SHIFT = std::is_same<T, __half>::value ? 7.f : 0.f;
    static constexpr uint32_t SLEEP_NS = 100000;
    // barriers: ring full/empty, S, both halves of P, O, Q full, Q empty of both sub-tiles,
    // segments full/empty, the last commit, raw ring full/empty
    static constexpr int NBAR = 2 * STAGES + 12 + 2 * SEGS + 1 + 2 * RAWS;
    static constexpr int SMEM = 1024 + STAGES * BLOCK_BYTES + RAWS * RAW_BYTES + 2 * Q_BYTES + NBAR * 8 + 16 + SEGS * 64;
    static_assert(SMEM <= 232448, "shared memory");
};

// What the roles of a CTA need to know of a segment: a range of K/V blocks
// of one item.
struct ExtSeg {
    int valid;
    int row0, ntok;      // the tile's first row of q and out, its tokens
    int h, slice, b;
    int m, lim, k0;
    int blk0, blk[2];    // blocks [blk0, blk[x]) of sub-tile x
    int slot;            // partial result, or -1: the whole item
};

__device__ __forceinline__ int ext_end(const ExtSeg &g) { return max(g.blk[0], g.blk[1]); }

// 32 bytes at a 32-byte aligned address in one store.
__device__ __forceinline__ void stg256(void *ptr, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(ptr), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 32 consecutive outputs, times f, from index idx (a multiple of 32) of a
// 16-byte aligned tensor.  A thread writes its own row, so a store touches
// as many lines as the warp has rows whatever its width: 32-byte stores (a
// whole sector each) where the tensor allows them.
__device__ __forceinline__ void store_out32(void *out, long long idx, int out_dtype, const float *x, float f)
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
                w[e] = __float_as_uint(x[8 * i + e] * f);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = x[(16 * i + 2 * e) & 31] * f, b = x[(16 * i + 2 * e + 1) & 31] * f;
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

// 16 E4M3 values as the 16-bit type, exactly: two 16-byte vectors.
template <typename T> __device__ __forceinline__ void e4m3_widen16(const uint4 &u, uint4 &lo, uint4 &hi)
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
    if (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = Mma<__half>::unpack(r[i]);
            r[i] = Mma<__nv_bfloat16>::pack(f.x, f.y);
        }
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

template <typename T, int D, bool F8>
__global__ void __launch_bounds__(ExtCfg<T, D, F8>::THREADS, 1) extend_kernel(const __grid_constant__ ExtendParams p)
{
    using C = ExtCfg<T, D, F8>;
    constexpr int ST = C::STAGES;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the merge waits for this grid's end
    extern __shared__ __align__(128) unsigned char smem_raw[];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);   // 1024-aligned
    const uint32_t ring = smem_addr(smem);
    const uint32_t rawring = ring + ST * C::BLOCK_BYTES;
    const uint32_t qbuf = rawring + C::RAWS * C::RAW_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + ST * C::BLOCK_BYTES + C::RAWS * C::RAW_BYTES + 2 * C::Q_BYTES);
    uint32_t *misc = reinterpret_cast<uint32_t *>(bars + C::NBAR);
    volatile ExtSeg *segs = reinterpret_cast<volatile ExtSeg *>(misc + 4);
    static_assert(sizeof(ExtSeg) <= 64, "segment slots");
    const uint32_t bar0 = smem_addr(bars);
    auto FULL = [&](int s) { return bar0 + 8u * (uint32_t)s; };
    auto EMPTY = [&](int s) { return bar0 + 8u * (uint32_t)(ST + s); };
    constexpr int B0 = 2 * ST;
    auto SFULL = [&](int x) { return bar0 + 8u * (uint32_t)(B0 + x); };
    auto PFULL = [&](int x, int half) { return bar0 + 8u * (uint32_t)(B0 + 2 + 2 * x + half); };
    auto OFULL = [&](int x) { return bar0 + 8u * (uint32_t)(B0 + 6 + x); };
    auto QFULL = [&](int x) { return bar0 + 8u * (uint32_t)(B0 + 8 + x); };
    auto QEMPTY = [&](int x) { return bar0 + 8u * (uint32_t)(B0 + 10 + x); };
    auto GFULL = [&](int s) { return bar0 + 8u * (uint32_t)(B0 + 12 + s); };
    auto GEMPTY = [&](int s) { return bar0 + 8u * (uint32_t)(B0 + 12 + C::SEGS + s); };
    const uint32_t FIN = bar0 + 8u * (uint32_t)(B0 + 12 + 2 * C::SEGS);
    auto RFULL = [&](int s) { return FIN + 8u * (uint32_t)(1 + s); };
    auto REMPTY = [&](int s) { return FIN + 8u * (uint32_t)(1 + C::RAWS + s); };

    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(FULL(s), F8 ? 4 : 1);   // the producer's arrival plus the copy's bytes, or the converting warps
            mbar_init(EMPTY(s), 1);   // commit behind the block's last MMA
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(SFULL(x), 1);   // commit behind S
            // the sub-tile's warps: S read, O rescaled, a half of P written
            mbar_init(PFULL(x, 0), 4);
            mbar_init(PFULL(x, 1), 4);
            mbar_init(OFULL(x), 1);   // commit behind the segment's last P.V
            mbar_init(QFULL(x), 1);
            mbar_init(QEMPTY(x), 1);  // commit behind the segment's last S
        }
        for (int s = 0; s < C::SEGS; ++s) {
            mbar_init(GFULL(s), 1);
            mbar_init(GEMPTY(s), F8 ? 15 : 11); // K/V, MMA, Q, the eight softmax warps and the converting ones
        }
        for (int s = 0; s < C::RAWS; ++s) {
            mbar_init(RFULL(s), 1);
            mbar_init(REMPTY(s), 4);
        }
        mbar_init(FIN, 1);
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
    bool dead = false;
    int sg = 0;   // segments taken so far

    // The next segment, by a whole warp; false at the end (or on expiry).
    auto next_seg = [&](ExtSeg &g) {
        const int s = sg % C::SEGS;
        if (!mbar_wait_bounded_soon(GFULL(s), (uint32_t)((sg / C::SEGS) & 1), C::SLEEP_NS)) {
            dead = true;
            return false;
        }
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
        g.blk[0] = x.blk[0];
        g.blk[1] = x.blk[1];
        g.slot = x.slot;
        __syncwarp();
        if (lane == 0)
            mbar_arrive(GEMPTY(s));
        ++sg;
        return g.valid != 0;
    };

    // (a warpgroup changes its share of the registers as a whole)
    if (w >= 8) {
        regs_dec<C::REGS_OTHER>();
    if (w == C::SCHED_WARP) {
        // ------------------------------------------------------------ scheduler
        if (lane == 0) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            const int G = p.grid, c = blockIdx.x, Hv = p.Hkv * p.NG;
            const ExtPlanHeader hd = *p.header;
            const ExtCut a = p.cuts[c], e = p.cuts[c + 1];
            // a segment of item `it`, blocks [blk0, blk1)
            auto push = [&](int it, const ExtTile &t, int blk0, int blk1, int slot) {
                const int s = sg % C::SEGS;
                if (sg >= C::SEGS && !mbar_wait_bounded_sleep_thread(GEMPTY(s), (uint32_t)(((sg / C::SEGS) - 1) & 1),
                                                                     C::SLEEP_NS)) {
                    dead = true;
                    return;
                }
                volatile ExtSeg &g = segs[s];
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
                    g.blk[x] = max(blk0, min(blk1, end));
                }
                g.slot = slot;
                mbar_arrive(GFULL(s));
                ++sg;
            };
            for (int it = a.item; it < hd.n_items && !dead; ++it) {
                const bool last = it == e.item;
                if (it > e.item || (last && e.off == 0))
                    break;
                const ExtTile t = p.tiles[it / Hv];
                const bool fresh = it > a.item || a.off == 0;
                const int b0 = it > a.item ? 0 : a.blk, b1 = last ? e.blk : t.nblk;
                if (t.nblk == 0 ? !fresh : b1 <= b0)
                    continue;
                const bool whole = b0 == 0 && b1 == t.nblk;
                push(it, t, b0, b1, whole ? -1 : b0 > 0 ? 2 * c + 1 : 2 * (c + 1));
            }
            for (int x = 0; x < hd.waves && !dead; ++x) {
                const int it = x * G + ((x & 1) ? G - 1 - c : c);
                const ExtTile t = p.tiles[it / Hv];
                push(it, t, 0, t.nblk, -1);
            }
            if (!dead) {
                const ExtTile none = {};
                push(-1, none, 0, 0, -1);
            }
        }
        __syncwarp();
    } else if (w == C::KV_WARP) {
        // ------------------------------------------------------------ K and V
        // Blocks K(j), V(j), K(j+1), ...: each lane one box of a block (row
        // group, plane), so the rows of a block may come from several pages.
        const int R = p.paged ? p.box_rows : C::CT;
        const int ng = C::CT / R;   // row groups (at most 8)
        const int grp = lane % ng, plane = lane / ng;
        const bool mine = plane < (F8 ? 1 : C::PLANES);
        constexpr int NS = F8 ? C::RAWS : ST;
        auto NFULL = [&](int s) { return F8 ? RFULL(s) : FULL(s); };
        auto NEMPTY = [&](int s) { return F8 ? REMPTY(s) : EMPTY(s); };
        long long n = 0;            // blocks issued
        ExtSeg g;
        while (!dead && next_seg(g)) {
            const int end = ext_end(g);
#pragma unroll 1
            for (int j = g.blk0; j < end && !dead; ++j) {
                int x = 0, y = 0;
                const int tok = j * C::CT + grp * R;
                const bool load = mine && tok < g.m;
                if (!p.paged) {
                    x = g.k0 + tok;
                    y = g.h;
                } else if (load) {
                    int page = p.table[(long long)g.b * p.max_pages + tok / p.page_size];
                    if (page < 0 || page >= p.num_pages) {
                        atomicOr(p.status, STATUS_BAD_PAGE);
                        page = 0;
                    }
                    x = tok % p.page_size;
                    y = page * p.Hkv + g.h;
                }
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(FULL_MASK, load)) * (uint32_t)(R * (F8 ? D : 128));
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++n) {
                    const int s = (int)(n % NS);
                    if (n >= NS &&
                        !mbar_wait_bounded_soon(NEMPTY(s), (uint32_t)(((n / NS) - 1) & 1), C::SLEEP_NS)) {
                        dead = true;
                        break;
                    }
                    if (lane == 0)
                        mbar_arrive_expect_tx(NFULL(s), bytes);
                    __syncwarp();
                    const CUtensorMap *tm = kv ? &p.tmv : &p.tmk;
                    if (F8 && load)
                        tma_load_3d(rawring + (uint32_t)(s * C::RAW_BYTES + grp * R * D), tm, 0, x, y, NFULL(s));
                    else if (load)
                        tma_load_4d(ring + (uint32_t)(s * C::BLOCK_BYTES + plane * C::PLANE + grp * R * 128), tm, 0, x, y,
                                    plane, NFULL(s));
                }
            }
        }
        // no copy may be in flight when the CTA ends: the last fill of each stage
        for (long long i = n > NS ? n - NS : 0; i < n; ++i)
            mbar_wait_bounded_soon(NFULL((int)(i % NS)), (uint32_t)((i / NS) & 1), C::SLEEP_NS);
    } else if (F8 && w >= C::CVT_WARP) {
        // ------------------------------------------------------------ E4M3 to 16 bits
        // A thread widens 16 values of a row at a time into the swizzled
        // planes that the MMAs read.  Eight lanes read 128 bytes in a row;
        // at d = 128 the upper four write the other plane, their two halves
        // in the other order, so that the eight 16-byte writes of a phase
        // fall in different banks.
        constexpr int NR = F8 ? C::RAWS : 1;
        constexpr int CPR = D / 16;   // 16-value pieces of a row
        const int ct = tid - C::CVT_WARP * 32;
        const int c = ct % CPR, r0 = ct / CPR;
        const bool swap = (c >> 2) != 0;
        long long n = 0;
        ExtSeg g;
        while (!dead && next_seg(g)) {
            const int end = ext_end(g);
#pragma unroll 1
            for (int j = g.blk0; j < end && !dead; ++j) {
                const int left = g.m - j * C::CT;
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++n) {
                    const int rs = (int)(n % NR), s = (int)(n % ST);
                    if (!mbar_wait_bounded_soon(RFULL(rs), (uint32_t)((n / NR) & 1), C::SLEEP_NS) ||
                        (n >= ST && !mbar_wait_bounded_soon(EMPTY(s), (uint32_t)(((n / ST) - 1) & 1), C::SLEEP_NS))) {
                        dead = true;
                        break;
                    }
                    const uint32_t src = rawring + (uint32_t)(rs * C::RAW_BYTES);
                    const uint32_t dst = ring + (uint32_t)(s * C::BLOCK_BYTES + (c >> 2) * C::PLANE);
#pragma unroll 4
                    for (int r = r0; r < C::CT; r += 128 / CPR) {
                        uint4 v = lds128(src + (uint32_t)(r * D + c * 16));
                        // rows behind the sequence's last key may hold
                        // anything, and 0 * NaN is NaN
                        if (r >= left)
                            v = make_uint4(0, 0, 0, 0);
                        uint4 lo, hi;
                        e4m3_widen16<T>(v, lo, hi);
                        const uint32_t a0 = dst + (uint32_t)(r * 128 + (((2 * (c & 3)) ^ (r & 7)) << 4));
                        const uint32_t a1 = dst + (uint32_t)(r * 128 + (((2 * (c & 3) + 1) ^ (r & 7)) << 4));
                        sts128(swap ? a1 : a0, swap ? hi : lo);
                        sts128(swap ? a0 : a1, swap ? lo : hi);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(FULL(s));
                        mbar_arrive(REMPTY(rs));
                    }
                }
            }
        }
    } else if (w == C::Q_WARP) {
        // ------------------------------------------------------------ Q
        // A sub-tile's rows: tps tokens of Gs heads each, plane by plane.
        // Rows behind the sequence's are other sequences' (or zeros): they
        // are computed and not written out.
        int n[2] = {0, 0};
        ExtSeg g;
        while (!dead && next_seg(g)) {
            if (lane == 0) {
                for (int x = 0; x < 2 && !dead; ++x) {
                    if (g.blk[x] <= g.blk0)
                        continue;
                    if (n[x] > 0 &&
                        !mbar_wait_bounded_sleep_thread(QEMPTY(x), (uint32_t)((n[x] - 1) & 1), C::SLEEP_NS)) {
                        dead = true;
                        break;
                    }
                    mbar_arrive_expect_tx(QFULL(x), (uint32_t)(C::PLANES * p.tps * p.Gs * 128));
                    for (int pl = 0; pl < C::PLANES; ++pl)
                        tma_load_4d(qbuf + (uint32_t)(x * C::Q_BYTES + pl * C::PLANE), &p.tmq, 0,
                                    g.h * p.G + g.slice * p.Gs, g.row0 + x * p.tps, pl, QFULL(x));
                    ++n[x];
                }
            }
            dead = __any_sync(FULL_MASK, dead);
        }
        if (lane == 0) {
            for (int x = 0; x < 2; ++x)
                if (n[x] > 0)
                    mbar_wait_bounded_sleep_thread(QFULL(x), (uint32_t)((n[x] - 1) & 1), C::SLEEP_NS);
        }
        __syncwarp();
    } else if (w == C::MMA_WARP) {
        // ------------------------------------------------------------ MMA issue
        constexpr int BF = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
        constexpr uint32_t ID_S = idesc_f16(BF, 0, 0, C::M, C::CT);   // Q K-major, K K-major
        constexpr uint32_t ID_O = idesc_f16(BF, 0, 1, C::M, D);       // P (TMEM) K-major, V MN-major
        long long n = 0;              // blocks taken from the ring
        int ns[2] = {0, 0};           // P of each sub-tile taken
        int nq[2] = {0, 0};           // Q of each sub-tile taken
        auto wait = [&](uint32_t bar, int phase) {
            if (!dead && !mbar_wait_bounded_soon(bar, (uint32_t)(phase & 1), C::SLEEP_NS))
                dead = true;
            return !dead;
        };
        // Descriptors: a base, plus offsets in its units of 16 bytes (an
        // address fits the field, so no carry leaves it).
        const uint64_t qdesc = smem_desc_sw128(qbuf, 16, 1024), kdesc = smem_desc_sw128(ring, 16, 1024);
        const uint64_t vdesc = smem_desc_sw128(ring, (uint32_t)C::PLANE, 1024);
        const uint32_t one = elect_one();
        auto issue_s = [&](int x, int st) {
            const uint64_t a = qdesc + (uint64_t)(x * (C::Q_BYTES >> 4)), b = kdesc + (uint64_t)(st * (C::BLOCK_BYTES >> 4));
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                // 16 elements = 32 bytes of each 128-byte row of plane ks / 4
                const uint64_t o = (uint64_t)(((ks >> 2) * C::PLANE + (ks & 3) * 32) >> 4);
                tc_mma_ss_if(one, tmem + (uint32_t)C::tm_s(x), a + o, b + o, ID_S, ks > 0 ? 1u : 0u);
            }
            tc_commit_if(one, SFULL(x));
        };
        // the keys of one half of P
        auto issue_pv = [&](int x, int st, int half, bool first) {
            const uint64_t b = vdesc + (uint64_t)(st * (C::BLOCK_BYTES >> 4));
#pragma unroll
            for (int i = 0; i < C::CT / 32; ++i) {
                const int ks = half * (C::CT / 32) + i;
                tc_mma_ts_if(one, tmem + (uint32_t)C::tm_o(x), tmem + (uint32_t)(C::tm_p(x) + ks * 8),
                             b + (uint64_t)(ks * (2048 >> 4)), ID_O, (!first || ks > 0) ? 1u : 0u);
            }
        };
        ExtSeg g;
        while (!dead && next_seg(g)) {
            const int end = ext_end(g);
            if (end <= g.blk0)
                continue;
            // S of the first block
            {
                const int s = (int)(n % ST);
                if (!wait(FULL(s), (int)((n / ST) & 1)))
                    break;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (g.blk[x] <= g.blk0)
                        continue;
                    if (!wait(QFULL(x), nq[x]))
                        break;
                    ++nq[x];
                    tc_fence_after();
                    issue_s(x, s);
                    if (g.blk[x] == g.blk0 + 1)
                        tc_commit_if(one, QEMPTY(x));
                }
                if (dead)
                    break;
                tc_commit_if(one, EMPTY(s));
                ++n;
            }
#pragma unroll 1
            for (int j = g.blk0; j < end && !dead; ++j) {
                const int vs = (int)(n % ST);
                const int vph = (int)((n / ST) & 1);
                ++n;
                const int ks = (int)(n % ST);
                const int kph = (int)((n / ST) & 1);
                const bool more = j + 1 < end;
                if (!wait(FULL(vs), vph))
                    break;
                const int left = g.m - j * C::CT;
                if (!F8 && left < C::CT) {
                    // V's rows behind the sequence's last key may hold
                    // anything, and 0 * NaN is NaN: zeros instead
                    const uint32_t vb = ring + (uint32_t)(vs * C::BLOCK_BYTES);
                    for (int i = lane; i < (C::CT - left) * C::PLANES * 8; i += 32) {
                        const int pl = i / ((C::CT - left) * 8), o = i % ((C::CT - left) * 8);
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         vb + (uint32_t)(pl * C::PLANE + left * 128 + o * 16)),
                                     "r"(0u)
                                     : "memory");
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                bool kready = false;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (j < g.blk[x]) {
                        if (!wait(PFULL(x, 0), ns[x]))
                            break;
                        tc_fence_after();
                        issue_pv(x, vs, 0, j == g.blk0);
                        if (!wait(PFULL(x, 1), ns[x]))
                            break;
                        ++ns[x];
                        tc_fence_after();
                        issue_pv(x, vs, 1, false);
                        if (j + 1 == g.blk[x])
                            tc_commit_if(one, OFULL(x));
                    }
                    if (x == 1)
                        tc_commit_if(one, EMPTY(vs));
                    if (j + 1 < g.blk[x]) {
                        if (!kready && !wait(FULL(ks), kph))
                            break;
                        kready = true;
                        tc_fence_after();
                        issue_s(x, ks);
                        if (j + 2 == g.blk[x])
                            tc_commit_if(one, QEMPTY(x));
                    }
                }
                if (dead)
                    break;
                if (more) {
                    tc_commit_if(one, EMPTY(ks));
                    ++n;
                }
            }
        }
        // every MMA issued here has completed before TMEM is freed
        __syncwarp();
        tc_commit_if(one, FIN);
        if (!mbar_wait_bounded_soon(FIN, 0, C::SLEEP_NS))
            dead = true;
    }
    } else {
        regs_inc<C::REGS_SOFTMAX>();
        // ------------------------------------------------------------ softmax
        const int x = w >> 2;              // sub-tile
        const int row = tid & 127;         // its row = TMEM lane
        const uint32_t tl = tmem + ((uint32_t)((w & 3) * 32) << 16);
        const int rtok = row / p.Gs, rg = row % p.Gs;
        const int tok = x * p.tps + rtok;  // token within the tile
        int ns = 0, no = 0;
        ExtSeg g;
        while (!dead && next_seg(g)) {
            const int gv = min(p.Gs, p.G - g.slice * p.Gs);
            const bool live = rtok < p.tps && tok < g.ntok && rg < gv;
            // keys this row sees; a row that is not written takes those of
            // the last one, so that its warp masks no block for its sake
            const int lim = p.causal ? min(g.m, g.lim + min(tok, g.ntok - 1)) : g.m;
            float sc = p.scale_log2;
            float vscale = 1.f;
            if (F8) {
                sc *= __ldg(p.k_scale + (long long)g.b * p.Hkv + g.h);
                vscale = __ldg(p.v_scale + (long long)g.b * p.Hkv + g.h);
            }
            float mref = -INFINITY, l = 0.f;
            const int end = g.blk[x];
            // blocks below this one hide nothing from any row of the warp
            const int whole = __reduce_min_sync(FULL_MASK, max(lim, 0)) / C::CT;
#pragma unroll 1
            for (int j = g.blk0; j < end; ++j) {
                if (!mbar_wait_bounded_soon(SFULL(x), (uint32_t)(ns & 1), C::SLEEP_NS)) {
                    dead = true;
                    break;
                }
                ++ns;
                tc_fence_after();
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
                // the tcgen05 loads and stores are warp-wide, so the whole
                // warp runs them when any of its rows grew (a = 1 for others)
                if (j > g.blk0 && __any_sync(FULL_MASK, grow)) {
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
                    if (i & 1) {
                        // half of P: its product with V may start
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(PFULL(x, i >> 1));
                    }
                }
                float la, lb;
                unpack2(add2(add2(ls[0], ls[1]), add2(ls[2], ls[3])), la, lb);
                l += la + lb;
            }
            if (dead)
                break;

            // ---- the segment's result ----
            const bool some = end > g.blk0;
            if (some) {
                if (!mbar_wait_bounded_soon(OFULL(x), (uint32_t)(no & 1), C::SLEEP_NS)) {
                    dead = true;
                    break;
                }
                ++no;
                tc_fence_after();
            }
            const bool any = !(l <= 0.f);   // NaN counts: it is the result then
            const float inv = any ? vscale / l : 0.f;
            const long long qrow = (long long)(g.row0 + tok) * p.Hq + g.h * p.G + g.slice * p.Gs + rg;
            const long long prow = ((long long)g.slot * 2 + x) * C::M + row;
            // an empty row is 0 whatever its accumulator holds
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                float o[32];
                if (some) {
                    tmem_ld32(tl + (uint32_t)(C::tm_o(x) + 32 * q), o);
                    tmem_wait_ld();
                }
                if (!some || !any) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = 0.f;
                }
                if (live && g.slot >= 0)
                    store_out32(p.part_o, prow * D + 32 * q, 0, o, 1.f);
                else if (live)
                    store_out32(p.out, qrow * D + 32 * q, p.out_dtype, o, inv);
                __syncwarp();
            }
            tc_fence_before();   // the next segment's P.V overwrites O behind this warp's next P
            if (live) {
                if (g.slot >= 0)
                    p.part_ml[prow] = make_float2(any ? mref - C::SHIFT : -INFINITY, l);
                else if (p.lse)
                    p.lse[qrow] = any ? (mref - C::SHIFT + log2f(l)) * 0.6931471805599453f : -INFINITY;
            }
        }
    }

    if (dead && lane == 0)
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
