// fd_extend_plan.cu -- what the attention of new tokens runs before and after
// its main kernel: the plan, made on the GPU from the sequences' lengths,
// and the merge of the tiles that were split over their keys.
//
// A tile costs its blocks of keys plus EXT_START for its queries, its result
// and the pipeline's refill.  Items (tile, virtual head) are dealt in
// descending cost: whole waves of one item a CTA, back and forth, as long as
// no CTA gets more than its even share of the total; what is left is cut
// into pieces that fill every CTA up to that share, at any block.  So few
// long tiles (a few drafted tokens over a long cache) are split over all
// SMs, many are mostly whole, and neighbours in a wave stream the same K/V.
// Everything follows from prefix sums in a fixed order: the split, and with
// it every rounding, is the same in every run.
//
// The plan is one CTA's chain of dependent steps (loads, scans, two passes of
// a sort, a bisection), bound by their latency: 5 us for one tile, 6 for 87,
// some 10 for 623 with 15 waves.  A smaller tail of cut items (whole ones
// where they are short) did not pay, nor did a scan out of line (+0.3 us).
// The merge reads every partial result once, from L2: some 6 us for the 151
// cut items of a mixed batch (14 with a warp a row), 2 where nothing is cut.
#include "fd_device.cuh"
#include "fd_extend.h"

namespace fd {
namespace {

constexpr int PT = 512;         // threads of the planning CTA
constexpr int PW = PT / 32;
static_assert(EXT_MAX_GRID < PT, "a thread a cut");
constexpr int BUCKETS = 64;     // of the sort by cost
constexpr int EXT_START = 3;    // cost of an item beside its blocks, in blocks
constexpr int EXT_MIN_CUT = EXT_START + 1;   // a share of the cut items is a block at least
constexpr int NEAR = 2048;      // up to so many sequences, or tiles, the tables below are in shared memory

// Inclusive sums over the block, and their total.
__device__ __forceinline__ long long scan_block(long long x, long long *warp_sums, long long &total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(FULL_MASK, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();   // the sums of the previous call have been read
    if (lane == 31)
        warp_sums[w] = x;
    __syncthreads();
    // every warp sums the warps before it, and all of them
    const long long s = lane < PW ? warp_sums[lane] : 0;
    long long before = lane < w ? s : 0, all = s;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        before += __shfl_xor_sync(FULL_MASK, before, o);
        all += __shfl_xor_sync(FULL_MASK, all, o);
    }
    total = all;
    return x + before;
}

__device__ __forceinline__ int max_block(int x, int *warp_max)
{
    x = __reduce_max_sync(FULL_MASK, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        warp_max[threadIdx.x >> 5] = x;
    __syncthreads();
    return __reduce_max_sync(FULL_MASK, warp_max[min(threadIdx.x & 31, PW - 1u)]);
}

// Sequence b's rows of q, clamped; true if the offsets had to be.
__device__ __forceinline__ bool q_rows(const ExtendParams &p, int b, int &lo, int &n)
{
    const int a = p.cu_q[b], e = p.cu_q[b + 1];
    lo = min(max(a, 0), p.total_q);
    n = min(max(e, lo), p.total_q) - lo;
    return lo != a || lo + n != e;
}

// Its keys, likewise.
__device__ __forceinline__ bool k_rows(const ExtendParams &p, int b, int &lo, int &m)
{
    if (p.paged) {
        lo = 0;
        m = (int)min((long long)max(p.seqlens[b], 0), (long long)p.page_size * p.max_pages);
        return false;
    }
    const int a = p.cu_k[b], e = p.cu_k[b + 1];
    lo = min(max(a, 0), p.total_k);
    m = min(max(e, lo), p.total_k) - lo;
    return lo != a || lo + m != e;
}

// Tile i (of all, in order of the sequences), of the tiles before each
// sequence.
__device__ __forceinline__ ExtTile tile_at(const ExtendParams &p, const int *tile_start, int i)
{
    int lo = 0, hi = p.B - 1;   // the last b with tile_start[b] <= i
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tile_start[mid] <= i)
            lo = mid;
        else
            hi = mid - 1;
    }
    ExtTile t;
    int r, n;
    q_rows(p, lo, r, n);
    k_rows(p, lo, t.k0, t.m);
    const int first = (i - tile_start[lo]) * 2 * p.tps;
    t.b = lo;
    t.row0 = r + first;
    t.ntok = min(2 * p.tps, n - first);
    // a token that sees nothing counts as negative or 0; m - n + first + 1 fits
    t.lim = p.causal ? t.m - n + first + 1 : t.m;
    const int see = p.causal ? min(t.m, t.lim + t.ntok - 1) : t.m;
    t.nblk = see > 0 ? (see + EXT_CT - 1) / EXT_CT : 0;
    t.pad = 0;
    return t;
}

__global__ void __launch_bounds__(PT, 1) extend_plan_kernel(const ExtendParams p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ long long sums[PW];
    __shared__ int maxs[PW];
    __shared__ int near_blk[NEAR];
    __shared__ long long near_sum[NEAR + 1];
    __shared__ int near_start[NEAR];
    __shared__ int hist[BUCKETS * PW];   // bucket-major, then warp
    __shared__ ExtCut near_cut[PT];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int Hv = p.Hkv * p.NG;
    const int tt = 2 * p.tps;

    int *start = p.B <= NEAR ? near_start : p.tile_start;

    // tiles before each sequence, and the most blocks of any tile
    long long tiles = 0;
    int top = 0;
    bool bad = false;
    for (int b0 = 0; b0 < p.B; b0 += PT) {
        const int b = b0 + tid;
        long long nt = 0, total;
        if (b < p.B) {
            int lo, n, k0, m;
            bad |= q_rows(p, b, lo, n);
            bad |= k_rows(p, b, k0, m);
            nt = (n + tt - 1) / tt;
            if (n > 0)
                top = max(top, (m + EXT_CT - 1) / EXT_CT);
        }
        const long long s = tiles + scan_block(nt, sums, total);
        tiles += total;
        if (b < p.B)
            start[b] = (int)min(s - nt, (long long)p.max_tiles);
    }
    if (bad)
        atomicOr(p.status, STATUS_BAD_OFFSETS);
    const int n = (int)min(tiles, (long long)p.max_tiles);   // fewer only if offsets overlap
    top = max(1, max_block(top, maxs));
    int *blk = n <= NEAR ? near_blk : p.tile_blk;   // blocks of the sorted tiles
    long long *sum = n <= NEAR ? near_sum : p.cost_sum;

    // stable counting sort by descending cost, each warp its share in order
    for (int i = tid; i < BUCKETS * PW; i += PT)
        hist[i] = 0;
    __syncthreads();
    const int share = ((n + PW - 1) / PW + 31) & ~31;
    const int i0 = w * share, i1 = min(n, i0 + share);
    ExtTile t = {};       // a thread's last one: its only one up to PT tiles
    int key = BUCKETS;
    auto take = [&](int i) {
        if (i < i1) {
            t = tile_at(p, start, i);
            // blocks are fewer than 2^25
            key = BUCKETS - 1 - (int)((unsigned)t.nblk * (unsigned)(BUCKETS - 1) / (unsigned)top);
        } else {
            key = BUCKETS;
        }
    };
    for (int i = i0; i < i1; i += 32) {
        take(i + lane);
        const bool on = i + lane < i1;
        const unsigned same = __match_any_sync(FULL_MASK, key);
        if (on && lane == __ffs(same) - 1)
            hist[key * PW + w] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    {
        const int h0 = hist[2 * tid], h1 = hist[2 * tid + 1];
        long long total;
        const int s = (int)scan_block(h0 + h1, sums, total);
        hist[2 * tid] = s - h0 - h1;
        hist[2 * tid + 1] = s - h1;
    }
    static_assert(BUCKETS * PW == 2 * PT, "two counts a thread");
    __syncthreads();
    for (int i = i0; i < i1; i += 32) {
        if (share > 32)
            take(i + lane);
        const bool on = i + lane < i1;
        const unsigned same = __match_any_sync(FULL_MASK, key);
        int at = 0;
        if (on)
            at = hist[key * PW + w] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (on) {
            p.tiles[at] = t;
            blk[at] = t.nblk;
            if (lane == __ffs(same) - 1)
                hist[key * PW + w] += __popc(same);
        }
        __syncwarp();
    }
    __syncthreads();

    // costs before each tile, over its virtual heads
    long long all = 0;
    for (int j0 = 0; j0 < n; j0 += PT) {
        const int j = j0 + tid;
        long long total;
        const long long c = j < n ? (long long)Hv * (blk[j] + EXT_START) : 0;
        const long long s = all + scan_block(c, sums, total);
        all += total;
        if (j < n)
            sum[j] = s - c;
    }
    if (tid == 0)
        sum[n] = all;
    __syncthreads();

    // whole waves, as many as leave every CTA within its even share
    const int G = p.grid;
    const long long items = (long long)n * Hv;
    const long long even = (all + G - 1) / G;
    int waves = (int)(items / G);
    if (n > 0 && blk[0] + EXT_START > even)
        waves = 0;
    long long load = 0;
    if (waves > 0) {
        // the tiles of this CTA's items, an even and an odd wave at a time:
        // items 2 G further on, without a division a step
        const int dj = 2 * G / Hv, dh = 2 * G % Hv;
        int fit = waves;   // waves that leave the CTA within the share
        auto walk = [&](int upto, auto each) {
            int ja = tid / Hv, ha = tid % Hv, jb = (2 * G - 1 - tid) / Hv, hb = (2 * G - 1 - tid) % Hv;
            for (int x = 0; x < upto; x += 2) {
                each(x, blk[ja] + EXT_START);
                if (x + 1 < upto)
                    each(x + 1, blk[jb] + EXT_START);
                ja += dj, ha += dh, jb += dj, hb += dh;
                if (ha >= Hv)
                    ha -= Hv, ++ja;
                if (hb >= Hv)
                    hb -= Hv, ++jb;
            }
        };
        if (tid < G) {
            long long sofar = 0;
            walk(waves, [&](int x, int cost) {
                sofar += cost;
                if (sofar > even)
                    fit = min(fit, x);
            });
        }
        waves = -max_block(-fit, maxs);
        if (tid < G)
            walk(waves, [&](int, int cost) { load += cost; });
    }

    // what is left, cut so that every CTA reaches the even share
    const long long first = (long long)waves * G;
    const int jf = (int)(first / Hv), hf = (int)(first % Hv);
    const long long base = jf < n ? sum[jf] + (long long)hf * (blk[jf] + EXT_START) : all;
    const long long rest = all - base;
    long long cap = 0;
    if (tid < G) {
        if (rest < (long long)EXT_MIN_CUT * G) {
            // slivers are not worth a merge: fewer, even shares
            const long long g = max(1LL, rest / EXT_MIN_CUT);
            cap = tid < g ? (rest + g - 1) / g : 0;
        } else {
            cap = even - load;
        }
    }
    long long total;
    const long long cut = min(rest, scan_block(cap, sums, total) - cap) + base;
    if (tid <= G) {
        const long long v = tid < G ? cut : all;
        ExtCut c = {(int)items, 0, 0, 0};
        if (v < all) {
            int lo = 0, hi = n - 1;   // the last tile with cost_sum <= v
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (sum[mid] <= v)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int cost = blk[lo] + EXT_START;
            const long long in = v - sum[lo];
            c.item = lo * Hv + (int)(in / cost);
            c.off = (int)(in % cost);
            c.blk = max(0, c.off - EXT_START);
        }
        p.cuts[tid] = c;
        near_cut[tid] = c;
    }
    __syncthreads();

    // the items with cuts inside, for the merge: a thread at each first cut
    const bool is = tid > 0 && tid < G && near_cut[tid].blk > 0 &&
                    !(near_cut[tid - 1].item == near_cut[tid].item && near_cut[tid - 1].blk > 0);
    ExtSplit sp = {};
    int rows = 0;
    if (is) {
        const int item = near_cut[tid].item;
        const ExtTile t = p.tiles[item / Hv];
        sp.c0 = tid;
        sp.c1 = tid + 1;
        while (sp.c1 < G && near_cut[sp.c1].item == item && near_cut[sp.c1].blk > 0)
            ++sp.c1;
        sp.row0 = t.row0;
        sp.ntok = t.ntok;
        sp.b = t.b;
        sp.vh = item % Hv;
        rows = t.ntok * p.Gs;
    }
    // counts below 2^20, rows below 2^40: one scan for both
    const long long both = scan_block(((long long)rows << 20) | (is ? 1 : 0), sums, total);
    if (is) {
        sp.rows = (int)(both >> 20) - rows;
        p.splits[(int)(both & ((1 << 20) - 1)) - 1] = sp;
    }
    if (tid == 0) {
        ExtPlanHeader hd;
        hd.n_items = (int)items;
        hd.waves = waves;
        hd.n_splits = (int)(total & ((1 << 20) - 1));
        hd.split_rows = (int)(total >> 20);
        *p.header = hd;
    }
}

// The merge of the split items, 16 lanes a row, the pieces in the order of
// the cuts:
//     M = max m_i,  out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
// Every CTA reads the list of the split items and takes its share of their
// rows.
constexpr int MT = 256;         // threads
constexpr int ML = 16;          // lanes a row
constexpr int U = 4;            // pieces in flight

template <int D> __global__ void __launch_bounds__(MT) extend_merge_kernel(const ExtendParams p)
{
    __shared__ ExtSplit splits[EXT_MAX_GRID];
    __shared__ int cut_blk[EXT_MAX_GRID];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid % ML;
    const ExtPlanHeader hd = *p.header;
    for (int i = tid; i < p.grid; i += MT) {
        splits[i] = p.splits[i];   // (those behind the last are not used)
        cut_blk[i] = p.cuts[i].blk;
    }
    __syncthreads();
    constexpr int E = D / ML, V = E / 4;   // a lane's elements, in float4 that lie 64 apart
    for (int x = blockIdx.x * (MT / ML) + tid / ML; x < hd.split_rows; x += gridDim.x * (MT / ML)) {
        int lo = 0, hi = hd.n_splits - 1;   // the last item with rows <= x
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (splits[mid].rows <= x)
                lo = mid;
            else
                hi = mid - 1;
        }
        const ExtSplit t = splits[lo];
        const int h = t.vh / p.NG, s = t.vh % p.NG;
        const int gv = min(p.Gs, p.G - s * p.Gs), hq0 = h * p.G + s * p.Gs;
        const int tok = (x - t.rows) / p.Gs, g = (x - t.rows) % p.Gs;
        if (g >= gv)
            continue;
        const int r = tok / p.tps * EXT_M + tok % p.tps * p.Gs + g;   // its row of the partials
        float o[E], M = -INFINITY, L = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = 0.f;
        // the piece left of the first cut, then the one right of each cut
        // inside the item (none where two cuts coincide)
        for (int i = t.c0 - 1; i < t.c1; i += U) {
            float2 ml[U];
            float4 v[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = i + u;
                ml[u] = make_float2(-INFINITY, 0.f);
                if (k < t.c0 || (k < t.c1 && (k + 1 == t.c1 || cut_blk[k + 1] > cut_blk[k]))) {
                    const long long row = (long long)(k >= t.c0 ? 2 * k + 1 : 2 * t.c0) * 2 * EXT_M + r;
                    ml[u] = __ldcg(p.part_ml + row);
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        v[u][e] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + row * D) + lane + ML * e);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!(ml[u].y <= 0.f)) {
                    const float mn = fmaxf(M, ml[u].x);
                    const float a = ex2(M - mn), b = ex2(ml[u].x - mn);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        o[4 * e] = fmaf(b, v[u][e].x, a * o[4 * e]);
                        o[4 * e + 1] = fmaf(b, v[u][e].y, a * o[4 * e + 1]);
                        o[4 * e + 2] = fmaf(b, v[u][e].z, a * o[4 * e + 2]);
                        o[4 * e + 3] = fmaf(b, v[u][e].w, a * o[4 * e + 3]);
                    }
                    L = fmaf(L, a, b * ml[u].y);
                    M = mn;
                }
            }
        }
        const float vs = p.f8 ? p.v_scale[(long long)t.b * p.Hkv + h] : 1.f;
        const long long qrow = (long long)(t.row0 + tok) * p.Hq + hq0 + g;
        const bool any = !(L <= 0.f);   // NaN counts: it is the result then
        const float inv = any ? vs / L : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = any ? o[e] * inv : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const long long at = qrow * D + 4 * (lane + ML * e);
            const float *y = o + 4 * e;
            if (p.out_dtype == 0)
                *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
            else if (p.out_dtype == 1)
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
                    make_uint2(Mma<__half>::pack(y[0], y[1]), Mma<__half>::pack(y[2], y[3]));
            else
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
                    make_uint2(Mma<__nv_bfloat16>::pack(y[0], y[1]), Mma<__nv_bfloat16>::pack(y[2], y[3]));
        }
        if (p.lse && lane == 0)
            p.lse[qrow] = any ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    }
}

}  // namespace

cudaError_t launch_extend_plan(const ExtendParams &p, cudaStream_t s)
{
    extend_plan_kernel<<<1, PT, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_extend_merge(const ExtendParams &p, cudaStream_t s)
{
    if (p.grid < 2)
        return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(4 * p.grid);
    cfg.blockDim = dim3(MT);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return p.d == 64 ? cudaLaunchKernelEx(&cfg, extend_merge_kernel<64>, p)
                     : cudaLaunchKernelEx(&cfg, extend_merge_kernel<128>, p);
}

}  // namespace fd
