// fd_beam_pages.cu -- the beams' cached states reordered: every beam's block
// table and length to those of its parent, pages that no beam names any more
// back on the stack of free pages, and a page of its own for each beam that
// would share a partly filled one.
//
// Beams of a request name the same pages at the same places of their tables
// (what they grew from together), so all that is decided about a place follows
// from the W entries there:
//   - a page comes back if an old table names it and no new one does;
//   - a new beam whose last page is partly filled keeps it if it is the first
//     of those that name it (and none names it as a full one), else it gets a
//     page from the stack and the filled rows are copied.
// No counts of owners are kept anywhere.  The order on the stack is that of
// (request, place, beam), the first of them on top, so that pages taken by a
// request's first step come back in the order that undoes it; it follows from
// sums over requests and tiles, not from the order of threads.
//
// Four phases: what comes back and what is needed, a CTA a tile of a request's
// tables; the sums and who is granted, one CTA; the stack and the tables; the
// pages for copies and the lengths, a warp a request.
#include "fd_beam.h"
#include "fd_device.cuh"
#include "fd_pages.h"

#include <limits.h>

namespace fd {
namespace {

constexpr int RT = REORDER_TILE;   // threads of a CTA, one a place
constexpr int RW = RT / 32;
constexpr int ST = 1024;           // threads of the sums

__device__ __forceinline__ bool is_page(const ReorderParams &p, int page) { return page >= 0 && page < p.num_pages; }

// A request's beams: lengths, pages, parents (-1: none).
struct Beams {
    int len[BEAM_MAX_W], pages[BEAM_MAX_W], parent[BEAM_MAX_W];
    unsigned parents;   // those that are a parent
};

// (The block's first warp loads; all threads call.)
__device__ __forceinline__ void load_beams(const ReorderParams &p, int r, Beams &b, bool report)
{
    __syncthreads();
    if (threadIdx.x < 32) {
        const int w = threadIdx.x;
        int parent = -1;
        if (w < p.W) {
            const long long cap = (long long)p.max_pages * p.page_size;
            const int len = (int)min(max((long long)p.seqlens[r * p.W + w], 0LL), cap);
            b.len[w] = len;
            b.pages[w] = (int)(((long long)len + p.page_size - 1) / p.page_size);
            parent = p.parents[r * p.W + w];
            if (parent >= p.W) {
                parent = -1;
                if (report)
                    atomicOr(p.status, STATUS_BAD_INDEX);
            }
            b.parent[w] = max(parent, -1);
        }
        const unsigned mine = parent >= 0 ? 1u << parent : 0u;
        const unsigned all = __reduce_or_sync(FULL_MASK, mine);
        if (w == 0)
            b.parents = all;
    }
    __syncthreads();
}

// The entries of a tile: place j0 + thread of every beam that has it.
struct Tile {
    int e[BEAM_MAX_W][RT];
};

__device__ __forceinline__ void load_tile(const ReorderParams &p, int r, int j, const Beams &b, Tile &t)
{
#pragma unroll 8
    for (int w = 0; w < p.W; ++w)
        if (j < b.pages[w])
            t.e[w][threadIdx.x] = p.table[(long long)(r * p.W + w) * p.max_pages + j];
}

// The beams whose page at place j comes back, the first to name each.
__device__ __forceinline__ unsigned released(const ReorderParams &p, int j, const Beams &b, const Tile &t, bool &bad)
{
    const int tid = threadIdx.x;
    unsigned gone = 0;
    for (int w = 0; w < p.W; ++w) {
        if ((b.parents >> w & 1) || j >= b.pages[w])
            continue;   // a parent's pages stay
        const int page = t.e[w][tid];
        bool stays = !is_page(p, page);
        bad |= stays;
        for (int v = 0; v < p.W && !stays; ++v)
            if (j < b.pages[v] && ((b.parents >> v & 1) || (gone >> v & 1)))
                stays = t.e[v][tid] == page;
        if (!stays)
            gone |= 1u << w;
    }
    return gone;
}

__device__ __forceinline__ int block_sum(int x, int *warps)
{
    x = __reduce_add_sync(FULL_MASK, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        warps[threadIdx.x >> 5] = x;
    __syncthreads();
    int all = 0;
    for (int i = 0; i < RW; ++i)
        all += warps[i];
    return all;
}

// Phase 1: pages that come back of each tile; the copies a request needs.
__global__ void __launch_bounds__(RT) count_kernel(const ReorderParams p)
{
    __shared__ Beams b;
    __shared__ Tile t;
    __shared__ int warps[RW];
    const int r = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
    load_beams(p, r, b, tile == 0);
    const int j = tile * RT + threadIdx.x;
    load_tile(p, r, j, b, t);
    bool bad = false;
    const unsigned gone = released(p, j, b, t, bad);
    if (bad)
        atomicOr(p.status, STATUS_BAD_PAGE);
    const int n = block_sum(__popc(gone), warps);
    if (threadIdx.x == 0)
        p.freed[blockIdx.x] = n;

    if (tile == 0 && threadIdx.x < 32) {
        // new beam w: its parent's last page, if that is partly filled
        const int w = threadIdx.x;
        const int parent = w < p.W ? b.parent[w] : -1;
        const int rows = parent >= 0 ? b.len[parent] % p.page_size : 0;
        bool copy = false;
        int page = -1;
        if (rows) {
            const int at = b.len[parent] / p.page_size;
            page = p.table[(long long)(r * p.W + parent) * p.max_pages + at];
            for (int v = 0; v < p.W && !copy; ++v) {
                const int q = b.parent[v];
                if (v == w || q < 0 || at >= b.pages[q])
                    continue;
                // named by a beam before it, or as a full page by any
                if (v < w || b.len[q] / p.page_size > at)
                    copy = p.table[(long long)(r * p.W + q) * p.max_pages + at] == page;
            }
            if (!is_page(p, page)) {
                copy = false;
                atomicOr(p.status, STATUS_BAD_PAGE);
            }
        }
        if (w < p.W) {
            int32_t *c = p.copies + (long long)(r * p.W + w) * 3;
            c[0] = copy ? page : -1;
            c[1] = -1;
            c[2] = copy ? rows : 0;
        }
        const unsigned who = __ballot_sync(FULL_MASK, copy);
        if (w == 0)
            p.needed[r] = __popc(who);
    }
}

// Inclusive sums of N values over the block of ST threads, and their totals.
template <int N> struct Scan {
    long long warp[N][ST / 32];
    __device__ __forceinline__ void run(long long (&x)[N], long long (&total)[N])
    {
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const long long y = __shfl_up_sync(FULL_MASK, x[i], o);
                if (lane >= o)
                    x[i] += y;
            }
        }
        __syncthreads();   // the sums of the previous call have been read
        if (lane == 31) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                warp[i][w] = x[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const long long s = warp[i][lane];
            long long before = lane < w ? s : 0, all = s;
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                before += __shfl_xor_sync(FULL_MASK, before, o);
                all += __shfl_xor_sync(FULL_MASK, all, o);
            }
            x[i] += before;
            total[i] = all;
        }
    }
};

// Phase 2: who is granted, and what lies before each.  A request that gives
// back as many pages as it needs is; of the others, in order, those up to
// which the needs (less what they give back) do not pass what is free and
// what the former leave over.
__global__ void __launch_bounds__(ST) settle_kernel(const ReorderParams p)
{
    __shared__ Scan<2> scan2;
    __shared__ Scan<1> scan1;
    const long long count0 = min(max(*p.free_count, 0), p.num_pages);
    long long left = count0;   // free, with what requests leave over
    auto freed_of = [&](int r) {
        long long n = 0;
        for (int i = 0; i < p.tiles; ++i)
            n += p.freed[(long long)r * p.tiles + i];
        return n;
    };
    for (int r0 = 0; r0 < p.R; r0 += ST) {
        const int r = r0 + (int)threadIdx.x;
        long long x[1] = {r < p.R ? max(0LL, freed_of(r) - p.needed[r]) : 0}, all[1];
        scan1.run(x, all);
        left += all[0];
    }
    long long wanted = 0, back = 0, taken = 0;
    for (int r0 = 0; r0 < p.R; r0 += ST) {
        const int r = r0 + (int)threadIdx.x;
        const long long f = r < p.R ? freed_of(r) : 0, c = r < p.R ? p.needed[r] : 0;
        long long x[1] = {max(0LL, c - f)}, all[1];
        scan1.run(x, all);
        const bool given = r < p.R && (c <= f || wanted + x[0] <= left);
        wanted += all[0];
        long long y[2] = {given ? f : 0, given ? c : 0}, sums[2];
        scan2.run(y, sums);
        if (r < p.R) {
            p.needed_before[r] = given ? (int)(taken + y[1] - c) : -1;
            if (p.granted)
                p.granted[r] = given;
            long long before = back + y[0] - f;
            for (int i = 0; i < p.tiles && given; ++i) {
                p.freed_before[(long long)r * p.tiles + i] = before;
                before += p.freed[(long long)r * p.tiles + i];
            }
        }
        back += sums[0];
        taken += sums[1];
    }
    if (threadIdx.x == 0) {
        // (pages given back twice could pass the stack's end)
        const long long raised = count0 + back, top = min(raised, (long long)p.num_pages);
        p.header->raised = raised;
        p.header->top = (int)top;
        p.header->taken = (int)min(taken, top);
        if (raised > top)
            atomicOr(p.status, STATUS_BAD_PAGE);
    }
}

// Phase 3: what comes back onto the stack; the tables' entries to their
// beams' children.
__global__ void __launch_bounds__(RT) apply_kernel(const ReorderParams p)
{
    __shared__ Beams b;
    __shared__ Tile t;
    __shared__ int warps[RW];
    const int r = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles, tid = threadIdx.x;
    if (p.needed_before[r] < 0)
        return;
    load_beams(p, r, b, false);
    const int j = tile * RT + tid;
    load_tile(p, r, j, b, t);
    bool bad = false;
    unsigned gone = released(p, j, b, t, bad);
    if (p.freed[blockIdx.x] > 0) {
        int before = __popc(gone);
        const int lane = tid & 31, warp = tid >> 5;
        const int own = before;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL_MASK, before, o);
            if (lane >= o)
                before += y;
        }
        if (lane == 31)
            warps[warp] = before;
        __syncthreads();
        for (int i = 0; i < warp; ++i)
            before += warps[i];
        long long at = p.header->raised - 1 - (p.freed_before[blockIdx.x] + before - own);
        for (; gone; gone &= gone - 1, --at)
            if (at >= 0 && at < p.num_pages)
                p.free_pages[at] = t.e[__ffs(gone) - 1][tid];
    }
    for (int w = 0; w < p.W; ++w) {
        const int q = b.parent[w];
        if (q < 0 || q == w || j >= b.pages[q])
            continue;
        if (j >= b.pages[w] || t.e[w][tid] != t.e[q][tid])
            p.table[(long long)(r * p.W + w) * p.max_pages + j] = t.e[q][tid];
    }
}

// Phase 4: pages for the copies, and the lengths.
__global__ void __launch_bounds__(RT) take_kernel(const ReorderParams p)
{
    const int lane = threadIdx.x & 31;
    const int top = p.header->top;
    for (long long r = blockIdx.x * RW + (threadIdx.x >> 5); r < p.R; r += (long long)gridDim.x * RW) {
        const long long row = r * p.W + lane;
        const bool in = lane < p.W;
        const int before = p.needed_before[r];
        int32_t *c = p.copies + row * 3;
        if (before < 0) {
            if (in) {
                c[0] = c[1] = -1;
                c[2] = 0;
            }
            continue;
        }
        const long long cap = (long long)p.max_pages * p.page_size;
        const int old = in ? (int)min(max((long long)p.seqlens[row], 0LL), cap) : 0;
        const int parent = in ? p.parents[row] : -1;
        const bool some = parent >= 0 && parent < p.W;
        const int len = __shfl_sync(FULL_MASK, old, some ? parent : 0);
        const bool copy = in && c[0] >= 0;
        const unsigned who = __ballot_sync(FULL_MASK, copy);
        if (copy) {
            const int at = top - 1 - (before + __popc(who & ((1u << lane) - 1)));
            const int page = at >= 0 ? p.free_pages[at] : -1;
            const bool ok = is_page(p, page);
            if (!ok) {
                atomicOr(p.status, STATUS_BAD_PAGE);
                c[0] = -1;
                c[2] = 0;
            }
            c[1] = ok ? page : -1;
            p.table[row * p.max_pages + len / p.page_size] = ok ? page : -1;
        }
        if (in)
            p.seqlens[row] = some ? len : 0;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *p.free_count = top - p.header->taken;
}

// Rows of a page to another one's, of every head: a CTA a copy and head of K
// or V.  The rows lie one behind the other.
__global__ void __launch_bounds__(256) copy_kernel(const CopyParams p)
{
    const int32_t *c = p.copies + (long long)blockIdx.x * 3;
    const int from = c[0], to = c[1], rows = min(c[2], p.page_size);
    if (from < 0 || rows <= 0)
        return;
    if (from >= p.num_pages || to < 0 || to >= p.num_pages) {
        if (threadIdx.x == 0)
            atomicOr(p.status, STATUS_BAD_PAGE);
        return;
    }
    const long long vecs = (long long)rows * p.row_vecs;
    const long long head = (long long)p.page_size * p.row_vecs;
    for (unsigned y = blockIdx.y; y < 2u * p.H; y += gridDim.y) {
        const bool isv = y >= (unsigned)p.H;
        uint4 *pages = static_cast<uint4 *>(isv ? p.v_pages : p.k_pages);
        const int h = (int)(isv ? y - p.H : y);
        const uint4 *src = pages + (from * (long long)p.H + h) * head;
        uint4 *dst = pages + (to * (long long)p.H + h) * head;
        for (long long i = threadIdx.x; i < vecs; i += 256)
            dst[i] = src[i];
    }
}

}  // namespace

cudaError_t launch_reorder(const ReorderParams &p, cudaStream_t s)
{
    const unsigned tiles = (unsigned)p.R * p.tiles;
    count_kernel<<<tiles, RT, 0, s>>>(p);
    settle_kernel<<<1, ST, 0, s>>>(p);
    apply_kernel<<<tiles, RT, 0, s>>>(p);
    take_kernel<<<(unsigned)min((p.R + RW - 1) / RW, 1024), RT, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_copy_pages(const CopyParams &p, cudaStream_t s)
{
    copy_kernel<<<dim3(p.n, (unsigned)min(2LL * p.H, 65535LL)), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace fd
