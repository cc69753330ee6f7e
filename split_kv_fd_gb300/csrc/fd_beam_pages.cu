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
// Two kernels, a CTA a tile of a request's tables in each: what comes back, what
// is needed and which places change; then, with the sums of these, the stack,
// the tables and the lengths.  The data is small, and what takes the time is the
// chain of dependent loads.
#include "fd_beam.h"
#include "fd_device.cuh"
#include "fd_pages.h"

namespace fd {
namespace {

constexpr int RT = REORDER_TILE;   // threads of a CTA, one a place
constexpr int RW = RT / 32;
constexpr int ST = 1024;           // threads of the sums' own kernel
static_assert(REORDER_SCAN == 4 * RT, "four numbers a thread");

__device__ __forceinline__ bool is_page(const ReorderParams &p, int page) { return page >= 0 && page < p.num_pages; }

__device__ __forceinline__ int pages_of(const ReorderParams &p, int len)
{
    return (int)(((long long)len + p.page_size - 1) / p.page_size);
}

// What comes back of a place: bit w where beam w is the first to name a page
// that no parent's table has there.
struct Beams {
    int len[BEAM_MAX_W], pages[BEAM_MAX_W], parent[BEAM_MAX_W];   // parent: -1 for none
    unsigned parents;   // those that are a parent
};

__global__ void __launch_bounds__(RT) look_kernel(const ReorderParams p)
{
    __shared__ Beams b;
    __shared__ int e[BEAM_MAX_W][RT + 1];
    __shared__ int warps[RW];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int r = blockIdx.x / p.tiles, tile = blockIdx.x - r * p.tiles;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = p.W;
    const int row0 = r * W, j = tile * RT + tid;

    // Lengths and parents, while the entries of the place are on their way
    // (those behind a length are read and not looked at).
    int mine[8];
    auto fetch = [&](int w0) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            mine[k] = w0 + k < W && j < p.max_pages ? p.table[(long long)(row0 + w0 + k) * p.max_pages + j] : 0;
    };
    fetch(0);
    if (warp == 0) {
        int parent = -1;
        if (lane < W) {
            const long long cap = (long long)p.max_pages * p.page_size;
            const int len = (int)min(max((long long)p.seqlens[row0 + lane], 0LL), cap);
            parent = max(p.parents[row0 + lane], -1);
            if (parent >= W) {
                parent = -1;
                if (tile == 0)
                    atomicOr(p.status, STATUS_BAD_INDEX);
            }
            b.len[lane] = len;
            b.pages[lane] = pages_of(p, len);
            b.parent[lane] = parent;
            if (tile == 0)
                p.lens[row0 + lane] = len;
        }
        const unsigned all = __reduce_or_sync(FULL_MASK, parent >= 0 ? 1u << parent : 0u);
        if (lane == 0)
            b.parents = all;
        if (blockIdx.x == 0 && lane == 0)
            p.header->count = min(max(*p.free_count, 0), p.num_pages);
    }
    for (int w0 = 0; w0 < W; w0 += 8) {
        if (w0)
            fetch(w0);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (w0 + k < W)
                e[w0 + k][tid] = mine[k];
    }
    __syncthreads();

    // Most places are of a part that all beams share: one page, named by all.
    unsigned have = 0;
    int first = 0;
    bool same = true, shorter = false;
    for (int w = 0; w < W; ++w) {
        if (j < b.pages[w]) {
            first = have ? first : e[w][tid];
            same &= e[w][tid] == first;
            have |= 1u << w;
        } else if (b.parent[w] >= 0) {
            shorter |= j < b.pages[b.parent[w]];
        }
    }
    bool bad = false;
    unsigned gone = 0;
    if (same && have && !(have & b.parents)) {
        bad = !is_page(p, first);
        gone = bad ? 0 : have & (0u - have);
    }
    // The others a warp at a time, a beam a lane.
    for (unsigned left = __ballot_sync(FULL_MASK, !same); left; left &= left - 1) {
        const int c = __ffs(left) - 1, jc = tile * RT + warp * 32 + c;
        const bool in = lane < W && jc < b.pages[lane];
        const int page = lane < W ? e[lane][warp * 32 + c] : 0;
        const unsigned who = __ballot_sync(FULL_MASK, in);
        bool mine = false;
        if (in) {
            const unsigned peers = __match_any_sync(who, page);
            mine = !(peers & b.parents) && lane == __ffs(peers) - 1;
            if (mine && !is_page(p, page)) {
                mine = false;
                bad = true;
            }
        }
        const unsigned g = __ballot_sync(FULL_MASK, mine);
        if (lane == c)
            gone = g;
    }
    if (bad)
        atomicOr(p.status, STATUS_BAD_PAGE);
    const unsigned changes = __ballot_sync(FULL_MASK, have && (!same || shorter));
    if (lane == 0)
        p.moved[(long long)blockIdx.x * RW + warp] = changes;

    // what comes back, in order of place and beam
    const int own = __popc(gone);
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL_MASK, sum, o);
        if (lane >= o)
            sum += y;
    }
    if (lane == 31)
        warps[warp] = sum;
    __syncthreads();
    int before = sum - own, all = 0;
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        before += i < warp ? warps[i] : 0;
        all += warps[i];
    }
    if (tid == 0)
        p.freed[blockIdx.x] = all;
    int32_t *to = p.pages + (long long)blockIdx.x * W * RT + before;
    for (; gone; gone &= gone - 1)
        *to++ = e[__ffs(gone) - 1][tid];

    // The copies, by the last warp (whose places are the rarest to be used).
    // New beam w: its parent's last page, if that is partly filled.
    if (tile == 0 && warp == RW - 1) {
        const int w = lane;
        const int parent = w < W ? b.parent[w] : -1;
        const int rows = parent >= 0 ? b.len[parent] % p.page_size : 0;
        const int at = rows ? b.len[parent] / p.page_size : 0;
        const int page = rows ? p.table[(long long)(row0 + parent) * p.max_pages + at] : -1;
        bool copy = false;
#pragma unroll 8
        for (int v = 0; v < W; ++v) {
            const int q = b.parent[v];
            // named by a beam before it, or as a full page by any
            if (rows && v != w && q >= 0 && at < b.pages[q] && (v < w || b.len[q] / p.page_size > at))
                copy |= p.table[(long long)(row0 + q) * p.max_pages + at] == page;
        }
        if (rows && !is_page(p, page)) {
            copy = false;
            atomicOr(p.status, STATUS_BAD_PAGE);
        }
        if (w < W) {
            int32_t *c = p.copies + (long long)(row0 + w) * 3;
            c[0] = copy ? page : -1;
            c[1] = -1;
            c[2] = copy ? rows : 0;
        }
        const unsigned who = __ballot_sync(FULL_MASK, copy);
        if (lane == 0)
            p.copied[r] = who;
    }
}

// Inclusive sums over the block of NT threads, and their total.
template <int NT> struct Scan {
    long long warp[NT / 32];
    __device__ __forceinline__ long long run(long long x, long long &total)
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
            warp[w] = x;
        __syncthreads();
        long long all = 0;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
            x += i < w ? warp[i] : 0;
            all += warp[i];
        }
        total = all;
        return x;
    }
};

// The stack's header from the totals.
__device__ __forceinline__ ReorderHeader heights(const ReorderParams &p, int count, long long back, long long taken)
{
    ReorderHeader h;
    // (pages given back twice could pass the stack's end)
    const long long raised = count + back, top = min(raised, (long long)p.num_pages);
    h.count = count;
    h.top = (int)top;
    h.taken = (int)min(taken, top);
    h.back = back;
    return h;
}

// Who is granted, and what lies before each, for many tiles.  A request that
// gives back as many pages as it needs is; of the others, in order, those up
// to which the needs (less what they give back) do not pass what is free and
// what the former leave over.
__global__ void __launch_bounds__(ST) settle_kernel(const ReorderParams p)
{
    __shared__ Scan<ST> scan;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int count = p.header->count;
    auto freed_of = [&](int r) {
        long long n = 0;
        for (int i = 0; i < p.tiles; ++i)
            n += p.freed[(long long)r * p.tiles + i];
        return n;
    };
    long long left = count, all;   // free, with what requests leave over
    for (int r0 = 0; r0 < p.R; r0 += ST) {
        const int r = r0 + (int)threadIdx.x;
        scan.run(r < p.R ? max(0LL, freed_of(r) - __popc(p.copied[r])) : 0, all);
        left += all;
    }
    long long wanted = 0, back = 0, taken = 0;
    for (int r0 = 0; r0 < p.R; r0 += ST) {
        const int r = r0 + (int)threadIdx.x;
        const long long f = r < p.R ? freed_of(r) : 0, c = r < p.R ? __popc(p.copied[r]) : 0;
        const long long x = scan.run(max(0LL, c - f), all);
        const bool given = r < p.R && (c <= f || wanted + x <= left);
        wanted += all;
        long long allf, allc;
        const long long sf = scan.run(given ? f : 0, allf), sc = scan.run(given ? c : 0, allc);
        if (r < p.R) {
            p.needed_before[r] = given ? (int)(taken + sc - c) : -1;
            long long before = back + sf - f;
            for (int i = 0; i < p.tiles; ++i) {
                p.freed_before[(long long)r * p.tiles + i] = before;
                before += given ? p.freed[(long long)r * p.tiles + i] : 0;
            }
        }
        back += allf;
        taken += allc;
    }
    if (threadIdx.x == 0)
        *p.header = heights(p, count, back, taken);
}

// The stack, the tables and the lengths.
template <bool SETTLED> __global__ void __launch_bounds__(RT) move_kernel(const ReorderParams p)
{
    __shared__ int e[BEAM_MAX_W][RT + 1];
    __shared__ int pages[BEAM_MAX_W], parent[BEAM_MAX_W], place[BEAM_MAX_W], taken_page[BEAM_MAX_W];
    __shared__ int freed_before[SETTLED ? 1 : REORDER_SCAN], needed_before[SETTLED ? 1 : REORDER_SCAN];
    __shared__ Scan<RT> scan;
    const int r = blockIdx.x / p.tiles, tile = blockIdx.x - r * p.tiles;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = p.W;
    const int row0 = r * W, j = tile * RT + tid, items = p.R * p.tiles;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int nfreed = p.freed[blockIdx.x];
    const bool moves = p.moved[(long long)blockIdx.x * RW + warp] >> lane & 1;
    ReorderHeader h;
    int need0;          // copies of granted requests before this one, -1 if it is refused
    long long free0;    // pages that come back before this tile's
    if (SETTLED) {
        h = *p.header;
        need0 = p.needed_before[r];
        free0 = p.freed_before[blockIdx.x];
    } else {
        // the sums over all tiles and requests, four a thread
        h.count = p.header->count;
        int f[4], c[4];
        long long total, sum = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = tid * 4 + k < items ? p.freed[tid * 4 + k] : 0;
            c[k] = tid * 4 + k < p.R ? __popc(p.copied[tid * 4 + k]) : 0;
        }
        auto before = [&](const int (&x)[4], int *to) {   // exclusive sums of x, and all of it
            const int s = x[0] + x[1] + x[2] + x[3];
            long long all;
            int at = (int)scan.run(s, all) - s;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                to[tid * 4 + k] = at;
                at += x[k];
            }
            return all;
        };
        const long long back0 = before(f, freed_before);
        __syncthreads();
        // what a request needs beyond what it gives back, and what it leaves
        long long lacks[4], leaves = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int q = tid * 4 + k;
            const int end = (q + 1) * p.tiles;
            const int own = q < p.R ? (end < items ? freed_before[end] : (int)back0) - freed_before[q * p.tiles] : 0;
            lacks[k] = max(0, c[k] - own);
            leaves += max(0, own - c[k]);
            sum += lacks[k];
        }
        long long left, lack;
        scan.run(leaves, left);
        left += h.count;
        long long at = scan.run(sum, lack) - sum;
        if (lack <= left) {   // all are granted
            need0 = 0;
            total = back0;
        } else {
            unsigned given = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                at += lacks[k];
                given |= (lacks[k] == 0 || at <= left) << k;
                c[k] = given >> k & 1 ? c[k] : 0;
            }
            __shared__ bool refused[REORDER_SCAN];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                refused[tid * 4 + k] = !(given >> k & 1);
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 4; ++k)
                f[k] = tid * 4 + k < items && refused[(tid * 4 + k) / p.tiles] ? 0 : f[k];
            total = before(f, freed_before);
            need0 = refused[r] ? -1 : 0;
        }
        const long long taken = before(c, needed_before);
        __syncthreads();
        h = heights(p, h.count, total, taken);
        need0 = need0 < 0 ? -1 : needed_before[r];
        free0 = freed_before[blockIdx.x];
    }
    if (blockIdx.x == 0 && tid == 0) {
        *p.free_count = h.top - h.taken;
        if (h.count + h.back > h.top)
            atomicOr(p.status, STATUS_BAD_PAGE);
    }
    if (tile == 0 && tid == 0 && p.granted)
        p.granted[r] = need0 >= 0;
    if (need0 < 0) {
        if (tile == 0 && tid < W) {
            int32_t *c = p.copies + (long long)(row0 + tid) * 3;
            c[0] = -1;
            c[2] = 0;
        }
        return;
    }

    // what comes back onto the stack, the first on top
    const int32_t *list = p.pages + (long long)blockIdx.x * W * RT;
    const long long raised = h.count + h.back;
    for (int i = tid; i < nfreed; i += RT) {
        const long long at = raised - 1 - (free0 + i);
        if (at >= 0 && at < p.num_pages)
            p.free_pages[at] = list[i];
    }

    // Lengths, and the pages for this request's copies: of those that came
    // back the t-th, or one that was free before.
    if (warp == 0) {
        const int q = lane < W ? p.parents[row0 + lane] : -1;
        const bool some = q >= 0 && q < W;
        const int old = lane < W ? p.lens[row0 + lane] : 0;
        const int len = __shfl_sync(FULL_MASK, old, some ? q : 0);
        const unsigned who = p.copied[r];
        const bool copy = who >> lane & 1;
        int page = -1;
        const int last = copy ? len / p.page_size : -1;
        if (copy && last / RT == tile) {
            const int t = need0 + __popc(who & ((1u << lane) - 1));
            const int at = h.top - 1 - t;
            if (at >= h.count) {
                const long long x = raised - 1 - at;   // the x-th that came back: of the last tile with no more before it
                int lo = 0, hi = items - 1;
                while (lo < hi) {
                    const int mid = (int)(((long long)lo + hi + 1) >> 1);
                    if ((SETTLED ? p.freed_before[mid] : (long long)freed_before[SETTLED ? 0 : mid]) <= x)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
                page = p.pages[(long long)lo * W * RT + (x - (SETTLED ? p.freed_before[lo] : (long long)freed_before[SETTLED ? 0 : lo]))];
            } else if (at >= 0) {
                page = p.free_pages[at];
            }
            int32_t *c = p.copies + (long long)(row0 + lane) * 3;
            if (!is_page(p, page)) {
                page = -1;
                atomicOr(p.status, STATUS_BAD_PAGE);
                c[0] = -1;
                c[2] = 0;
            }
            c[1] = page;
        }
        if (lane < W) {
            pages[lane] = pages_of(p, old);
            parent[lane] = some ? q : -1;
            place[lane] = last;
            taken_page[lane] = page;
            if (tile == 0)
                p.seqlens[row0 + lane] = some ? len : 0;
        }
    }
    __syncthreads();
    if (moves) {
#pragma unroll 8
        for (int w = 0; w < W; ++w)
            if (j < pages[w])
                e[w][tid] = p.table[(long long)(row0 + w) * p.max_pages + j];
        for (int w = 0; w < W; ++w) {
            const int q = parent[w];
            if (q >= 0 && q != w && j < pages[q] && j != place[w] && !(j < pages[w] && e[w][tid] == e[q][tid]))
                p.table[(long long)(row0 + w) * p.max_pages + j] = e[q][tid];
        }
    }
    // (a beam may keep its parent's table, itself, and still need a copy: no other thread writes there)
    __syncthreads();
    if (tid < W && place[tid] >= 0 && place[tid] / RT == tile)
        p.table[(long long)(row0 + tid) * p.max_pages + place[tid]] = taken_page[tid];
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

namespace {

// A launch whose CTAs may start while the kernel before it ends.
template <typename P> cudaError_t launch_behind(void (*kernel)(P), dim3 grid, int threads, cudaStream_t s, const P &p)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_reorder(const ReorderParams &p, cudaStream_t s)
{
    const unsigned items = (unsigned)p.R * p.tiles;
    look_kernel<<<items, RT, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    if (items <= REORDER_SCAN)
        return launch_behind(move_kernel<false>, items, RT, s, p);
    e = launch_behind(settle_kernel, 1, ST, s, p);
    return e == cudaSuccess ? launch_behind(move_kernel<true>, items, RT, s, p) : e;
}

cudaError_t launch_copy_pages(const CopyParams &p, cudaStream_t s)
{
    copy_kernel<<<dim3(p.n, (unsigned)min(2LL * p.H, 65535LL)), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace fd
