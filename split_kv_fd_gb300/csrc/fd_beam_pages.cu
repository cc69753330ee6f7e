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
// chain of dependent loads: 32 requests of 8 beams over 1K-32K tokens 9 us, 24
// of 16 11, and the copies of the former (8 MB) 6 us behind them.
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

// A request's beams before the step.
struct Beams {
    int len[BEAM_MAX_W], pages[BEAM_MAX_W], parent[BEAM_MAX_W];   // parent: -1 for none
    int wants[BEAM_MAX_W];   // pages of the parent's
    unsigned parents;        // those that are a parent
};

// (Loops over beams go in steps of BATCH with nothing to wait for within a
// step: rolled ones cost a latency a beam.)
constexpr int BATCH = 8;

// What comes back of a tile's places (`gone`: the beams that are the first to
// name a page that no parent's table has there), the places whose entries
// change, and, of a request's first tile, the copies it needs.
__global__ void __launch_bounds__(RT) look_kernel(const ReorderParams p)
{
    __shared__ Beams b;
    __shared__ int e[BEAM_MAX_W][RT + 1];
    __shared__ int warps[RW], list[RT];
    __shared__ unsigned back[RT];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int r = blockIdx.x / p.tiles, tile = blockIdx.x - r * p.tiles;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = p.W;
    const int row0 = r * W, j = tile * RT + tid;

    // Lengths and parents, while the entries of the place are on their way
    // (those behind a length are read and not looked at).
    int mine[2 * BATCH];
    auto fetch = [&](int w0) {
#pragma unroll
        for (int k = 0; k < 2 * BATCH; ++k)
            mine[k] = w0 + k < W && j < p.max_pages ? p.table[(long long)(row0 + w0 + k) * p.max_pages + j] : 0;
    };
    fetch(0);
    if (warp == 0) {
        int parent = -1, len = 0;
        if (lane < W) {
            const long long cap = (long long)p.max_pages * p.page_size;
            len = (int)min(max((long long)p.seqlens[row0 + lane], 0LL), cap);
            parent = max(p.parents[row0 + lane], -1);
            if (parent >= W) {
                parent = -1;
                if (tile == 0)
                    atomicOr(p.status, STATUS_BAD_INDEX);
            }
            if (tile == 0)
                p.lens[row0 + lane] = len;
        }
        const int pages = pages_of(p, len), theirs = __shfl_sync(FULL_MASK, pages, max(parent, 0));
        b.len[lane] = len;
        b.pages[lane] = pages;
        b.parent[lane] = parent;
        b.wants[lane] = parent >= 0 ? theirs : 0;
        const unsigned all = __reduce_or_sync(FULL_MASK, parent >= 0 ? 1u << parent : 0u);
        if (lane == 0)
            b.parents = all;
        if (blockIdx.x == 0 && lane == 0)
            p.header->count = min(max(*p.free_count, 0), p.num_pages);
    }
    for (int w0 = 0; w0 < W; w0 += 2 * BATCH) {
        if (w0)
            fetch(w0);
#pragma unroll
        for (int k = 0; k < 2 * BATCH; ++k)
            e[w0 + k][tid] = mine[k];
    }
    __syncthreads();

    // Most places are of a part that all beams share: one page, named by all.
    unsigned have = 0, wants = 0;
    int first = 0;
    for (int w0 = 0; w0 < W; w0 += BATCH) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int w = w0 + k;
            have |= (j < b.pages[w]) << w;
            wants |= (j < b.wants[w]) << w;
        }
    }
    if (have)
        first = e[__ffs(have) - 1][tid];
    bool same = true;
    for (int w0 = 0; w0 < W; w0 += BATCH) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            same &= !(have >> (w0 + k) & 1) || e[w0 + k][tid] == first;
    }
    bool bad = false;
    unsigned gone = 0;
    if (same && have && !(have & b.parents)) {
        bad = !is_page(p, first);
        gone = bad ? 0 : have & (0u - have);
    }
    // The others by all warps alike, a beam a lane, as many places at a time as
    // a warp has lanes for.
    const unsigned odd = __ballot_sync(FULL_MASK, !same);
    if (lane == 0)
        warps[warp] = __popc(odd);
    __syncthreads();
    int at = 0, odds = 0;
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        at += i < warp ? warps[i] : 0;
        odds += warps[i];
    }
    if (!same)
        list[at + __popc(odd & ((1u << lane) - 1))] = tid;
    __syncthreads();
    int width = 1;   // lanes of a place
    while (width < W)
        width *= 2;
    const int group = lane / width, w = lane & (width - 1), each = 32 / width;
    const unsigned in_group = width == 32 ? FULL_MASK : ((1u << width) - 1) << group * width;
    for (int i = warp * each; i < odds; i += RW * each) {
        const int c = i + group < odds ? list[i + group] : -1;
        const bool in = c >= 0 && w < W && tile * RT + c < b.pages[w];
        const int page = in ? e[w][c] : 0;
        const unsigned who = __ballot_sync(FULL_MASK, in) & in_group;
        bool mine = false;
        if (in) {
            const unsigned peers = __match_any_sync(who, page);
            mine = !(peers >> group * width & b.parents) && lane == __ffs(peers) - 1;
            if (mine && !is_page(p, page)) {
                mine = false;
                bad = true;
            }
        }
        const unsigned g = (__ballot_sync(FULL_MASK, mine) & in_group) >> group * width;
        if (c >= 0 && w == 0)
            back[c] = g;
    }
    __syncthreads();
    if (!same)
        gone = back[tid];
    if (bad)
        atomicOr(p.status, STATUS_BAD_PAGE);
    const unsigned changes = __ballot_sync(FULL_MASK, have && (!same || (wants & ~have)));
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
        const int w = lane, parent = b.parent[w], len = parent >= 0 ? b.len[parent] : 0;
        const int rows = len % p.page_size, at = len / p.page_size;
        const int page = rows ? p.table[(long long)(row0 + parent) * p.max_pages + at] : -1;
        // named as its last page by a beam before it
        const unsigned part = __ballot_sync(FULL_MASK, rows != 0);
        bool copy = false;
        if (rows)
            copy = __match_any_sync(part, (unsigned long long)(unsigned)at << 32 | (unsigned)page) & ((1u << w) - 1);
        // or as a full page by any (of another length)
        const int longest = __reduce_max_sync(FULL_MASK, at);
        if (__any_sync(FULL_MASK, rows && at < longest)) {
            for (int v = 0; v < W; ++v) {
                const int q = b.parent[v];
                if (rows && q >= 0 && b.len[q] / p.page_size > at)
                    copy |= p.table[(long long)(row0 + q) * p.max_pages + at] == page;
            }
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
    const int q = lane < W ? p.parents[row0 + lane] : -1;   // (older than the kernel before)
    const bool some = q >= 0 && q < W;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // Everything that is read without the sums, on its way at once.
    const int nfreed = p.freed[blockIdx.x];
    const unsigned changes = p.moved[(long long)blockIdx.x * RW + warp], who = p.copied[r];
    const int old = lane < W ? p.lens[row0 + lane] : 0, count = p.header->count;
    int f[4], c[4];   // of four tiles and requests a thread
    if (!SETTLED) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = tid * 4 + k < items ? p.freed[tid * 4 + k] : 0;
            c[k] = tid * 4 + k < p.R ? __popc(p.copied[tid * 4 + k]) : 0;
        }
    }
    const bool moves = changes >> lane & 1;
    int mine[BATCH];
    auto fetch = [&](int w0) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            mine[k] = w0 + k < W ? p.table[(long long)(row0 + w0 + k) * p.max_pages + j] : 0;
    };
    if (moves)
        fetch(0);
    const int len = __shfl_sync(FULL_MASK, old, some ? q : 0);
    const int last = who >> lane & 1 ? len / p.page_size : -1;   // the place of a copy
    if (warp == 0) {
        pages[lane] = pages_of(p, old);
        parent[lane] = some ? q : -1;
        place[lane] = last;
    }

    ReorderHeader h;
    int need0;          // copies of granted requests before this one, -1 if it is refused
    long long free0;    // pages that come back before this tile's
    if (SETTLED) {
        h = *p.header;
        need0 = p.needed_before[r];
        free0 = p.freed_before[blockIdx.x];
    } else {
        // The sums over all tiles and requests, four a thread: of what comes
        // back in the lower half of a word, of what is needed in the upper.
        long long both;
        auto sums = [&] {
            const long long s = (long long)(c[0] + c[1] + c[2] + c[3]) << 32 | (unsigned)(f[0] + f[1] + f[2] + f[3]);
            const long long at = scan.run(s, both) - s;
            int fb = (int)at, cb = (int)(at >> 32);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                freed_before[tid * 4 + k] = fb;
                needed_before[tid * 4 + k] = cb;
                fb += f[k];
                cb += c[k];
            }
            __syncthreads();
        };
        sums();
        // what a request needs beyond what it gives back, and what it leaves
        int lacks[4];
        long long own2 = 0, all2;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = tid * 4 + k, end = (i + 1) * p.tiles;
            const int own = i < p.R ? (end < items ? freed_before[end] : (int)both) - freed_before[i * p.tiles] : 0;
            lacks[k] = max(0, c[k] - own);
            own2 += (long long)lacks[k] << 32 | (unsigned)max(0, own - c[k]);
        }
        long long at = (scan.run(own2, all2) >> 32) - (own2 >> 32);
        const long long left = (int)all2 + (long long)count;
        need0 = 0;
        if ((all2 >> 32) > left) {   // not all are granted: the sums of those that are
            __shared__ bool refused[REORDER_SCAN];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                at += lacks[k];
                refused[tid * 4 + k] = lacks[k] != 0 && at > left;
                c[k] = refused[tid * 4 + k] ? 0 : c[k];
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 4; ++k)
                f[k] = tid * 4 + k < items && refused[(tid * 4 + k) / p.tiles] ? 0 : f[k];
            sums();
            need0 = refused[r] ? -1 : 0;
        }
        h = heights(p, count, (int)both, both >> 32);
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

    // The pages for this request's copies: of those that came back the t-th,
    // or one that was free before.
    const long long raised = h.count + h.back;
    if (warp == 0) {
        int page = -1;
        if (last >= 0 && last / RT == tile) {
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
            taken_page[lane] = page;
            if (tile == 0)
                p.seqlens[row0 + lane] = some ? len : 0;
        }
    }
    // what comes back onto the stack, the first on top
    const int32_t *list = p.pages + (long long)blockIdx.x * W * RT;
    for (int i = tid; i < nfreed; i += RT) {
        const long long at = raised - 1 - (free0 + i);
        if (at >= 0 && at < p.num_pages)
            p.free_pages[at] = list[i];
    }
    if (moves) {
        for (int w0 = 0; w0 < W; w0 += BATCH) {
            if (w0)
                fetch(w0);
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                e[w0 + k][tid] = mine[k];
        }
    }
    __syncthreads();
    if (moves) {
        for (int w0 = 0; w0 < W; w0 += BATCH) {
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int w = w0 + k, from = parent[w];
                const int entry = e[max(from, 0)][tid];
                if (from >= 0 && from != w && j < pages[from] && j != place[w] && !(j < pages[w] && e[w][tid] == entry))
                    p.table[(long long)(row0 + w) * p.max_pages + j] = entry;
            }
        }
    }
    // (no other thread writes to a copy's place)
    if (tid < W && place[tid] >= 0 && place[tid] / RT == tile)
        p.table[(long long)(row0 + tid) * p.max_pages + place[tid]] = taken_page[tid];
}

// Rows of a page to another one's, of every head of K and V: the filled rows of
// a head lie one behind the other, and a CTA takes a slice of all of them,
// COPY_DEEP vectors a thread on their way at once.
constexpr int COPY_THREADS = 256, COPY_DEEP = 8;

__global__ void __launch_bounds__(COPY_THREADS) copy_kernel(const CopyParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t *c = p.copies + (long long)blockIdx.x * 3;
    const int from = c[0], to = c[1], rows = min(c[2], p.page_size);
    if (from < 0 || rows <= 0)
        return;
    if (from >= p.num_pages || to < 0 || to >= p.num_pages) {
        if (threadIdx.x == 0 && blockIdx.y == 0)
            atomicOr(p.status, STATUS_BAD_PAGE);
        return;
    }
    const unsigned head = (unsigned)rows * p.row_vecs;   // filled vectors of a head
    const unsigned all = 2u * p.H * head;                // (below 2^31)
    const unsigned inverse = 0xffffffffu / head + 1;     // i / head by a product: one too many at most (head >= 4)
    const long long pitch = (long long)p.page_size * p.row_vecs, src = from * (long long)p.H, dst = to * (long long)p.H;
    for (unsigned i0 = blockIdx.y * COPY_THREADS * COPY_DEEP; i0 < all; i0 += gridDim.y * COPY_THREADS * COPY_DEEP) {
        uint4 x[COPY_DEEP];
        uint4 *at[COPY_DEEP];
#pragma unroll
        for (int k = 0; k < COPY_DEEP; ++k) {
            const unsigned i = i0 + k * COPY_THREADS + threadIdx.x;
            at[k] = nullptr;
            if (i < all) {
                unsigned y = __umulhi(i, inverse), v = i - y * head;
                if (v >= head) {
                    --y;
                    v += head;
                }
                const bool isv = y >= (unsigned)p.H;
                const unsigned h = isv ? y - p.H : y;
                uint4 *pages = static_cast<uint4 *>(isv ? p.v_pages : p.k_pages);
                x[k] = pages[(src + h) * pitch + v];
                at[k] = pages + (dst + h) * pitch + v;
            }
        }
#pragma unroll
        for (int k = 0; k < COPY_DEEP; ++k)
            if (at[k])
                *at[k] = x[k];
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
    const long long most = 2LL * p.H * p.page_size * p.row_vecs, slice = COPY_THREADS * COPY_DEEP;
    return launch_behind(copy_kernel, dim3(p.n, (unsigned)min((most + slice - 1) / slice, 65535LL)), COPY_THREADS, s, p);
}

}  // namespace fd
