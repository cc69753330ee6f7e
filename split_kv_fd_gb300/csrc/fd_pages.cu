// fd_pages.cu -- page bookkeeping of a paged KV cache on the GPU: every
// sequence to its target length, its pages taken from and given back to a
// stack of free pages, and the slots and positions of the tokens it grew by.
//
// With pages(n) = ceil(n / page_size), sequence b releases r_b =
// max(0, pages(old) - pages(new)) pages and needs g_b = max(0, pages(new) -
// pages(old)).  Released pages go on the stack in reverse order of (b,
// logical page), pages are taken in order of (b, logical page) from the top:
// a release undoes the growth before it.  All of it follows from exclusive
// prefix sums over b, so the result does not depend on any order of threads.
//
// The data is a few KB, and what takes the time is a chain of dependent
// steps: lengths, two scans, stack and table.  So one CTA keeps the books with
// up to 1024 sequences' numbers in registers, and only the slots and
// positions, which may be many, are written by the whole cluster behind it.
// 256 sequences one token on and back: 7.1 us each way; 64 with 48 new ones,
// 16K tokens: 7.9.  (The scans are of 1024 threads in 64 bits whatever the
// batch; what fewer and narrower ones would take is not measured.)
#include "fd_device.cuh"
#include "fd_pages.h"

#include <limits.h>

namespace fd {
namespace {

constexpr int RT = 1024;     // threads of a CTA
constexpr int CLUSTER = 8;   // CTAs that write slots and positions
constexpr int RW = RT / 32;

// Inclusive sums of N values over the block, and their totals.
template <int N> struct Scan {
    long long warp[N][RW];
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
        // every warp sums the warps before it, and all of them
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

struct Change {
    int oldn, newn, po, pn;
    bool fits;
};

__device__ __forceinline__ Change change_of(const ResizeParams &p, int b)
{
    Change c;
    const long long cap = (long long)p.max_pages * p.page_size;
    c.oldn = (int)min(max((long long)p.seqlens[b], 0LL), cap);
    c.newn = max(p.target[b], 0);
    c.fits = c.newn <= cap;
    c.po = (int)(((long long)c.oldn + p.page_size - 1) / p.page_size);
    c.pn = (int)(((long long)c.newn + p.page_size - 1) / p.page_size);
    return c;
}

// A page id, or -1 (reported) where it names no page of the pool: nothing
// else may reach the stack, the table or a slot, whose product with
// page_size could lie in another sequence's page.
__device__ __forceinline__ int page_or_none(const ResizeParams &p, int page, unsigned &bad)
{
    if (page >= 0 && page < p.num_pages)
        return page;
    bad |= STATUS_BAD_PAGE;
    return -1;
}

// The pages of a chunk of sequences: thread b's are x[b] .. x[b + 1] - 1 of
// the chunk's (counted from those that are dropped), its first one page
// `page0[b]` of its sequence.
struct Flat {
    int x[RT];
    int page0[RT];
    // the thread whose pages i is among
    __device__ __forceinline__ int owner(int i) const
    {
        int lo = 0, hi = RT - 1;   // the last with x <= i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (x[mid] <= i)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo;
    }
};

__device__ __forceinline__ void keep_books(const ResizeParams &p)
{
    __shared__ Scan<3> scan3;
    __shared__ Scan<2> scan2;
    __shared__ Flat flat;
    const int tid = threadIdx.x;
    const long long count0 = min(max(*p.free_count, 0), p.num_pages);
    unsigned bad = 0;
    const bool once = p.B <= RT;   // one chunk: its changes and sums stay in registers

    // how many pages come back
    long long back = 0;
    Change c = {};
    long long sum[3] = {0, 0, 0}, total[3], own[3] = {0, 0, 0};   // released, needed, new tokens
    auto load = [&](int b0) {
        const int b = b0 + tid;
        c = {};
        own[0] = own[1] = own[2] = 0;
        if (b < p.B) {
            c = change_of(p, b);
            own[0] = max(0, c.po - c.pn);
            if (c.fits) {
                own[1] = max(0, c.pn - c.po);
                own[2] = max(0, c.newn - c.oldn);
            }
        }
#pragma unroll
        for (int i = 0; i < 3; ++i)
            sum[i] = own[i];
        scan3.run(sum, total);
    };
    for (int b0 = 0; b0 < p.B; b0 += RT) {
        load(b0);
        back += total[0];
    }
    // Onto the stack, the last of them first; one that is no page goes there
    // as -1, and is none again for who takes it.  What would pass the stack's
    // end (pages given back twice) is not stored, so that the stack is what
    // lies below `top` in any case.
    const long long raised = count0 + back, top = min(raised, (long long)p.num_pages);
    if (raised > top)
        bad |= STATUS_BAD_PAGE;
    long long done = 0;
    for (int b0 = 0; back > 0 && b0 < p.B; b0 += RT) {
        if (!once)
            load(b0);
        __syncthreads();   // the pages before have been written
        // Lengths that name the same pages many times can pass 2^31 pages, but
        // those behind the dropped ones are num_pages at most, and a thread's
        // own fit an int: only the places of threads that own none of the
        // former are clamped.
        const long long skip = max(0LL, raised - top - done);
        flat.x[tid] = (int)min(max(sum[0] - own[0] - skip, (long long)INT_MIN), (long long)INT_MAX);
        flat.page0[tid] = c.pn;
        __syncthreads();
        const unsigned kept = (unsigned)max(0LL, total[0] - skip);
        for (unsigned u = tid; u < kept; u += RT) {
            const int i = (int)u, o = flat.owner(i), b = b0 + o;
            p.free_pages[raised - 1 - (done + skip + i)] =
                page_or_none(p, p.table[(long long)b * p.max_pages + flat.page0[o] + (i - flat.x[o])], bad);
        }
        done += total[0];
    }
    __syncthreads();   // what is taken below may have come back above

    // growth, in order of b, as far as the pages (and the slots) last
    long long pages = 0, tokens = 0, grown = 0, taken = 0;
    for (int b0 = 0; b0 < p.B; b0 += RT) {
        if (!once)
            load(b0);
        const int b = b0 + tid;
        const bool given = b < p.B && c.fits &&
                           (own[1] == 0 || pages + sum[1] <= top) &&
                           (own[2] == 0 || tokens + sum[2] <= p.max_tokens);
        pages += total[1];
        tokens += total[2];
        const long long mine = given ? own[1] : 0, g = given ? own[2] : 0;
        long long two[2] = {mine, g}, all[2];
        scan2.run(two, all);
        if (b < p.B) {
            p.seqlens[b] = given ? c.newn : c.oldn;
            if (p.cu)
                p.cu[b + 1] = (int)(grown + two[1]);
        }
        if (all[0] > 0) {
            __syncthreads();   // the pages before have been written
            flat.x[tid] = (int)(two[0] - mine);
            flat.page0[tid] = c.po;
            __syncthreads();
            for (unsigned u = tid; u < (unsigned)all[0]; u += RT) {
                const int i = (int)u, o = flat.owner(i);
                const long long at = top - 1 - (taken + i);
                p.table[(long long)(b0 + o) * p.max_pages + flat.page0[o] + (i - flat.x[o])] =
                    page_or_none(p, p.free_pages[at], bad);
            }
        }
        taken += all[0];
        grown += all[1];
    }
    if (tid == 0) {
        if (p.cu)
            p.cu[0] = 0;
        *p.free_count = (int)(top - taken);
    }
    if (bad)
        atomicOr(p.status, bad);
}

// The cluster's first CTA keeps the books; then all of them write a slot and
// a position a thread: the token's sequence by bisection of the offsets,
// its position and its page from what the first CTA wrote.
__global__ void __launch_bounds__(RT, 1) resize_kernel(const ResizeParams p)
{
    if (blockIdx.x == 0)
        keep_books(p);
    if (!p.slots && !p.positions)
        return;
    // the first CTA's writes, to the others
    __threadfence();
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    const int grown = p.cu[p.B];
    unsigned bad = 0;
    // (unsigned: the step behind the last of 2^31 - 1 slots passes an int)
    for (unsigned u = blockIdx.x * RT + threadIdx.x; u < (unsigned)p.max_tokens; u += gridDim.x * RT) {
        const int i = (int)u;
        int slot = -1, pos = 0;
        if (i < grown) {
            int lo = 0, hi = p.B - 1;   // the last b with cu[b] <= i
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.cu[mid] <= i)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            pos = p.seqlens[lo] - (p.cu[lo + 1] - i);
            const int page = page_or_none(p, p.table[(long long)lo * p.max_pages + pos / p.page_size], bad);
            slot = page < 0 ? -1 : page * p.page_size + pos % p.page_size;
        }
        if (p.slots)
            p.slots[i] = slot;
        if (p.positions)
            p.positions[i] = pos;
    }
    if (bad)
        atomicOr(p.status, bad);
}

}  // namespace

cudaError_t launch_resize(const ResizeParams &p, cudaStream_t s)
{
    // one CTA where one can write the slots in a pass (or there are none)
    const bool tokens = p.slots || p.positions;
    const int ctas = tokens && p.max_tokens > RT ? CLUSTER : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(RT);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, resize_kernel, p);
}

}  // namespace fd
