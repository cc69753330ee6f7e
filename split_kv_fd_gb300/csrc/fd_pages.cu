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
#include "fd_device.cuh"
#include "fd_pages.h"

namespace fd {
namespace {

constexpr int RT = 1024;   // threads of the one CTA that keeps the books

// Inclusive sum over the block, and the block's total.
__device__ __forceinline__ long long block_scan(long long x, long long *warp_sums, long long &total)
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
    if (w == 0) {
        long long s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(FULL_MASK, s, o);
            if (lane >= o)
                s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[31];
    return x + (w ? warp_sums[w - 1] : 0);
}

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

__global__ void __launch_bounds__(RT, 1) resize_kernel(const ResizeParams p)
{
    __shared__ long long sums[32];
    const int tid = threadIdx.x;
    const long long count0 = min(max(*p.free_count, 0), p.num_pages);
    unsigned bad = 0;

    // how many pages come back
    long long back = 0;
    for (int b0 = 0; b0 < p.B; b0 += RT) {
        const int b = b0 + tid;
        long long r = 0, total;
        if (b < p.B) {
            const Change c = change_of(p, b);
            r = max(0, c.po - c.pn);
        }
        block_scan(r, sums, total);
        back += total;
    }
    const long long top = count0 + back;

    // onto the stack, the last of them first; a page that is none is kept
    // out of later calls by the range checks of whoever reads the table
    long long done = 0;
    for (int b0 = 0; back > 0 && b0 < p.B; b0 += RT) {
        const int b = b0 + tid;
        long long r = 0, total;
        Change c = {};
        if (b < p.B) {
            c = change_of(p, b);
            r = max(0, c.po - c.pn);
        }
        const long long first = done + block_scan(r, sums, total) - r;
        for (int j = 0; j < r; ++j) {
            const long long at = top - 1 - (first + j);
            const int page = p.table[(long long)b * p.max_pages + c.pn + j];
            if (page < 0 || page >= p.num_pages || at >= p.num_pages)
                bad |= STATUS_BAD_PAGE;
            if (at < p.num_pages)
                p.free_pages[at] = page;
        }
        done += total;
    }
    __syncthreads();   // what is taken below may have come back above

    // growth, in order of b, as far as the pages (and the slots) last
    long long pages = 0, tokens = 0, grown = 0, taken = 0;
    for (int b0 = 0; b0 < p.B; b0 += RT) {
        const int b = b0 + tid;
        long long need = 0, more = 0, total;
        Change c = {};
        if (b < p.B) {
            c = change_of(p, b);
            if (c.fits) {
                need = max(0, c.pn - c.po);
                more = max(0, c.newn - c.oldn);
            }
        }
        const long long cp = pages + block_scan(need, sums, total);
        pages += total;
        const long long ct = tokens + block_scan(more, sums, total);
        tokens += total;
        const bool given = b < p.B && c.fits && (need == 0 || cp <= min(top, (long long)p.num_pages)) &&
                           (more == 0 || !p.slots || ct <= p.max_tokens);
        const long long mine = given ? need : 0;
        const long long first = taken + block_scan(mine, sums, total) - mine;
        taken += total;
        for (int j = 0; j < mine; ++j) {
            const long long at = top - 1 - (first + j);
            p.table[(long long)b * p.max_pages + c.po + j] = at < p.num_pages ? p.free_pages[at] : -1;
        }
        const long long g = given ? more : 0;
        const long long cu = grown + block_scan(g, sums, total);
        grown += total;
        if (b < p.B) {
            p.seqlens[b] = given ? c.newn : c.oldn;
            if (p.cu)
                p.cu[b + 1] = (int)cu;
        }
    }
    if (tid == 0) {
        if (p.cu)
            p.cu[0] = 0;
        *p.free_count = (int)min(top - taken, (long long)p.num_pages);
    }
    if (bad)
        atomicOr(p.status, bad);
}

// A thread a token: its sequence by bisection of the offsets, then its
// position and its page.
__global__ void slots_kernel(const ResizeParams p)
{
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= p.max_tokens)
        return;
    int slot = -1, pos = 0;
    if (i < p.cu[p.B]) {
        int lo = 0, hi = p.B - 1;   // the last b with cu[b] <= i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.cu[mid] <= i)
                lo = mid;
            else
                hi = mid - 1;
        }
        pos = p.seqlens[lo] - (p.cu[lo + 1] - i);
        const int page = p.table[(long long)lo * p.max_pages + pos / p.page_size];
        slot = page < 0 ? -1 : (int)((long long)page * p.page_size + pos % p.page_size);
    }
    if (p.slots)
        p.slots[i] = slot;
    if (p.positions)
        p.positions[i] = pos;
}

}  // namespace

cudaError_t launch_resize(const ResizeParams &p, cudaStream_t s)
{
    resize_kernel<<<1, RT, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.max_tokens == 0 || (!p.slots && !p.positions))
        return e;
    slots_kernel<<<(p.max_tokens + 255) / 256, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace fd
