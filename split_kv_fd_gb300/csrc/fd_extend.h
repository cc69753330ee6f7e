// fd_extend.h -- parameter block, plan and launchers of attention with
// several new tokens a sequence (fd_extend.cuh): over a paged cache, or over
// packed prompts.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fd {

// Status word bit, beside those of fd_device.cuh: offsets had to be clamped.
constexpr unsigned STATUS_BAD_OFFSETS = 4u;

// A tile's MMA rows are (token, query head of the slice) pairs, token major:
// two sub-tiles of EXT_M rows, each of EXT_M / Gs tokens.
constexpr int EXT_M = 128;
// Keys per block.
constexpr int EXT_CT = 128;
// Blocks of a link: longer ranges are taken as a chain of segments, each with
// sums of its own, joined in float32.  The tensor cores add a product to the
// running sum cut at that sum's last bits, so values of one sign come out low
// by some 6.3e-9 a key (measured, f16 and bf16): 4e-4 at a link's 64 K keys,
// below f16's half step, but 6.6e-3 at a million.  A link's end costs some 16
// us beside its 600 (2048 tokens of 64 heads over 128 K keys, three links a
// tile: 5.26 -> 5.48 ms; links of 256 blocks 5.59).
constexpr int EXT_LINK = 512;
// CTAs of the main kernel at most: the plan deals with a thread for each.
constexpr int EXT_MAX_GRID = 255;
// Boxes of a paged K/V block: at most EXT_CT / 16 row groups.
constexpr int EXT_MIN_PAGE = 16;

// One tile of a sequence's new tokens, written by the plan (as 16-byte words,
// like the other records of the plan: a warp's tiles are scattered, and word
// by word their stores took half of the plan's time).
struct alignas(16) ExtTile {
    int row0;    // first token's row of q and out
    int ntok;    // tokens
    int b;       // sequence
    int m;       // its keys
    int lim;     // keys that the tile's first token sees (may be negative)
    int k0;      // packed K/V: first row
    int nblk;    // blocks of EXT_CT keys that any of its tokens sees
    int pad;
};

// Where a CTA's share of the split tiles begins: an item (tile, virtual
// head), the offset in it in cost units, and the block that offset lies in.
struct alignas(16) ExtCut {
    int item, off, blk, pad;
};

// An item that was cut: the cuts inside it are [c0, c1).
struct alignas(16) ExtSplit {
    int c0, c1;
    int rows;    // rows of the split items before it
    int row0, ntok, b;   // its tile
    int vh;      // virtual head
    int pad;
};

struct alignas(16) ExtPlanHeader {
    int n_items;   // tiles * virtual heads
    int waves;     // whole items each CTA takes: item w * grid + c (odd w: from the far end)
    int n_splits;
    int split_rows;   // rows of all split items
};

struct ExtendParams {
    CUtensorMap tmq, tmk, tmv;
    const void *q;           // [total_q, Hq, d], q_stride elements between tokens
    long long q_stride;
    const void *k, *v;       // packed [total_k, Hkv, d] with strides, or pages [num_pages, Hkv, page_size, d]
    long long k_stride, v_stride;
    const int32_t *table;    // [B, max_pages] (paged)
    int paged, page_size, max_pages;
    int box_rows;            // rows of a K/V box
    long long num_pages;
    const int32_t *cu_q;     // [B + 1] rows of q
    const int32_t *cu_k;     // [B + 1] rows of k, v (packed)
    const int32_t *seqlens;  // [B] tokens in the cache, the new ones among them (paged)
    int B, total_q, total_k, Hq, Hkv, d;
    int G;                   // query heads per K/V head
    int NG, Gs;              // slices of a K/V head's query heads, heads per slice
    int tps;                 // tokens per sub-tile
    int causal;
    float scale_log2;        // scale * log2(e): scores are kept in base 2
    int f8;                  // E4M3 K/V
    const float *k_scale, *v_scale;   // [B, Hkv]
    int dtype;               // of q, and of K/V unless f8
    void *out;               // [total_q, Hq, d]
    int out_dtype;
    float *lse;              // [total_q, Hq] or null
    unsigned *status;
    // workspace
    int grid, max_tiles;
    unsigned long long wait_ns;   // after which a wait is given up
    ExtPlanHeader *header;
    int *tile_start;         // [B] tiles before each sequence
    int *tile_blk;           // [max_tiles] blocks of the sorted tiles
    ExtTile *tiles;          // [max_tiles] by descending cost
    long long *cost_sum;     // [max_tiles + 1] costs before, over the virtual heads
    ExtCut *cuts;            // [grid + 1]
    ExtSplit *splits;        // [grid]
    float *part_o;           // [slots][2 * EXT_M][d] sums of weights times V
    float2 *part_ml;         // [slots][2 * EXT_M] (reference max, sum of weights)
};

// How long a wait of the main kernel may last: 1 s, and what a role may
// rightly wait for.  That is the plan, which deals with a tile in some 0.04
// us (12 M sequences of a token: 0.46 s with the attention), and another
// role's whole segment (the next load of Q waits for the last block of the
// segment before), whose blocks take 1.1 to 1.5 us each; both several times
// over, for other work on the GPU.  1 s alone would end calls over some 85 M
// keys a sequence.
inline unsigned long long ext_wait_ns(long long max_tiles, long long max_keys)
{
    return 1000000000ull + 1000ull * (unsigned long long)max_tiles +
           10000ull * (unsigned long long)(max_keys / EXT_CT);
}

// Partial results: the piece that ends at a cut and the one that starts
// there, and two for each CTA: what the links of a chain have given so far,
// and what its present link gives.
inline int ext_slots(int grid) { return 2 * (grid + 1) + 2 * grid; }

cudaError_t launch_extend_plan(const ExtendParams &p, cudaStream_t s);
cudaError_t launch_extend_bf16(const ExtendParams &p, cudaStream_t s);
cudaError_t launch_extend_f16(const ExtendParams &p, cudaStream_t s);
cudaError_t launch_extend_e4m3(const ExtendParams &p, cudaStream_t s);
cudaError_t launch_extend_merge(const ExtendParams &p, cudaStream_t s);

}  // namespace fd
