// fd_beam.h -- parameter blocks and launchers of beam search: selection
// (fd_beam_select.cu) and the reordering of the beams' cached states
// (fd_beam_pages.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fd {

constexpr int BEAM_MAX_W = 32;   // beams of a request
constexpr int BEAM_MAX_K = 64;   // candidates chosen of them

// A row of logits is cut into segments of SEG_BYTES, counted from the 16-byte
// boundary at or below its first element.
constexpr int SEG_BYTES = 512;
constexpr int SEL_SEGS = 4;       // segments that a warp reads at a time
constexpr int SEL_THREADS = 256;
constexpr int SEL_CTAS = 4;       // of the rows' kernel on an SM
constexpr int SEL_RUN = 8;        // reads of a part, at most
constexpr int SEL_STAGES = 3;     // reads under way or taken, of a warp

struct SelectParams {
    const void *logits;          // [R, W, V], strides in elements
    long long r_stride, w_stride;
    int dtype;
    const float *scores;         // [R, W]
    const uint8_t *finished;     // [R, W] or null
    int R, W, V, K, eos;
    float *out_scores;           // [R, K]
    int32_t *out_parents, *out_tokens;
    uint8_t *out_finished;       // [R, K] or null
    // workspace: of every row the largest value of each segment, and the
    // maximum and sum of exponentials of each part
    int segs;                    // segments of a row
    int parts;                   // of a row
    int reads, longer;           // of SEL_SEGS segments: a part's, and how many parts have one more
    float *seg_max;              // [R * W, segs]
    float2 *part;                // [R * W, parts]
};

// Segments that a row may have, whatever its alignment.
inline int select_segs(int V, int elem)
{
    return (int)(((long long)V * elem + 16 - elem + SEG_BYTES - 1) / SEG_BYTES);
}

cudaError_t launch_select(const SelectParams &p, cudaStream_t s);

// A request's tables are taken in tiles of this many places.
constexpr int REORDER_TILE = 256;
// Up to this many tiles (and requests) every CTA adds up what lies before it
// by itself; a kernel of its own does for more.
constexpr int REORDER_SCAN = 1024;

struct ReorderHeader {
    int count;           // the stack's height before the call
    int top, taken;      // its height with what came back, as far as that is kept, and pages taken from there
    long long back;      // pages that came back
};

struct ReorderParams {
    const int32_t *parents;      // [R, W]
    int R, W;
    int32_t *seqlens;            // [R, W] in, out
    int32_t *table;              // [R * W, max_pages] in, out
    int max_pages, page_size;
    int32_t *free_pages;         // [num_pages] stack, in, out
    int32_t *free_count;         // [1] in, out
    int num_pages;
    int32_t *copies;             // [R, W, 3]: page from, page to, rows
    int32_t *granted;            // [R] or null
    unsigned *status;
    // workspace
    int tiles;                   // of a request
    ReorderHeader *header;
    int32_t *lens;               // [R, W] lengths before the call
    unsigned *copied;            // [R] new beams that need a copy
    int32_t *freed;              // [R, tiles] pages that come back ...
    int32_t *pages;              // [R, tiles, W * REORDER_TILE] ... and which
    unsigned *moved;             // [R, tiles, REORDER_TILE / 32] places whose entries change hands
    long long *freed_before;     // [R, tiles] of granted requests before it (more than REORDER_SCAN)
    int32_t *needed_before;      // [R] of granted requests before it, -1 if it is refused
};

cudaError_t launch_reorder(const ReorderParams &p, cudaStream_t s);

struct CopyParams {
    const int32_t *copies;       // [n, 3]
    int n, H, page_size;
    int row_vecs;                // 16-byte vectors of a row
    void *k_pages, *v_pages;     // [num_pages, H, page_size, row]
    long long num_pages;
    unsigned *status;
};

cudaError_t launch_copy_pages(const CopyParams &p, cudaStream_t s);

}  // namespace fd
