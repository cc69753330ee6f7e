// fd_beam.h -- parameter blocks and launchers of beam search's selection
// (fd_beam_select.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fd {

constexpr int BEAM_MAX_W = 32;   // beams of a request
constexpr int BEAM_MAX_K = 64;   // candidates chosen of them

// A row of logits is cut into segments of SEG_BYTES, counted from the 16-byte
// boundary at or below its first element.
constexpr int SEG_BYTES = 2048;
constexpr int SEL_THREADS = 256;

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
    int per_part, parts;         // segments of a part, parts of a row
    float *seg_max;              // [R * W, segs]
    float2 *part;                // [R * W, parts]
};

// Segments that a row may have, whatever its alignment.
inline int select_segs(int V, int elem)
{
    return (int)(((long long)V * elem + 16 - elem + SEG_BYTES - 1) / SEG_BYTES);
}

cudaError_t launch_select(const SelectParams &p, cudaStream_t s);

}  // namespace fd
