// fd_serve_api.cu -- host side of the calls around decode: page bookkeeping,
// cache append, attention of new tokens over a paged cache and over packed
// prompts.  Argument checks and launches.
#include "fd.h"
#include "fd_beam.h"
#include "fd_device.cuh"
#include "fd_extend.h"
#include "fd_host.h"
#include "fd_pages.h"

#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <string.h>

using namespace fd;

namespace {

cudaStream_t stream_of(void *s) { return static_cast<cudaStream_t>(s); }

// The kernels step through sequences, tiles and keys by whole CTAs and
// blocks, in 32 bits: a step behind the last one must still fit.
constexpr int MAX_SEQUENCES = 1 << 30;
constexpr int MAX_TOKENS = INT_MAX - 2 * EXT_CT;

bool is16(int t) { return t == FD_F16 || t == FD_BF16; }

// `rows` token rows of `row` elements, `stride` elements apart, each on a
// 16-byte boundary (16 bytes are `of` elements).  A single row's stride may
// be anything.
bool stride_ok(long long stride, int rows, long long row, int of)
{
    return rows <= 1 || (stride >= row && stride % of == 0);
}

// What prefill and extend check alike.
fd_status check_extend(const ExtendParams &p, float scale)
{
    if (p.B < 0 || p.total_q < 0 || p.total_q > MAX_TOKENS || p.Hkv <= 0 || p.Hq < 0 || p.Hq % p.Hkv != 0 ||
        (long long)p.B * p.Hkv > INT_MAX || !(scale > 0.f) || isinf(scale))
        return FD_ERR_INVALID_ARG;
    if (!is16(p.dtype) || (p.d != 64 && p.d != 128) ||
        (p.out_dtype != FD_F32 && p.out_dtype != FD_F16 && p.out_dtype != FD_BF16))
        return FD_ERR_UNSUPPORTED;
    if (!stride_ok(p.q_stride, p.total_q, (long long)p.Hq * p.d, 8))
        return FD_ERR_INVALID_ARG;
    return FD_OK;
}

fd_status check_extend_pointers(const ExtendParams &p)
{
    if (!p.q || !p.cu_q || !p.out || !aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(p.v, 16) ||
        !aligned(p.out, 16) || !aligned(p.cu_q, 4) || (p.lse && !aligned(p.lse, 4)))
        return FD_ERR_INVALID_ARG;
    return FD_OK;
}

// A map of 16-bit elements [64, n1, n2, d/64 planes] with boxes [64, box1,
// box2, planes] and the 128-byte swizzle; strides in bytes.
bool map_16bit(CUtensorMap *m, const void *base, int dtype, int d, long long n1, long long s1, long long n2,
               long long s2, int box1, int box2, int planes)
{
    EncodeTiledFn fn = encode_tiled();
    if (!fn)
        return false;
    const cuuint64_t dims[4] = {64, (cuuint64_t)n1, (cuuint64_t)n2, (cuuint64_t)(d / 64)};
    const cuuint64_t strides[3] = {(cuuint64_t)s1, (cuuint64_t)s2, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)box1, (cuuint32_t)box2, (cuuint32_t)planes};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, dtype == FD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
              const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map of bytes [d, n1, n2] with boxes [d, box1, 1]: E4M3 blocks as they
// are, rows swizzled over their own length.
bool map_8bit(CUtensorMap *m, const void *base, int d, long long n1, long long n2, int box1)
{
    EncodeTiledFn fn = encode_tiled();
    if (!fn)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)n1, (cuuint64_t)n2};
    const cuuint64_t strides[2] = {(cuuint64_t)d, (cuuint64_t)n1 * d};
    const cuuint32_t box[3] = {(cuuint32_t)d, (cuuint32_t)box1, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The slices, the tiles and the workspace of a call.
struct ExtLayout {
    int G, NG, Gs, tps, grid;
    long long max_tiles;
    size_t header, tile_start, tile_blk, tiles, cost_sum, cuts, splits, part_ml, part_o, total;
};

bool ext_layout(int B, int total_q, int Hq, int Hkv, int d, ExtLayout &l)
{
    if (B < 0 || total_q < 0 || Hkv <= 0 || Hq < 0 || Hq % Hkv != 0 || (d != 64 && d != 128))
        return false;
    const int sms = sm_count();
    if (sms <= 0)
        return false;
    l.grid = sms < EXT_MAX_GRID ? sms : EXT_MAX_GRID;
    l.G = Hq > 0 ? Hq / Hkv : 1;
    l.NG = (l.G + EXT_M - 1) / EXT_M;
    l.Gs = (l.G + l.NG - 1) / l.NG;
    l.tps = EXT_M / l.Gs;
    l.max_tiles = total_q / (2 * l.tps) + (long long)B;
    const long long slots = ext_slots(l.grid);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t was = at;
        at += round_up(bytes, 256);
        return was;
    };
    l.header = take(sizeof(ExtPlanHeader));
    l.tile_start = take((size_t)B * sizeof(int));
    l.tile_blk = take((size_t)l.max_tiles * sizeof(int));
    l.tiles = take((size_t)l.max_tiles * sizeof(ExtTile));
    l.cost_sum = take((size_t)(l.max_tiles + 1) * sizeof(long long));
    l.cuts = take((size_t)(l.grid + 1) * sizeof(ExtCut));
    l.splits = take((size_t)l.grid * sizeof(ExtSplit));
    l.part_ml = take((size_t)slots * 2 * EXT_M * sizeof(float2));
    l.part_o = take((size_t)slots * 2 * EXT_M * d * sizeof(float));
    l.total = at;
    return l.max_tiles * Hkv * l.NG <= MAX_SEQUENCES;
}

fd_status run_extend(ExtendParams &p, float scale, void *workspace, size_t workspace_bytes, void *stream)
{
    p.scale_log2 = scale * 1.4426950408889634f;
    if (!(p.scale_log2 > 0.f) || isinf(p.scale_log2))
        return FD_ERR_INVALID_ARG;
    if (sm_count() <= 0)
        return FD_ERR_CUDA;
    ExtLayout l;
    if (!ext_layout(p.B, p.total_q, p.Hq, p.Hkv, p.d, l))
        return FD_ERR_UNSUPPORTED;   // too many tiles
    if (!workspace || workspace_bytes < l.total || !aligned(workspace, 256))
        return FD_ERR_WORKSPACE;
    p.status = status_ptr();
    if (!p.status)
        return FD_ERR_CUDA;
    const cudaStream_t cs = stream_of(stream);

    p.G = l.G;
    p.NG = l.NG;
    p.Gs = l.Gs;
    p.tps = l.tps;
    p.grid = l.grid;
    p.max_tiles = (int)l.max_tiles;
    p.wait_ns = ext_wait_ns(l.max_tiles, p.paged ? (long long)p.page_size * p.max_pages : p.total_k);
    char *ws = static_cast<char *>(workspace);
    p.header = reinterpret_cast<ExtPlanHeader *>(ws + l.header);
    p.tile_start = reinterpret_cast<int *>(ws + l.tile_start);
    p.tile_blk = reinterpret_cast<int *>(ws + l.tile_blk);
    p.tiles = reinterpret_cast<ExtTile *>(ws + l.tiles);
    p.cost_sum = reinterpret_cast<long long *>(ws + l.cost_sum);
    p.cuts = reinterpret_cast<ExtCut *>(ws + l.cuts);
    p.splits = reinterpret_cast<ExtSplit *>(ws + l.splits);
    p.part_ml = reinterpret_cast<float2 *>(ws + l.part_ml);
    p.part_o = reinterpret_cast<float *>(ws + l.part_o);

    // (a map's strides are checked whatever its extents)
    if (p.total_q == 1)
        p.q_stride = (long long)p.Hq * p.d;
    if (p.total_k == 1)
        p.k_stride = p.v_stride = (long long)p.Hkv * p.d;

    const long long row = (long long)p.d * 2;
    bool ok = map_16bit(&p.tmq, p.q, p.dtype, p.d, p.Hq, row, p.total_q, p.q_stride * 2, p.Gs, p.tps, 1);
    if (p.paged) {
        p.box_rows = EXT_MIN_PAGE;   // the largest power of two up to a block that divides the page
        while (p.box_rows < EXT_CT && p.page_size % (2 * p.box_rows) == 0)
            p.box_rows *= 2;
    }
    if (p.paged ? p.max_pages > 0 : p.total_k > 0) {
        for (int i = 0; i < 2; ++i) {
            CUtensorMap *m = i ? &p.tmv : &p.tmk;
            const void *x = i ? p.v : p.k;
            ok = ok && (p.f8      ? map_8bit(m, x, p.d, p.page_size, p.num_pages * p.Hkv, p.box_rows)
                        : p.paged ? map_16bit(m, x, p.dtype, p.d, p.page_size, row, p.num_pages * p.Hkv,
                                              row * p.page_size, p.box_rows, 1, p.box_rows == EXT_CT ? p.d / 64 : 1)
                                  : map_16bit(m, x, p.dtype, p.d, p.total_k, (i ? p.v_stride : p.k_stride) * 2,
                                              p.Hkv, row, EXT_CT, 1, p.d / 64));
        }
    } else {
        p.tmk = p.tmv = p.tmq;   // no key anywhere: never used
    }
    if (!ok)
        return FD_ERR_CUDA;
    cudaError_t e = launch_extend_plan(p, cs);
    if (e == cudaSuccess)
        e = p.f8                 ? launch_extend_e4m3(p, cs)
            : p.dtype == FD_BF16 ? launch_extend_bf16(p, cs)
                                 : launch_extend_f16(p, cs);
    if (e == cudaSuccess)
        e = launch_extend_merge(p, cs);
    return e == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

fd_status extend_paged(const void *q, fd_dtype q_dtype, const void *k_pages, const void *v_pages,
                       const float *k_scale, const float *v_scale, const int32_t *block_table,
                       const int32_t *cu_q, const int32_t *seqlens, int B, int total_q, int Hq, int Hkv, int d,
                       long long q_stride, int page_size, int max_pages, long long num_pages, bool f8,
                       float scale, void *out, fd_dtype out_dtype, float *lse, void *workspace,
                       size_t workspace_bytes, void *stream)
{
    ExtendParams p;
    memset(&p, 0, sizeof p);
    p.q = q;
    p.q_stride = q_stride;
    p.k = k_pages;
    p.v = v_pages;
    p.paged = 1;
    p.table = block_table;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.cu_q = cu_q;
    p.seqlens = seqlens;
    p.B = B;
    p.total_q = total_q;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.d = d;
    p.causal = 1;
    p.f8 = f8;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.dtype = q_dtype;
    p.out = out;
    p.out_dtype = out_dtype;
    p.lse = lse;
    if (page_size < 1 || max_pages < 0 || num_pages < 0 || (long long)page_size * max_pages > MAX_TOKENS)
        return FD_ERR_INVALID_ARG;
    fd_status st = check_extend(p, scale);
    if (st != FD_OK)
        return st;
    if (page_size % 16 != 0 || num_pages * Hkv > INT_MAX)
        return FD_ERR_UNSUPPORTED;
    if (B == 0 || total_q == 0 || Hq == 0)
        return FD_OK;
    if ((st = check_extend_pointers(p)) != FD_OK)
        return st;
    if (!seqlens || !aligned(seqlens, 4) || !aligned(block_table, 4) ||
        (max_pages > 0 && (!k_pages || !v_pages || !block_table || num_pages < 1)) ||
        (f8 && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4))))
        return FD_ERR_INVALID_ARG;
    return run_extend(p, scale, workspace, workspace_bytes, stream);
}

}  // namespace

extern "C" {

size_t fd_workspace_size_extend(int B, int total_q, int Hq, int Hkv, int d)
{
    ExtLayout l;
    return ext_layout(B, total_q, Hq, Hkv, d, l) ? l.total : 0;
}

fd_status fd_prefill(const void *q, const void *k, const void *v, const int32_t *cu_q, const int32_t *cu_k, int B,
                     int total_q, int total_k, int Hq, int Hkv, int d, long long q_stride, long long k_stride,
                     long long v_stride, fd_dtype in_dtype, int causal, float scale, void *out, fd_dtype out_dtype,
                     float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    ExtendParams p;
    memset(&p, 0, sizeof p);
    p.q = q;
    p.q_stride = q_stride;
    p.k = k;
    p.v = v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.B = B;
    p.total_q = total_q;
    p.total_k = total_k;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.d = d;
    p.causal = causal != 0;
    p.dtype = in_dtype;
    p.out = out;
    p.out_dtype = out_dtype;
    p.lse = lse;
    if (total_k < 0 || total_k > MAX_TOKENS)
        return FD_ERR_INVALID_ARG;
    fd_status st = check_extend(p, scale);
    if (st != FD_OK)
        return st;
    if (!stride_ok(k_stride, total_k, (long long)Hkv * d, 8) || !stride_ok(v_stride, total_k, (long long)Hkv * d, 8))
        return FD_ERR_INVALID_ARG;
    if (B == 0 || total_q == 0 || Hq == 0)
        return FD_OK;
    if ((st = check_extend_pointers(p)) != FD_OK)
        return st;
    if (!cu_k || !aligned(cu_k, 4) || (total_k > 0 && (!k || !v)))
        return FD_ERR_INVALID_ARG;
    return run_extend(p, scale, workspace, workspace_bytes, stream);
}

fd_status fd_extend_paged(const void *q, const void *k_pages, const void *v_pages, const int32_t *block_table,
                          const int32_t *cu_q, const int32_t *seqlens, int B, int total_q, int Hq, int Hkv, int d,
                          long long q_stride, int page_size, int max_pages, long long num_pages, fd_dtype in_dtype,
                          float scale, void *out, fd_dtype out_dtype, float *lse, void *workspace,
                          size_t workspace_bytes, void *stream)
{
    return extend_paged(q, in_dtype, k_pages, v_pages, nullptr, nullptr, block_table, cu_q, seqlens, B, total_q, Hq,
                        Hkv, d, q_stride, page_size, max_pages, num_pages, false, scale, out, out_dtype, lse,
                        workspace, workspace_bytes, stream);
}

fd_status fd_extend_paged_fp8(const void *q, fd_dtype q_dtype, const void *k_pages, const void *v_pages,
                              const float *k_scale, const float *v_scale, const int32_t *block_table,
                              const int32_t *cu_q, const int32_t *seqlens, int B, int total_q, int Hq, int Hkv,
                              int d, long long q_stride, int page_size, int max_pages, long long num_pages,
                              float scale, void *out, fd_dtype out_dtype, float *lse, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    return extend_paged(q, q_dtype, k_pages, v_pages, k_scale, v_scale, block_table, cu_q, seqlens, B, total_q, Hq,
                        Hkv, d, q_stride, page_size, max_pages, num_pages, true, scale, out, out_dtype, lse,
                        workspace, workspace_bytes, stream);
}

fd_status fd_resize_pages(int32_t *seqlens, const int32_t *target, int B, int32_t *block_table, int max_pages,
                          int32_t *free_pages, int32_t *free_count, int num_pages, int page_size, int32_t *slots,
                          int32_t *positions, int max_tokens, int32_t *cu_new, void *stream)
{
    if (B < 0 || B > MAX_SEQUENCES || max_pages < 0 || num_pages < 0 || page_size < 1 || max_tokens < 0 ||
        (long long)page_size * max_pages > INT_MAX || (long long)page_size * num_pages > INT_MAX)
        return FD_ERR_INVALID_ARG;
    const bool tokens = slots || positions;
    if (!free_count || !aligned(free_count, 4) || (num_pages > 0 && !free_pages) || !aligned(free_pages, 4) ||
        (B > 0 && (!seqlens || !target)) || !aligned(seqlens, 4) || !aligned(target, 4) ||
        (B > 0 && max_pages > 0 && !block_table) || !aligned(block_table, 4) || !aligned(slots, 4) ||
        !aligned(positions, 4) || !aligned(cu_new, 4) || (tokens && !cu_new))
        return FD_ERR_INVALID_ARG;
    ResizeParams p;
    memset(&p, 0, sizeof p);
    p.seqlens = seqlens;
    p.target = target;
    p.B = B;
    p.table = block_table;
    p.max_pages = max_pages;
    p.page_size = page_size;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.num_pages = num_pages;
    p.slots = slots;
    p.positions = positions;
    p.max_tokens = tokens ? max_tokens : INT_MAX;
    p.cu = cu_new;
    p.status = status_ptr();
    if (!p.status)
        return FD_ERR_CUDA;
    return launch_resize(p, stream_of(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

namespace {

fd_status append(AppendParams &p, long long num_pages, void *stream)
{
    const int of = p.dtype == FD_F32 ? 4 : 8;   // elements of 16 bytes
    if (p.T < 0 || p.H < 0 || p.page_size < 1 || num_pages < 0 || p.d < 1 ||
        num_pages > INT_MAX / p.page_size || (long long)p.H * p.d > INT_MAX)
        return FD_ERR_INVALID_ARG;
    if ((p.dtype != FD_F32 && !is16(p.dtype)) || (p.d != 64 && p.d != 128 && p.d != 256))
        return FD_ERR_UNSUPPORTED;
    if (!stride_ok(p.k_stride, p.T, (long long)p.H * p.d, of) || !stride_ok(p.v_stride, p.T, (long long)p.H * p.d, of))
        return FD_ERR_INVALID_ARG;
    if (p.T == 0 || p.H == 0)
        return FD_OK;
    if (!p.k || !p.v || !p.slots || !p.k_pages || !p.v_pages || !aligned(p.k, 16) || !aligned(p.v, 16) ||
        !aligned(p.k_pages, 16) || !aligned(p.v_pages, 16) || !aligned(p.slots, 4) ||
        (p.f8 && (p.B < 1 || p.B > MAX_SEQUENCES || !p.cu || !p.k_scale || !p.v_scale || !aligned(p.cu, 4) || !aligned(p.k_scale, 4) ||
                  !aligned(p.v_scale, 4))))
        return FD_ERR_INVALID_ARG;
    p.num_slots = num_pages * p.page_size;
    p.status = status_ptr();
    if (!p.status)
        return FD_ERR_CUDA;
    return launch_append(p, stream_of(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

}  // namespace

fd_status fd_append_paged(const void *k, const void *v, const int32_t *slots, int total, int Hkv, int d,
                          long long k_stride, long long v_stride, fd_dtype dtype, void *k_pages, void *v_pages,
                          int page_size, long long num_pages, void *stream)
{
    AppendParams p;
    memset(&p, 0, sizeof p);
    p.k = k;
    p.v = v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.T = total;
    p.H = Hkv;
    p.d = d;
    p.dtype = dtype;
    p.slots = slots;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.page_size = page_size;
    return append(p, num_pages, stream);
}

fd_status fd_append_paged_fp8(const void *k, const void *v, const float *k_scale, const float *v_scale,
                              const int32_t *cu_new, const int32_t *slots, int B, int total, int Hkv, int d,
                              long long k_stride, long long v_stride, fd_dtype dtype, void *k_pages, void *v_pages,
                              int page_size, long long num_pages, void *stream)
{
    AppendParams p;
    memset(&p, 0, sizeof p);
    p.k = k;
    p.v = v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.T = total;
    p.H = Hkv;
    p.d = d;
    p.dtype = dtype;
    p.slots = slots;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.page_size = page_size;
    p.f8 = 1;
    p.B = B;
    p.cu = cu_new;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    return append(p, num_pages, stream);
}

namespace {

fd_status append_rope(RopeParams &p, long long num_pages, void *stream)
{
    const int of = p.dtype == FD_F32 ? 4 : 8;   // elements of 16 bytes
    if (p.T < 0 || p.H < 1 || p.Hq < 0 || p.page_size < 1 || num_pages < 0 || p.d < 1 || p.max_position < 0 ||
        num_pages > INT_MAX / p.page_size || ((long long)p.Hq + 2LL * p.H) * p.d > INT_MAX)
        return FD_ERR_INVALID_ARG;
    if ((p.dtype != FD_F32 && !is16(p.dtype)) || (p.d != 64 && p.d != 128 && p.d != 256) || p.rot < 16 ||
        p.rot > p.d || p.rot % 16 != 0)
        return FD_ERR_UNSUPPORTED;
    const long long row = (long long)p.H * p.d, qrow = (long long)p.Hq * p.d;
    if (!stride_ok(p.k_stride, p.T, row, of) || !stride_ok(p.v_stride, p.T, row, of) ||
        (p.Hq > 0 && (!stride_ok(p.q_stride, p.T, qrow, of) || !stride_ok(p.q_out_stride, p.T, qrow, of))))
        return FD_ERR_INVALID_ARG;
    if (p.T == 0)
        return FD_OK;
    if (!p.k || !p.v || !p.slots || !p.positions || !p.table || !p.k_pages || !p.v_pages || !aligned(p.k, 16) ||
        !aligned(p.v, 16) || !aligned(p.table, 16) || !aligned(p.k_pages, 16) || !aligned(p.v_pages, 16) ||
        !aligned(p.slots, 4) || !aligned(p.positions, 4) ||
        (p.Hq > 0 && (!p.q || !p.q_out || !aligned(p.q, 16) || !aligned(p.q_out, 16))) ||
        (p.f8 && (p.B < 1 || p.B > MAX_SEQUENCES || !p.cu || !p.k_scale || !p.v_scale || !aligned(p.cu, 4) ||
                  !aligned(p.k_scale, 4) || !aligned(p.v_scale, 4))))
        return FD_ERR_INVALID_ARG;
    p.num_slots = num_pages * p.page_size;
    p.status = status_ptr();
    p.sms = sm_count();
    if (!p.status || p.sms <= 0)
        return FD_ERR_CUDA;
    return launch_rope(p, stream_of(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

}  // namespace

fd_status fd_append_rope_paged(const void *q, const void *k, const void *v, const int32_t *slots,
                               const int32_t *positions, const float *rope, int max_position, int rot,
                               int interleaved, int total, int Hq, int Hkv, int d, long long q_stride,
                               long long k_stride, long long v_stride, fd_dtype dtype, void *q_out,
                               long long q_out_stride, void *k_pages, void *v_pages, int page_size,
                               long long num_pages, void *stream)
{
    RopeParams p;
    memset(&p, 0, sizeof p);
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.q_stride = q_stride;
    p.q_out_stride = q_out_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.positions = positions;
    p.table = rope;
    p.max_position = max_position;
    p.rot = rot;
    p.pairs = interleaved != 0;
    p.T = total;
    p.Hq = Hq;
    p.H = Hkv;
    p.d = d;
    p.dtype = dtype;
    p.slots = slots;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.page_size = page_size;
    return append_rope(p, num_pages, stream);
}

fd_status fd_append_rope_paged_fp8(const void *q, const void *k, const void *v, const float *k_scale,
                                   const float *v_scale, const int32_t *cu_new, const int32_t *slots,
                                   const int32_t *positions, const float *rope, int max_position, int rot,
                                   int interleaved, int B, int total, int Hq, int Hkv, int d, long long q_stride,
                                   long long k_stride, long long v_stride, fd_dtype dtype, void *q_out,
                                   long long q_out_stride, void *k_pages, void *v_pages, int page_size,
                                   long long num_pages, void *stream)
{
    RopeParams p;
    memset(&p, 0, sizeof p);
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.q_stride = q_stride;
    p.q_out_stride = q_out_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.positions = positions;
    p.table = rope;
    p.max_position = max_position;
    p.rot = rot;
    p.pairs = interleaved != 0;
    p.T = total;
    p.Hq = Hq;
    p.H = Hkv;
    p.d = d;
    p.dtype = dtype;
    p.slots = slots;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.page_size = page_size;
    p.f8 = 1;
    p.B = B;
    p.cu = cu_new;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    return append_rope(p, num_pages, stream);
}

namespace {

// The parts of a selection and its workspace, for the type with the most
// segments (`elem` bytes an element).
struct SelectLayout {
    int segs, parts;
    size_t part, total;
};

bool select_sizes_ok(int R, int W, int V, int K)
{
    return R >= 0 && W >= 1 && W <= BEAM_MAX_W && V >= 1 && K >= 1 && K <= BEAM_MAX_K &&
           (long long)W * V <= MAX_SEQUENCES && K <= (long long)W * V && (long long)R * W <= INT_MAX;
}

SelectLayout select_layout(int R, int W, int V, int elem, int sms)
{
    SelectLayout l;
    l.segs = select_segs(V, elem);
    // A warp a part: as many as the card holds at once beside a CTA for each
    // request's choice, which then waits there already (32 requests of 4 beams,
    // float32: 17.8 us, with all places taken 19.5); and more where a part would
    // be longer than SEL_RUN reads: shorter ones even out what finished beams
    // leave over (64 requests of 8 beams, a tenth finished: 30.6, of 14 reads
    // 34.6).
    const long long reads = (l.segs + SEL_SEGS - 1) / SEL_SEGS, rows = (long long)R * W;
    const long long least = (reads + SEL_RUN - 1) / SEL_RUN, ctas = (long long)sms * SEL_CTAS - (R < sms ? R : sms);
    long long parts = rows > 0 ? ctas * (SEL_THREADS / 32) / rows : 1;
    parts = parts < least ? least : parts;
    l.parts = (int)(parts < reads ? parts : reads);
    l.part = round_up((size_t)R * W * l.segs * sizeof(float), 256);
    l.total = l.part + (size_t)R * W * l.parts * sizeof(float2);
    return l;
}

}  // namespace

size_t fd_workspace_size_beam(int R, int W, int V, int K)
{
    const int sms = sm_count();
    if (!select_sizes_ok(R, W, V, K) || sms <= 0)
        return 0;
    const size_t a = select_layout(R, W, V, 4, sms).total, b = select_layout(R, W, V, 2, sms).total;
    return round_up(a > b ? a : b, 256) + (R == 0 ? 256 : 0);
}

fd_status fd_beam_select(const void *logits, fd_dtype dtype, long long request_stride, long long beam_stride,
                         const float *scores, const uint8_t *finished, int R, int W, int V, int K, int eos,
                         float *out_scores, int32_t *out_parents, int32_t *out_tokens, uint8_t *out_finished,
                         void *workspace, size_t workspace_bytes, void *stream)
{
    if (!select_sizes_ok(R, W, V, K) || request_stride < 0 || beam_stride < 0 || eos < -1 || eos >= V ||
        (finished && eos < 0))
        return FD_ERR_INVALID_ARG;
    if (dtype != FD_F32 && !is16(dtype))
        return FD_ERR_UNSUPPORTED;
    if (R == 0)
        return FD_OK;
    const int elem = dtype == FD_F32 ? 4 : 2;
    if (!logits || !aligned(logits, elem) || !scores || !aligned(scores, 4) || !out_scores || !out_parents ||
        !out_tokens || !aligned(out_scores, 4) || !aligned(out_parents, 4) || !aligned(out_tokens, 4))
        return FD_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms <= 0)
        return FD_ERR_CUDA;
    const SelectLayout l = select_layout(R, W, V, elem, sms);
    if ((long long)R * W * l.parts > INT_MAX)
        return FD_ERR_UNSUPPORTED;   // more rows than a card holds
    if (!workspace || workspace_bytes < l.total || !aligned(workspace, 256))
        return FD_ERR_WORKSPACE;
    SelectParams p;
    memset(&p, 0, sizeof p);
    p.logits = logits;
    p.r_stride = request_stride;
    p.w_stride = beam_stride;
    p.dtype = dtype;
    p.scores = scores;
    p.finished = finished;
    p.R = R;
    p.W = W;
    p.V = V;
    p.K = K;
    p.eos = eos;
    p.out_scores = out_scores;
    p.out_parents = out_parents;
    p.out_tokens = out_tokens;
    p.out_finished = out_finished;
    p.segs = l.segs;
    p.parts = l.parts;
    p.reads = (l.segs + SEL_SEGS - 1) / SEL_SEGS / l.parts;
    p.longer = (l.segs + SEL_SEGS - 1) / SEL_SEGS % l.parts;
    p.seg_max = static_cast<float *>(workspace);
    p.part = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + l.part);
    return launch_select(p, stream_of(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

namespace {

struct ReorderLayout {
    int tiles;
    size_t lens, copied, freed, pages, moved, freed_before, needed_before, total;
};

bool reorder_layout(int R, int W, int max_pages, ReorderLayout &l)
{
    if (R < 0 || W < 1 || W > BEAM_MAX_W || max_pages < 0 || (long long)R * W > MAX_SEQUENCES)
        return false;
    l.tiles = max_pages > 0 ? (int)(((long long)max_pages + REORDER_TILE - 1) / REORDER_TILE) : 1;
    const size_t all = (size_t)R * l.tiles;
    size_t at = round_up(sizeof(ReorderHeader), 256);
    auto take = [&](size_t bytes) {
        const size_t was = at;
        at += round_up(bytes, 256);
        return was;
    };
    l.lens = take((size_t)R * W * sizeof(int32_t));
    l.copied = take((size_t)R * sizeof(unsigned));
    l.freed = take(all * sizeof(int32_t));
    l.pages = take(all * W * REORDER_TILE * sizeof(int32_t));
    l.moved = take(all * (REORDER_TILE / 8));
    l.freed_before = take(all * sizeof(long long));
    l.needed_before = take((size_t)R * sizeof(int32_t));
    l.total = at;
    return (long long)R * l.tiles <= INT_MAX;
}

}  // namespace

size_t fd_workspace_size_reorder(int R, int W, int max_pages)
{
    ReorderLayout l;
    return reorder_layout(R, W, max_pages, l) ? l.total : 0;
}

fd_status fd_reorder_pages(const int32_t *parents, int R, int W, int32_t *seqlens, int32_t *block_table,
                           int max_pages, int32_t *free_pages, int32_t *free_count, int num_pages, int page_size,
                           int32_t *copies, int32_t *granted, void *workspace, size_t workspace_bytes, void *stream)
{
    ReorderLayout l;
    if (!reorder_layout(R, W, max_pages, l) || num_pages < 0 || page_size < 1 ||
        (long long)page_size * max_pages > INT_MAX || (long long)page_size * num_pages > INT_MAX)
        return FD_ERR_INVALID_ARG;
    if (R == 0)
        return FD_OK;
    if (!parents || !aligned(parents, 4) || !seqlens || !aligned(seqlens, 4) || !free_count ||
        !aligned(free_count, 4) || (num_pages > 0 && !free_pages) || !aligned(free_pages, 4) ||
        (max_pages > 0 && !block_table) || !aligned(block_table, 4) || !copies || !aligned(copies, 4) ||
        !aligned(granted, 4))
        return FD_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < l.total || !aligned(workspace, 256))
        return FD_ERR_WORKSPACE;
    ReorderParams p;
    memset(&p, 0, sizeof p);
    p.parents = parents;
    p.R = R;
    p.W = W;
    p.seqlens = seqlens;
    p.table = block_table;
    p.max_pages = max_pages;
    p.page_size = page_size;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.num_pages = num_pages;
    p.copies = copies;
    p.granted = granted;
    p.status = status_ptr();
    if (!p.status)
        return FD_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    p.tiles = l.tiles;
    p.header = reinterpret_cast<ReorderHeader *>(ws);
    p.lens = reinterpret_cast<int32_t *>(ws + l.lens);
    p.copied = reinterpret_cast<unsigned *>(ws + l.copied);
    p.freed = reinterpret_cast<int32_t *>(ws + l.freed);
    p.pages = reinterpret_cast<int32_t *>(ws + l.pages);
    p.moved = reinterpret_cast<unsigned *>(ws + l.moved);
    p.freed_before = reinterpret_cast<long long *>(ws + l.freed_before);
    p.needed_before = reinterpret_cast<int32_t *>(ws + l.needed_before);
    return launch_reorder(p, stream_of(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

fd_status fd_copy_pages(const int32_t *copies, int n, int Hkv, int d, fd_dtype dtype, void *k_pages, void *v_pages,
                        int page_size, long long num_pages, void *stream)
{
    if (n < 0 || Hkv < 0 || page_size < 1 || num_pages < 0 || d < 1 || num_pages > INT_MAX / page_size ||
        (long long)Hkv * d > INT_MAX)
        return FD_ERR_INVALID_ARG;
    if ((dtype != FD_F32 && dtype != FD_E4M3 && !is16(dtype)) || (d != 64 && d != 128 && d != 256))
        return FD_ERR_UNSUPPORTED;
    const int row_vecs = d * (dtype == FD_F32 ? 4 : dtype == FD_E4M3 ? 1 : 2) / 16;
    if ((long long)Hkv * page_size > INT_MAX / 2 / row_vecs)
        return FD_ERR_UNSUPPORTED;   // pages of 16 GB and more
    if (n == 0 || Hkv == 0)
        return FD_OK;
    if (!copies || !aligned(copies, 4) || !k_pages || !v_pages || !aligned(k_pages, 16) || !aligned(v_pages, 16))
        return FD_ERR_INVALID_ARG;
    CopyParams p;
    memset(&p, 0, sizeof p);
    p.copies = copies;
    p.n = n;
    p.H = Hkv;
    p.page_size = page_size;
    p.row_vecs = row_vecs;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.num_pages = num_pages;
    p.status = status_ptr();
    if (!p.status)
        return FD_ERR_CUDA;
    return launch_copy_pages(p, stream_of(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

}  // extern "C"
