// fd_extend_e4m3.cu -- attention with several new tokens a sequence: token t of
// sequence b, the i-th of its n new ones over m keys, sees the keys below
// m - n + i + 1 (causal) or all m,
//     out = softmax(scale q K^T) V,   lse = ln sum exp(scale q K^T),
// in one pass over the keys with a running maximum and sum.
#include "fd_device.cuh"
#include "fd_extend.h"

namespace fd {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__nv_fp8_e4m3 x) { return (float)x; }

// One warp a (token, query head); lane l holds elements l, l + 32, ...
template <typename T, typename KT, int D> __global__ void extend_simple_kernel(const ExtendParams p)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x;
    // the token's sequence: the last b whose rows start at or before it
    int b = -1, n = 0, i = 0;
    for (int lo = 0, x = 0; x < p.B; ++x) {
        const int a = min(max(p.cu_q[x], lo), p.total_q), e = min(max(p.cu_q[x + 1], a), p.total_q);
        if (t == 0 && threadIdx.x == 0 && (a != p.cu_q[x] || e != p.cu_q[x + 1]))
            atomicOr(p.status, STATUS_BAD_OFFSETS);
        if (t >= a && t < e) {
            b = x;
            n = e - a;
            i = t - a;
        }
        lo = e;
    }
    if (b < 0)
        return;   // behind the last sequence
    long long m, k0 = 0;
    if (p.paged) {
        m = min((long long)max(p.seqlens[b], 0), (long long)p.page_size * p.max_pages);
    } else {
        const int a = min(max(p.cu_k[b], 0), p.total_k), e = min(max(p.cu_k[b + 1], a), p.total_k);
        k0 = a;
        m = e - a;
    }
    const long long see = p.causal ? max(0LL, min(m, m - n + i + 1)) : m;
    const int G = p.Hq / p.Hkv;
    for (int hq = threadIdx.x >> 5; hq < p.Hq; hq += blockDim.x >> 5) {
        const int h = hq / G;
        float q[E], o[E], mx = -INFINITY, l = 0.f;
        float ks = p.scale_log2, vs = 1.f;
        if (p.f8) {
            ks *= p.k_scale[(long long)b * p.Hkv + h];
            vs = p.v_scale[(long long)b * p.Hkv + h];
        }
        for (int e = 0; e < E; ++e) {
            q[e] = to_f(static_cast<const T *>(p.q)[t * p.q_stride + (long long)hq * D + lane + 32 * e]);
            o[e] = 0.f;
        }
        for (long long j = 0; j < see; ++j) {
            long long kr, vr;
            if (p.paged) {
                int page = p.table[(long long)b * p.max_pages + j / p.page_size];
                if (page < 0 || page >= p.num_pages) {
                    if (lane == 0)
                        atomicOr(p.status, STATUS_BAD_PAGE);
                    page = 0;
                }
                kr = vr = (((long long)page * p.Hkv + h) * p.page_size + j % p.page_size) * D;
            } else {
                kr = (k0 + j) * p.k_stride + (long long)h * D;
                vr = (k0 + j) * p.v_stride + (long long)h * D;
            }
            float s = 0.f;
            for (int e = 0; e < E; ++e)
                s = fmaf(q[e], to_f(static_cast<const KT *>(p.k)[kr + lane + 32 * e]), s);
            for (int x = 16; x; x >>= 1)
                s += __shfl_xor_sync(FULL_MASK, s, x);
            s *= ks;
            const float mn = fmaxf(mx, s);
            const float a = mn == -INFINITY ? 1.f : ex2(mx - mn);
            const float w = mn == -INFINITY ? 0.f : ex2(s - mn);
            l = fmaf(l, a, w);
            for (int e = 0; e < E; ++e)
                o[e] = fmaf(w, to_f(static_cast<const KT *>(p.v)[vr + lane + 32 * e]), o[e] * a);
            mx = mn;
        }
        const long long row = (long long)t * p.Hq + hq;
        const float inv = l > 0.f ? vs / l : 0.f;
        for (int e = 0; e < E; ++e)
            store_out(p.out, row * D + lane + 32 * e, p.out_dtype, o[e] * inv);
        if (p.lse && lane == 0)
            p.lse[row] = l > 0.f ? (mx + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

template <typename T> cudaError_t launch_t(const ExtendParams &p, cudaStream_t s)
{
    auto kern = p.d == 64 ? extend_simple_kernel<T, __nv_fp8_e4m3, 64> : extend_simple_kernel<T, __nv_fp8_e4m3, 128>;
    kern<<<p.total_q, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_extend_e4m3(const ExtendParams &p, cudaStream_t s)
{
    return p.dtype == 1 ? launch_t<__half>(p, s) : launch_t<__nv_bfloat16>(p, s);
}

}  // namespace fd
