// fd_extend_bf16_e4m3.cu -- attention of new tokens, bf16 inputs over an E4M3 cache.
#include "fd_extend.cuh"

namespace fd {

cudaError_t launch_extend_bf16_e4m3(const ExtendParams &p, cudaStream_t s)
{
    return p.d == 64 ? launch_extend_t<__nv_bfloat16, 64, true>(p, s) : launch_extend_t<__nv_bfloat16, 128, true>(p, s);
}

}  // namespace fd
