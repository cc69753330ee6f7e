// fd_extend_bf16.cu -- attention of new tokens, bf16 inputs.
#include "fd_extend.cuh"

namespace fd {

cudaError_t launch_extend_bf16(const ExtendParams &p, cudaStream_t s)
{
    return p.d == 64 ? launch_extend_t<__nv_bfloat16, 64, false>(p, s) : launch_extend_t<__nv_bfloat16, 128, false>(p, s);
}

}  // namespace fd
