// fd_extend_f16.cu -- attention of new tokens, f16 inputs.
#include "fd_extend.cuh"

namespace fd {

cudaError_t launch_extend_f16(const ExtendParams &p, cudaStream_t s)
{
    return p.d == 64 ? launch_extend_t<__half, 64, false>(p, s) : launch_extend_t<__half, 128, false>(p, s);
}

}  // namespace fd
