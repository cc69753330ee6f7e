// fd_extend_e4m3.cu -- attention of new tokens over an E4M3 cache, f16
// products (f16 and bf16 queries).
#include "fd_extend.cuh"

namespace fd {

cudaError_t launch_extend_e4m3(const ExtendParams &p, cudaStream_t s)
{
    return p.d == 64 ? launch_extend_t<__half, 64, true>(p, s) : launch_extend_t<__half, 128, true>(p, s);
}

}  // namespace fd
