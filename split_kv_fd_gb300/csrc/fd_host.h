// fd_host.h -- what the host files of the C ABI share: the current device's
// properties, its status word, the tensor-map encoder and argument checks.
#pragma once

#include <cuda.h>
#include <stddef.h>
#include <stdint.h>

namespace fd {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// The current device, its SM count (-1 on a CUDA error), and the device
// address of its status word (null on a CUDA error).
int current_device();
int sm_count();
unsigned *status_ptr();

// cuTensorMapEncodeTiled, fetched from the driver through the runtime (no
// link-time dependency on the driver library); null if it is missing.
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled();

}  // namespace fd
