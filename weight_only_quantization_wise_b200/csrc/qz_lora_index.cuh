// qz_lora_index.cuh -- how the warps of the adapters' first product share K.
// Plain C++ for host and device; the CPU tests compile it with the host compiler.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define QZ_HD __host__ __device__ __forceinline__
#else
#define QZ_HD inline
#endif

namespace qz {
namespace lora {

// First of the `steps` K steps that part `part` of `parts` takes (part =
// parts: the end).  steps < 2^26, but part * steps passes 2^31.
QZ_HD int part_begin(int part, int steps, int parts) {
    return (int)((int64_t)part * steps / parts);
}

}  // namespace lora
}  // namespace qz
