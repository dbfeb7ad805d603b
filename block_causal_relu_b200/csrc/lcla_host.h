// lcla_host.h -- host-side argument checks shared by the operators' entry points.
#ifndef LCLA_HOST_H
#define LCLA_HOST_H

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "lcla.h"

namespace lcla {
namespace host {

inline bool misaligned(const void *ptr) { return ((uintptr_t)ptr & 15u) != 0; }

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb)
{
    if (!a || !b || !na || !nb) return false;
    const uintptr_t a0 = (uintptr_t)a, a1 = a0 + na, b0 = (uintptr_t)b, b1 = b0 + nb;
    return a0 < b1 && b0 < a1;
}

inline int launched() { return cudaGetLastError() == cudaSuccess ? LCLA_OK : LCLA_ERR_CUDA; }

}  // namespace host
}  // namespace lcla

#endif
