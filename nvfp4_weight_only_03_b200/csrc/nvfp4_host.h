// Host-side helpers shared by the library's translation units (defined in nvfp4_host.cu).
#ifndef NVFP4_HOST_H
#define NVFP4_HOST_H

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "nvfp4.h"

namespace nvfp4_host {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The current device (NVFP4_ERR_ARCH unless a B200), its SM count and the tensor-map encoder.
int device(int* dev, int* sms, EncodeFn* encode);

inline bool misaligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0;
}

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte.
inline bool overlaps(const void* a, uint64_t na, const void* b, uint64_t nb) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return a && b && na && nb && pa < pb + nb && pb < pa + na;
}

// Clears a failed launch's error and turns it into a status.
inline int launched() { return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH; }

}  // namespace nvfp4_host

#endif
