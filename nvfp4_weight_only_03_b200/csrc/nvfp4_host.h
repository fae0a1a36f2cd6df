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

// Elements from the first to the last of [n0][n1][n2][inner] with these strides, at most 2^60.
inline uint64_t span(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2,
                     int64_t inner) {
    const unsigned __int128 n = (unsigned __int128)(n0 - 1) * s0 + (unsigned __int128)(n1 - 1) * s1 +
                                (unsigned __int128)(n2 - 1) * s2 + inner;
    return n >> 60 ? 1ull << 60 : (uint64_t)n;
}

// Bytes that K (or V) of a cache with at least one page takes.
inline uint64_t cache_bytes(const nvfp4_kv_cache_t& c) {
    return (c.type == NVFP4_KV_E4M3 ? 1ull : 2ull) * span(c.blocks, c.block_stride, c.block_size,
                                                          c.slot_stride, c.heads, c.head_stride, c.dim);
}

// Launches a kernel whose blocks may be set up while the work before it on the stream ends; it waits
// (griddepcontrol.wait) before it reads or writes anything.  cluster 0: no cluster.
template <typename... P, typename... A>
int launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                  cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return NVFP4_OK;
    cudaGetLastError();
    return NVFP4_ERR_LAUNCH;
}

}  // namespace nvfp4_host

#endif
