// Elements of 16-byte vectors, and the checks that the stateless operators on them share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tkv.h"
#include "tkv_internal.h"

namespace tkv {

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* at, float x) { *at = x; }
__device__ __forceinline__ void put(__nv_bfloat16* at, float x) { *at = __float2bfloat16_rn(x); }

// Elements as they lie in a 16-byte vector.
template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void unpack(const int4& v, float* x) {
    x[0] = __int_as_float(v.x); x[1] = __int_as_float(v.y); x[2] = __int_as_float(v.z); x[3] = __int_as_float(v.w);
  }
  static __device__ __forceinline__ int4 pack(const float* x) {
    return make_int4(__float_as_int(x[0]), __float_as_int(x[1]), __float_as_int(x[2]), __float_as_int(x[3]));
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void unpack(const int4& v, float* x) {
    const int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __int_as_float(w[i] << 16);
      x[2 * i + 1] = __int_as_float(w[i] & 0xffff0000);
    }
  }
  static __device__ __forceinline__ int4 pack(const float* x) {
    int w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const int*>(&h);
    }
    return make_int4(w[0], w[1], w[2], w[3]);
  }
};

inline bool misaligned(const void* ptr, size_t to) { return reinterpret_cast<uintptr_t>(ptr) % to != 0; }

inline int launched(const char* what, cudaError_t e) {
  return e == cudaSuccess ? TKV_OK : report(TKV_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
}

// Launches a kernel whose CTAs may be set up while the kernel ahead of it on the
// stream ends. Every thread of it waits for that one (cudaGridDependencySynchronize)
// before it touches memory, so that its own end is the end of all before it. cluster:
// CTAs of a cluster.
template <typename P, typename... A>
cudaError_t launch_early(void (*kernel)(P, A...), dim3 ctas, int threads, int bytes, cudaStream_t s, int cluster, const P& p, A... more) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = ctas;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, more...);
}

inline int check_dtype(int32_t dtype) {
  return dtype == TKV_DTYPE_F32 || dtype == TKV_DTYPE_BF16 ? TKV_OK : report(TKV_ERR_INVALID_ARG, "dtype");
}

}  // namespace tkv
