// Shared by the operators of a paged cache held in 8 bits.
//
// A BLOCK is the 16 slots of a page, one KV head, K or V: 16 rows of int8 codes
// and one fp32 scale; a row's value is code * scale. The pool is
// [pages][Hkv][2][16][D] codes, the scales [pages][Hkv][2].
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tkv.h"
#include "tkv_internal.h"

namespace tkv {

constexpr uint32_t kFullMask = 0xffffu;

struct PoolRef {
  int8_t* codes;
  float* scales;
  int64_t pages;
  const int32_t* table;
  int64_t table_stride;
  uint32_t* mask;         // may be null
  int32_t hkv;
};

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

inline int check_dtype(int32_t dtype) {
  return dtype == TKV_DTYPE_F32 || dtype == TKV_DTYPE_BF16 ? TKV_OK : report(TKV_ERR_INVALID_ARG, "dtype");
}

inline int check_pool(PoolRef* p, const int8_t* pool, const float* scales, int64_t pool_pages, int32_t n_kv_heads,
                      int32_t head_dim, const int32_t* page_table, int32_t max_pages, const uint32_t* slot_mask) {
  if (n_kv_heads < 1 || n_kv_heads > 65535 || pool_pages < 1 || pool_pages > (int64_t(1) << 29) / n_kv_heads)
    return report(TKV_ERR_INVALID_ARG, "pool_pages x n_kv_heads must be 1 to 2^29");
  if (head_dim != 64 && head_dim != 128) return report(TKV_ERR_INVALID_ARG, "head_dim must be 64 or 128");
  if (max_pages < 1 || max_pages > kMaxSeqPages) return report(TKV_ERR_INVALID_ARG, "max_pages must be 1 to %d", kMaxSeqPages);
  if (!pool || !scales || !page_table) return report(TKV_ERR_INVALID_ARG, "null pointer");
  if (misaligned(pool, 16) || misaligned(scales, 8)) return report(TKV_ERR_INVALID_ARG, "pool must be 16-byte, scales 8-byte aligned");
  *p = {const_cast<int8_t*>(pool), const_cast<float*>(scales), pool_pages, page_table, max_pages, const_cast<uint32_t*>(slot_mask),
        n_kv_heads};
  return TKV_OK;
}

}  // namespace tkv
