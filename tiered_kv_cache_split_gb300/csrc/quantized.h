// Shared by the operators of a paged cache held in 8 bits.
//
// A BLOCK is the 16 slots of a page, one KV head, K or V: 16 rows of int8 codes
// and one fp32 scale; a row's value is code * scale. The pool is
// [pages][Hkv][2][16][D] codes, the scales [pages][Hkv][2].
#pragma once

#include <cstdint>

#include "elements.h"

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
