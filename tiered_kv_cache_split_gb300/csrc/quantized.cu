// A paged cache held in 8 bits: tokens quantised as they are written, read back,
// and attended by one token per sequence.
//
// A BLOCK is the 16 slots of a page, one KV head, K or V: 16 rows of int8 codes
// and one fp32 scale; a row's value is code * scale. The pool is
// [pages][Hkv][2][16][D] codes, the scales [pages][Hkv][2].
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "tkv.h"
#include "tkv_internal.h"

namespace tkv {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyWarps = kCopyThreads / 32;
constexpr uint32_t kFullMask = 0xffffu;
constexpr float kNegInf = -INFINITY;

// Elements as they lie in a 16-byte vector.
template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int n = 4;
  using Codes = uint32_t;
  static __device__ __forceinline__ void unpack(const int4& v, float* x) {
    x[0] = __int_as_float(v.x); x[1] = __int_as_float(v.y); x[2] = __int_as_float(v.z); x[3] = __int_as_float(v.w);
  }
  static __device__ __forceinline__ int4 pack(const float* x) {
    return make_int4(__float_as_int(x[0]), __float_as_int(x[1]), __float_as_int(x[2]), __float_as_int(x[3]));
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  using Codes = uint2;
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

union CodeBytes {
  uint32_t w[2];
  int8_t c[8];
};
__device__ __forceinline__ CodeBytes load_codes(const uint32_t* at) { CodeBytes b; b.w[0] = *at; b.w[1] = 0; return b; }
__device__ __forceinline__ CodeBytes load_codes(const uint2* at) { const uint2 v = *at; CodeBytes b; b.w[0] = v.x; b.w[1] = v.y; return b; }
__device__ __forceinline__ void store_codes(uint32_t* at, const CodeBytes& b) { *at = b.w[0]; }
__device__ __forceinline__ void store_codes(uint2* at, const CodeBytes& b) { *at = make_uint2(b.w[0], b.w[1]); }

// The rows a call covers: slots [first, last) of each row, in items of one page.
struct RowRange {
  int32_t rows;
  int32_t first[kMaxBatch], last[kMaxBatch];
  int64_t page0[kMaxBatch + 1];  // prefix sums of the pages touched
  int64_t token0[kMaxBatch];     // packed index of slot `first`
};

struct PoolRef {
  int8_t* codes;
  float* scales;
  int64_t pages;
  const int32_t* table;
  int64_t table_stride;
  uint32_t* mask;         // may be null
  int32_t hkv;
};

struct Item {
  int row, h, kv;
  int slot0;        // first slot of the page in its row
  int lo, hi;       // slots of the page that the call covers
  int64_t id;       // page id, -1: outside the pool
  int64_t token;    // packed index of slot lo
};

// Item w of a call: K or V fastest, then the head, then the page, so that
// neighbouring warps take neighbouring pieces of the packed tokens and of a page.
__device__ __forceinline__ Item item_of(const RowRange& r, const PoolRef& p, int64_t w) {
  Item t;
  t.kv = static_cast<int>(w & 1);
  w >>= 1;
  t.h = static_cast<int>(w % p.hkv);
  w /= p.hkv;
  int lo = 0, hi = r.rows - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (r.page0[mid] <= w) lo = mid; else hi = mid - 1;
  }
  t.row = lo;
  const int page = r.first[lo] / kPage + static_cast<int>(w - r.page0[lo]);
  t.slot0 = page * kPage;
  t.lo = max(r.first[lo] - t.slot0, 0);
  t.hi = min(r.last[lo] - t.slot0, kPage);
  t.token = r.token0[lo] + t.slot0 + t.lo - r.first[lo];
  const int32_t id = p.table[lo * p.table_stride + page];
  t.id = id < 0 || id >= p.pages ? -1 : id;
  return t;
}

// ---- append

struct AppendQParams {
  RowRange r;
  PoolRef p;
  const void *k, *v;
  int64_t k_stride, v_stride;
  const int32_t* refs;  // may be null
  int32_t* status;      // may be null
  int64_t items;
};

__device__ __forceinline__ int8_t to_code(float x, float scale) {
  const float c = rintf(x / scale);
  return static_cast<int8_t>(fminf(fmaxf(c, -127.f), 127.f));
}

// A warp per block: the rows of the block that are written stay in registers
// between the maximum and the codes, so K and V are read once. Of a block that
// holds earlier tokens the scale only grows; where it does, their codes are
// scaled to it.
template <typename T, int D>
__global__ void __launch_bounds__(kCopyThreads) append_quantized_kernel(const __grid_constant__ AppendQParams p) {
  using V = Vec<T>;
  using Codes = typename V::Codes;
  constexpr int kLanes = D / V::n;                       // lanes of a row
  constexpr int kRows = 32 / kLanes, kPasses = kPage / kRows;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5);
  if (w >= p.items) return;
  const int lane = threadIdx.x & 31, r0 = lane / kLanes, c0 = (lane % kLanes) * V::n;
  const Item t = item_of(p.r, p.p, w);
  if (t.id < 0 || (p.refs && p.refs[t.id] != 1)) {
    if (lane == 0 && p.status) *p.status = -1;
    return;
  }
  const T* from = static_cast<const T*>(t.kv ? p.v : p.k) + t.h * D + c0;
  const int64_t stride = t.kv ? p.v_stride : p.k_stride;
  int4 x[kPasses];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int s = i * kRows + r0;
    x[i] = make_int4(0, 0, 0, 0);
    if (s >= t.lo && s < t.hi) x[i] = *reinterpret_cast<const int4*>(from + (t.token + s - t.lo) * stride);
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    float f[V::n];
    V::unpack(x[i], f);
#pragma unroll
    for (int j = 0; j < V::n; ++j) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);  // a NaN is above infinity
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const int64_t block = (t.id * p.p.hkv + t.h) * 2 + t.kv;
  const float old = t.lo > 0 ? p.p.scales[block] : 0.f;
  const float mine = __uint_as_float(top) / 127.f;
  const float grown = mine > old || mine != mine ? mine : old;  // a NaN stays
  const bool finite = grown < INFINITY;
  const float scale = finite ? grown : NAN;                     // every value of the block reads as NaN
  int8_t* codes = p.p.codes + block * kPage * D + c0;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int s = i * kRows + r0;
    if (s >= t.lo && s < t.hi) {
      float f[V::n];
      V::unpack(x[i], f);
      CodeBytes b;
#pragma unroll
      for (int j = 0; j < V::n; ++j) b.c[j] = finite && scale > 0.f ? to_code(f[j], scale) : 0;
      store_codes(reinterpret_cast<Codes*>(codes + s * D), b);
    }
  }
  if (t.lo > 0 && scale > old && finite) {
    const float ratio = old / scale;
    for (int s = r0; s < t.lo; s += kRows) {
      Codes* at = reinterpret_cast<Codes*>(codes + s * D);
      CodeBytes b = load_codes(at);
#pragma unroll
      for (int j = 0; j < V::n; ++j) b.c[j] = static_cast<int8_t>(rintf(b.c[j] * ratio));
      store_codes(at, b);
    }
  }
  __syncwarp();
  if (lane == 0) {
    p.p.scales[block] = scale;
    if (p.p.mask && t.h == 0 && t.kv == 0) {
      const uint32_t bits = (1u << t.hi) - (1u << t.lo);
      p.p.mask[t.id] = t.lo > 0 ? p.p.mask[t.id] | bits : bits;
    }
  }
}

// ---- read

struct ReadQParams {
  RowRange r;
  PoolRef p;
  void *k, *v;
  int64_t k_stride, v_stride;
  int64_t items;
};

// A warp per block, as the append's.
template <typename T, int D>
__global__ void __launch_bounds__(kCopyThreads) read_quantized_kernel(const __grid_constant__ ReadQParams p) {
  using V = Vec<T>;
  using Codes = typename V::Codes;
  constexpr int kLanes = D / V::n;
  constexpr int kRows = 32 / kLanes, kPasses = kPage / kRows;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5);
  if (w >= p.items) return;
  const int lane = threadIdx.x & 31, r0 = lane / kLanes, c0 = (lane % kLanes) * V::n;
  const Item t = item_of(p.r, p.p, w);
  const uint32_t live = t.id < 0 ? 0 : p.p.mask ? p.p.mask[t.id] : kFullMask;
  const int64_t block = (max(t.id, int64_t(0)) * p.p.hkv + t.h) * 2 + t.kv;
  const float scale = t.id < 0 ? 0.f : p.p.scales[block];
  const int8_t* codes = p.p.codes + block * kPage * D + c0;
  T* to = static_cast<T*>(t.kv ? p.v : p.k) + t.h * D + c0;
  const int64_t stride = t.kv ? p.v_stride : p.k_stride;
  CodeBytes b[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int s = i * kRows + r0;
    b[i].w[0] = b[i].w[1] = 0;
    if (s >= t.lo && s < t.hi && (live >> s & 1)) b[i] = load_codes(reinterpret_cast<const Codes*>(codes + s * D));
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int s = i * kRows + r0;
    if (s < t.lo || s >= t.hi) continue;
    float f[V::n];
#pragma unroll
    for (int j = 0; j < V::n; ++j) f[j] = live >> s & 1 ? b[i].c[j] * scale : 0.f;
    *reinterpret_cast<int4*>(to + (t.token + s - t.lo) * stride) = V::pack(f);
  }
}

// ---- attention

struct AttendQParams {
  PoolRef p;
  const void* q;
  void* out;
  float* alpha;          // may be null
  float2* stats;         // [B][Hq] running maximum (base 2) and sum
  int32_t B, Hq, G, max_pages;
  float qscale;          // log2(e) / sqrt(D)
  int32_t count[kMaxBatch];
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* at, float x) { *at = x; }
__device__ __forceinline__ void put(__nv_bfloat16* at, float x) { *at = __float2bfloat16_rn(x); }

__device__ __forceinline__ float finite_or_nan(float x) { return fabsf(x) < INFINITY ? x : NAN; }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// A warp per (sequence, query head): keys one after another, D / 32 elements per lane.
template <typename T, int D>
__global__ void __launch_bounds__(128) attend_quantized_kernel(const __grid_constant__ AttendQParams p) {
  constexpr int E = D / 32;
  const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (w >= p.B * p.Hq) return;
  const int b = w / p.Hq, hq = w % p.Hq, h = hq / p.G;
  float q[E], o[E] = {};
#pragma unroll
  for (int j = 0; j < E; ++j) q[j] = to_float(static_cast<const T*>(p.q)[static_cast<int64_t>(w) * D + lane * E + j]);
  float m = kNegInf, z = 0.f;
  for (int i = 0; i < p.count[b]; ++i) {
    const int32_t id = p.p.table[b * p.p.table_stride + i];
    if (id < 0 || id >= p.p.pages) continue;
    const uint32_t live = p.p.mask[id];
    const int64_t block = (static_cast<int64_t>(id) * p.p.hkv + h) * 2;
    const float sk = finite_or_nan(p.p.scales[block]), sv = finite_or_nan(p.p.scales[block + 1]);
    for (int s = 0; s < kPage; ++s) {
      if (!(live >> s & 1)) continue;
      const int8_t* k = p.p.codes + (block * kPage + s) * D + lane * E;
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j) dot += q[j] * k[j];
      const float l = warp_sum(dot) * sk * p.qscale;
      if (l == kNegInf) continue;
      const float top = fmaxf(m, l), keep = exp2f(m - top), x = exp2f(l - top);
      const float before = z * keep;
      z = before + x;
      const float wo = before / z, wx = x / z;  // a mean at every key: sums of V could pass the type's largest value
#pragma unroll
      for (int j = 0; j < E; ++j) o[j] = o[j] * wo + wx * (k[kPage * D + j] * sv);
      m = top;
    }
  }
#pragma unroll
  for (int j = 0; j < E; ++j) put(static_cast<T*>(p.out) + static_cast<int64_t>(w) * D + lane * E + j, o[j]);
  if (p.stats && lane == 0) p.stats[w] = make_float2(m, z);
}

// A warp per (sequence, KV head, page): the weights of its slots, summed over the heads.
template <typename T, int D>
__global__ void __launch_bounds__(128) alpha_quantized_kernel(const __grid_constant__ AttendQParams p) {
  constexpr int E = D / 32;
  const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int i = w % p.max_pages, h = w / p.max_pages % p.p.hkv, b = w / p.max_pages / p.p.hkv;
  if (b >= p.B || i >= p.count[b]) return;
  const int32_t id = p.p.table[b * p.p.table_stride + i];
  if (id < 0 || id >= p.p.pages) return;
  const uint32_t live = p.p.mask[id];
  const int64_t block = (static_cast<int64_t>(id) * p.p.hkv + h) * 2;
  const float sk = finite_or_nan(p.p.scales[block]);
  float* to = p.alpha + (static_cast<int64_t>(b) * p.p.hkv + h) * p.max_pages * kPage + i * kPage;
  for (int s = 0; s < kPage; ++s) {
    if (!(live >> s & 1)) continue;
    const int8_t* k = p.p.codes + (block * kPage + s) * D + lane * E;
    float sum = 0.f;
    for (int g = 0; g < p.G; ++g) {
      const T* q = static_cast<const T*>(p.q) + (static_cast<int64_t>(b) * p.Hq + h * p.G + g) * D + lane * E;
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j) dot += to_float(q[j]) * k[j];
      const float l = warp_sum(dot) * sk * p.qscale;
      const float2 st = p.stats[b * p.Hq + h * p.G + g];
      sum += l == kNegInf ? 0.f : exp2f(l - st.x) / st.y;
    }
    if (lane == 0) to[s] += sum;
  }
}

// ---- host side

bool misaligned(const void* ptr, size_t to) { return reinterpret_cast<uintptr_t>(ptr) % to != 0; }

int launched(const char* what, cudaError_t e) {
  return e == cudaSuccess ? TKV_OK : report(TKV_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
}

int check_pool(PoolRef* p, int8_t* pool, float* scales, int64_t pool_pages, int32_t n_kv_heads, int32_t head_dim,
               const int32_t* page_table, int32_t max_pages, uint32_t* slot_mask) {
  if (n_kv_heads < 1 || n_kv_heads > 65535 || pool_pages < 1 || pool_pages > (int64_t(1) << 29) / n_kv_heads)
    return report(TKV_ERR_INVALID_ARG, "pool_pages x n_kv_heads must be 1 to 2^29");
  if (head_dim != 64 && head_dim != 128) return report(TKV_ERR_INVALID_ARG, "head_dim must be 64 or 128");
  if (max_pages < 1 || max_pages > kMaxSeqPages) return report(TKV_ERR_INVALID_ARG, "max_pages must be 1 to %d", kMaxSeqPages);
  if (!pool || !scales || !page_table) return report(TKV_ERR_INVALID_ARG, "null pointer");
  if (misaligned(pool, 16) || misaligned(scales, 8)) return report(TKV_ERR_INVALID_ARG, "pool must be 16-byte, scales 8-byte aligned");
  *p = {pool, scales, pool_pages, page_table, max_pages, slot_mask, n_kv_heads};
  return TKV_OK;
}

// Fills the ranges [first, last) of each row; *tokens, *pages their sums.
int check_rows(RowRange* r, int32_t rows, const int32_t* first, const int32_t* last, int32_t max_pages, int64_t* tokens) {
  *tokens = 0;
  r->rows = rows;
  r->page0[0] = 0;
  for (int i = 0; i < rows; ++i) {
    r->first[i] = first[i];
    r->last[i] = last[i];
    r->token0[i] = *tokens;
    *tokens += last[i] - first[i];
    r->page0[i + 1] = r->page0[i] + (last[i] > first[i] ? (last[i] + kPage - 1) / kPage - first[i] / kPage : 0);
    if (last[i] > max_pages * kPage) return report(TKV_ERR_INVALID_ARG, "row %d: more tokens than its max_pages hold", i);
  }
  return TKV_OK;
}

int check_tokens(int32_t dtype, int32_t n_kv_heads, int32_t head_dim, const void* k, int64_t k_stride, const void* v, int64_t v_stride) {
  if (!k || !v) return report(TKV_ERR_INVALID_ARG, "null pointer");
  const int64_t row = static_cast<int64_t>(n_kv_heads) * head_dim, unit = dtype == TKV_DTYPE_BF16 ? 8 : 4;
  if (misaligned(k, 16) || misaligned(v, 16)) return report(TKV_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  if (k_stride < row || v_stride < row || k_stride % unit || v_stride % unit || (k_stride | v_stride) >> 36)
    return report(TKV_ERR_INVALID_ARG, "token strides must hold a token and be multiples of 16 bytes");
  return TKV_OK;
}

int check_dtype(int32_t dtype) {
  return dtype == TKV_DTYPE_F32 || dtype == TKV_DTYPE_BF16 ? TKV_OK : report(TKV_ERR_INVALID_ARG, "dtype");
}

int check_heads(int32_t Hq, int32_t Hkv, int32_t D) {
  if (Hkv < 1 || Hq < 1 || Hkv > 65535 || Hq % Hkv || Hq / Hkv > 64)
    return report(TKV_ERR_INVALID_ARG, "n_q_heads must be 1 to 64 times n_kv_heads");
  if (D != 64 && D != 128) return report(TKV_ERR_INVALID_ARG, "head_dim must be 64 or 128");
  return TKV_OK;
}

int plan_attend(AttendQParams* p, int32_t batch, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype, const int32_t* page_counts,
                int32_t max_pages, int want_alpha, size_t* bytes) {
  if (batch < 1 || batch > kMaxBatch) return report(TKV_ERR_INVALID_ARG, "batch must be 1 to %d", kMaxBatch);
  if (int st = check_heads(Hq, Hkv, D)) return st;
  if (int st = check_dtype(dtype)) return st;
  if (max_pages < 1 || max_pages > kMaxSeqPages) return report(TKV_ERR_INVALID_ARG, "max_pages must be 1 to %d", kMaxSeqPages);
  if (!page_counts) return report(TKV_ERR_INVALID_ARG, "null pointer");
  for (int b = 0; b < batch; ++b) {
    if (page_counts[b] < 0 || page_counts[b] > max_pages) return report(TKV_ERR_INVALID_ARG, "page_counts[%d] out of 0..max_pages", b);
    p->count[b] = page_counts[b];
  }
  p->B = batch; p->Hq = Hq; p->G = Hq / Hkv; p->max_pages = max_pages;
  p->qscale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
  *bytes = want_alpha ? (static_cast<size_t>(batch) * Hq * sizeof(float2) + 255) / 256 * 256 : 0;
  return TKV_OK;
}

template <typename T, int D>
cudaError_t launch_attend(const AttendQParams& p, cudaStream_t s) {
  attend_quantized_kernel<T, D><<<(p.B * p.Hq + 3) / 4, 128, 0, s>>>(p);
  if (p.alpha) alpha_quantized_kernel<T, D><<<static_cast<unsigned>((static_cast<int64_t>(p.B) * p.p.hkv * p.max_pages + 3) / 4), 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace tkv

using namespace tkv;

extern "C" {

tkv_status tkv_append_quantized(int32_t rows, const int32_t* lens, const int32_t* new_lens, int32_t n_kv_heads,
                                int32_t head_dim, int32_t dtype, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, int8_t* pool, float* scales, int64_t pool_pages,
                                const int32_t* page_table, int32_t max_pages, uint32_t* slot_mask,
                                const int32_t* page_refs, int32_t* status, tkv_stream stream) {
  if (rows < 1 || rows > kMaxBatch) return tkv_status(report(TKV_ERR_INVALID_ARG, "rows must be 1 to %d", kMaxBatch));
  AppendQParams p{};
  if (int st = check_dtype(dtype)) return tkv_status(st);
  if (int st = check_pool(&p.p, pool, scales, pool_pages, n_kv_heads, head_dim, page_table, max_pages, slot_mask)) return tkv_status(st);
  if (!lens || !new_lens) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  int32_t ends[kMaxBatch];
  for (int i = 0; i < rows; ++i) {
    if (lens[i] < 0 || new_lens[i] < 0 || lens[i] > INT32_MAX - new_lens[i])
      return tkv_status(report(TKV_ERR_INVALID_ARG, "row %d: lens and new_lens must be at least 0", i));
    ends[i] = lens[i] + new_lens[i];
  }
  int64_t tokens;
  if (int st = check_rows(&p.r, rows, lens, ends, max_pages, &tokens)) return tkv_status(st);
  if (tokens == 0) return TKV_OK;
  if (int st = check_tokens(dtype, n_kv_heads, head_dim, k, k_stride, v, v_stride)) return tkv_status(st);
  p.k = k; p.v = v; p.k_stride = k_stride; p.v_stride = v_stride;
  p.refs = page_refs; p.status = status;
  p.items = p.r.page0[rows] * n_kv_heads * 2;
  const int64_t ctas = (p.items + kCopyWarps - 1) / kCopyWarps;
  if (ctas > INT32_MAX) return tkv_status(report(TKV_ERR_INVALID_ARG, "too many blocks in one call"));
  const unsigned n = static_cast<unsigned>(ctas);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == TKV_DTYPE_BF16) {
    if (head_dim == 64) append_quantized_kernel<__nv_bfloat16, 64><<<n, kCopyThreads, 0, s>>>(p);
    else append_quantized_kernel<__nv_bfloat16, 128><<<n, kCopyThreads, 0, s>>>(p);
  } else {
    if (head_dim == 64) append_quantized_kernel<float, 64><<<n, kCopyThreads, 0, s>>>(p);
    else append_quantized_kernel<float, 128><<<n, kCopyThreads, 0, s>>>(p);
  }
  return tkv_status(launched("quantised append", cudaGetLastError()));
}

tkv_status tkv_read_quantized(int32_t rows, const int32_t* first, const int32_t* lens, int32_t n_kv_heads,
                              int32_t head_dim, int32_t dtype, const int8_t* pool, const float* scales,
                              int64_t pool_pages, const int32_t* page_table, int32_t max_pages,
                              const uint32_t* slot_mask, void* k, int64_t k_stride, void* v, int64_t v_stride,
                              tkv_stream stream) {
  if (rows < 1 || rows > kMaxBatch) return tkv_status(report(TKV_ERR_INVALID_ARG, "rows must be 1 to %d", kMaxBatch));
  ReadQParams p{};
  if (int st = check_dtype(dtype)) return tkv_status(st);
  if (int st = check_pool(&p.p, const_cast<int8_t*>(pool), const_cast<float*>(scales), pool_pages, n_kv_heads, head_dim, page_table,
                          max_pages, const_cast<uint32_t*>(slot_mask)))
    return tkv_status(st);
  if (!first || !lens) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  for (int i = 0; i < rows; ++i)
    if (first[i] < 0 || lens[i] < first[i]) return tkv_status(report(TKV_ERR_INVALID_ARG, "row %d: 0 <= first <= len", i));
  int64_t tokens;
  if (int st = check_rows(&p.r, rows, first, lens, max_pages, &tokens)) return tkv_status(st);
  if (tokens == 0) return TKV_OK;
  if (int st = check_tokens(dtype, n_kv_heads, head_dim, k, k_stride, v, v_stride)) return tkv_status(st);
  p.k = k; p.v = v; p.k_stride = k_stride; p.v_stride = v_stride;
  p.items = p.r.page0[rows] * n_kv_heads * 2;
  const int64_t ctas = (p.items + kCopyWarps - 1) / kCopyWarps;
  if (ctas > INT32_MAX) return tkv_status(report(TKV_ERR_INVALID_ARG, "too many blocks in one call"));
  const unsigned n = static_cast<unsigned>(ctas);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == TKV_DTYPE_BF16) {
    if (head_dim == 64) read_quantized_kernel<__nv_bfloat16, 64><<<n, kCopyThreads, 0, s>>>(p);
    else read_quantized_kernel<__nv_bfloat16, 128><<<n, kCopyThreads, 0, s>>>(p);
  } else {
    if (head_dim == 64) read_quantized_kernel<float, 64><<<n, kCopyThreads, 0, s>>>(p);
    else read_quantized_kernel<float, 128><<<n, kCopyThreads, 0, s>>>(p);
  }
  return tkv_status(launched("quantised read", cudaGetLastError()));
}

tkv_status tkv_quantized_attention_scratch_size(int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                                int32_t dtype, const int32_t* page_counts, int32_t max_pages,
                                                int32_t want_alpha, size_t* scratch_bytes) {
  if (!scratch_bytes) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  AttendQParams p{};
  return tkv_status(plan_attend(&p, batch, n_q_heads, n_kv_heads, head_dim, dtype, page_counts, max_pages, want_alpha, scratch_bytes));
}

tkv_status tkv_quantized_attention(int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t dtype,
                                   const void* q, const int8_t* pool, const float* scales, int64_t pool_pages,
                                   const int32_t* page_table, const uint32_t* slot_mask, const int32_t* page_counts,
                                   int32_t max_pages, void* out, float* alpha_sum, void* scratch, size_t scratch_bytes,
                                   tkv_stream stream) {
  AttendQParams p{};
  size_t need;
  if (int st = plan_attend(&p, batch, n_q_heads, n_kv_heads, head_dim, dtype, page_counts, max_pages, alpha_sum != nullptr, &need))
    return tkv_status(st);
  if (int st = check_pool(&p.p, const_cast<int8_t*>(pool), const_cast<float*>(scales), pool_pages, n_kv_heads, head_dim, page_table,
                          max_pages, const_cast<uint32_t*>(slot_mask)))
    return tkv_status(st);
  if (!q || !out || !slot_mask) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  if (misaligned(q, 16) || misaligned(out, 16) || misaligned(alpha_sum, 16))
    return tkv_status(report(TKV_ERR_INVALID_ARG, "q, out and alpha_sum must be 16-byte aligned"));
  if (need) {
    if (!scratch) return tkv_status(report(TKV_ERR_INVALID_ARG, "null scratch: need %zu bytes", need));
    if (scratch_bytes < need) return tkv_status(report(TKV_ERR_CAPACITY, "scratch too small: need %zu bytes", need));
    if (misaligned(scratch, 256)) return tkv_status(report(TKV_ERR_INVALID_ARG, "scratch not 256-byte aligned"));
  }
  p.q = q; p.out = out; p.alpha = alpha_sum;
  p.stats = need ? static_cast<float2*>(scratch) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == TKV_DTYPE_BF16) e = head_dim == 64 ? launch_attend<__nv_bfloat16, 64>(p, s) : launch_attend<__nv_bfloat16, 128>(p, s);
  else e = head_dim == 64 ? launch_attend<float, 64>(p, s) : launch_attend<float, 128>(p, s);
  return tkv_status(launched("quantised attention", e));
}

}  // extern "C"
