// A paged cache held in 8 bits: tokens quantised as they are written, and read
// back (quantized.h has the layout).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "quantized.h"

namespace tkv {
namespace {

constexpr int kCopyThreads = 128;
constexpr int kCopyWarps = kCopyThreads / 32;

// int8 codes of the elements of a 16-byte vector
template <typename T> struct CodesOf;
template <> struct CodesOf<float> { using type = uint32_t; };
template <> struct CodesOf<__nv_bfloat16> { using type = uint2; };
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
  int32_t page0[kMaxBatch + 1];  // prefix sums of the pages touched
  int64_t token0[kMaxBatch];     // packed index of slot `first`
};

struct Item {
  int h, kv;
  int slot0;        // first slot of the page in its row
  int lo, hi;       // slots of the page that the call covers
  int64_t id;       // page id, -1: outside the pool
  int64_t token;    // packed index of slot lo
};

// Item w of a call: K or V fastest, then the head, then the page, so that
// neighbouring warps take neighbouring pieces of the packed tokens and of a page.
__device__ __forceinline__ Item item_of(const RowRange& r, const PoolRef& p, uint32_t w) {
  Item t;
  t.kv = static_cast<int>(w & 1);
  w >>= 1;
  const uint32_t heads = p.hkv;
  t.h = static_cast<int>(w % heads);
  w /= heads;
  int lo = 0, hi = r.rows - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (r.page0[mid] <= static_cast<int32_t>(w)) lo = mid; else hi = mid - 1;
  }
  const int page = r.first[lo] / kPage + static_cast<int>(w) - r.page0[lo];
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
  uint32_t items;
};

// Absolute bits of the largest element of a vector; a NaN is above infinity.
__device__ __forceinline__ uint32_t top_bits(const int4& v, float) {
  const uint32_t m = 0x7fffffffu;
  return max(max(v.x & m, v.y & m), max(v.z & m, v.w & m));
}
__device__ __forceinline__ uint32_t top_bits(const int4& v, __nv_bfloat16) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t w = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
  return max(w << 16, w & 0xffff0000u);
}

// Two fp32 operations at a time.
struct Two {
  float x, y;
};
__device__ __forceinline__ unsigned long long bits(Two v) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ Two two(unsigned long long v) {
  Two r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return two(r);
}

// Codes rint(x / scale) of a vector, the quotient correctly rounded without a division
// (Markstein 1990): a quotient by the correctly rounded reciprocal, once corrected by
// its residual, is next to x / scale, and once more is x / scale rounded. That holds
// while nothing underflows: kLeastScale keeps residuals of quotients from 1/4 up in
// range, and smaller ones give code 0 whatever their error. Adding 1.5 * 2^23 rounds to a whole number
// and leaves it in the low byte. Divisions were half of the time; a reciprocal
// alone would need them wherever a quotient is near a border, which in bf16 the
// elements of half the largest one always are.
constexpr float kLeastScale = 0x1p-60f;
template <int N>
__device__ __forceinline__ CodeBytes to_codes(const float (&x)[N], float scale, float inverse) {
  const Two inv = {inverse, inverse}, minus = {-scale, -scale}, zero = {-0.f, -0.f}, one = {1.f, 1.f}, round = {0x1.8p23f, 0x1.8p23f};
  CodeBytes b;
  b.w[0] = b.w[1] = 0;
  uint32_t t[N];
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const Two a = {x[j], x[j + 1]};
    Two q = fma2(a, inv, zero);
    q = fma2(fma2(q, minus, a), inv, q);
    q = fma2(fma2(q, minus, a), inv, q);
    q = fma2(q, one, round);
    t[j] = __float_as_uint(q.x);
    t[j + 1] = __float_as_uint(q.y);
  }
#pragma unroll
  for (int j = 0; j < N; j += 4)
    b.w[j / 4] = __byte_perm(__byte_perm(t[j], t[j + 1], 0x0040), __byte_perm(t[j + 2], t[j + 3], 0x0040), 0x5410);
  return b;
}

// A warp per block: the rows of the block that are written stay in registers
// between the maximum and the codes, so K and V are read once; they are on their
// way before the page id is here. Of a block that holds earlier tokens the scale only
// grows in size; where it does, their codes are scaled to it. HBM bounds the large calls: 40959
// tokens of 8 heads at d 128 in bf16 (168 MB in, 84 out) take 44 us, 5.7 TB/s, the
// issue slots being 51 % busy; 20479 tokens in fp32 36 us, 5.8 TB/s; the least call 4 us, and
// 4 more for a token in each of 64 rows whose blocks' scales all grow.
template <typename T, int D>
__global__ void __launch_bounds__(kCopyThreads) append_quantized_kernel(const __grid_constant__ AppendQParams p) {
  using V = Vec<T>;
  using Codes = typename CodesOf<T>::type;
  constexpr int kLanes = D / V::n;                       // lanes of a row
  constexpr int kRows = 32 / kLanes, kPasses = kPage / kRows;
  cudaGridDependencySynchronize();
  const uint32_t w = blockIdx.x * kCopyWarps + (threadIdx.x >> 5);
  if (w >= p.items) return;
  const int lane = threadIdx.x & 31, r0 = lane / kLanes, c0 = (lane % kLanes) * V::n;
  const Item t = item_of(p.r, p.p, w);
  const T* from = static_cast<const T*>(t.kv ? p.v : p.k) + (t.token + r0 - t.lo) * (t.kv ? p.v_stride : p.k_stride) + t.h * D + c0;
  const int64_t stride = (t.kv ? p.v_stride : p.k_stride) * kRows;  // of a pass
  const bool whole = t.lo == 0 && t.hi == kPage;
  auto written = [&](int i) { return i * kRows + r0 >= t.lo && i * kRows + r0 < t.hi; };
  int4 x[kPasses];
  uint32_t top = 0;
  if (whole) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) x[i] = *reinterpret_cast<const int4*>(from + i * stride);
  } else {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      x[i] = make_int4(0, 0, 0, 0);
      if (written(i)) x[i] = *reinterpret_cast<const int4*>(from + i * stride);
    }
  }
  if (t.id < 0 || (p.refs && p.refs[t.id] != 1)) {
    if (lane == 0 && p.status) *p.status = -1;
    return;
  }
  const int64_t block = (t.id * p.p.hkv + t.h) * 2 + t.kv;
  const float old = t.lo > 0 ? p.p.scales[block] : 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) top = max(top, top_bits(x[i], T()));
  top = __reduce_max_sync(0xffffffffu, top);
  const float mine = __uint_as_float(top) / 127.f;
  const bool grows = mine > fabsf(old);                         // a caller's pool may hold scales below 0
  const float grown = grows || mine != mine ? mine : old;       // a NaN stays
  const bool finite = fabsf(grown) < INFINITY;
  const float scale = finite ? grown : NAN;                     // every value of the block reads as NaN
  int8_t* codes = p.p.codes + block * kPage * D + c0;
  const float inverse = 1.f / scale;
  auto store = [&](int i) {
    float f[V::n];
    V::unpack(x[i], f);
    CodeBytes b = to_codes(f, scale, inverse);
    if (!finite) b.w[0] = b.w[1] = 0;
    store_codes(reinterpret_cast<Codes*>(codes + (i * kRows + r0) * D), b);
  };
  if (fabsf(scale) < kLeastScale) {
    // by division, whose quotients pass 127 where the scale itself was rounded down
#pragma unroll 1
    for (int i = 0; i < kPasses; ++i)
#pragma unroll 1
      for (int j = 0; j < V::n && written(i); ++j)
        codes[(i * kRows + r0) * D + j] = scale != 0.f ? static_cast<int8_t>(fminf(fmaxf(rintf(to_float(from[i * stride + j]) / scale), -127.f), 127.f)) : 0;
  } else if (whole) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) store(i);
  } else {
    // a token or two of a decode step: most passes have none (a branch of the warp)
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      if ((i + 1) * kRows > t.lo && i * kRows < t.hi && written(i)) store(i);
  }
  if (t.lo > 0 && grows && finite) {
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
  uint32_t items;
};

// A warp per block, as the append's. 28296 tokens of 8 heads at d 128 to bf16 (58 MB in,
// 116 out) take 31 us with inputs past the L2, 5.6 TB/s, and 28 in a row of calls on the same
// ones; to fp32 50 us, 5.8 TB/s.
template <typename T, int D>
__global__ void __launch_bounds__(kCopyThreads) read_quantized_kernel(const __grid_constant__ ReadQParams p) {
  using V = Vec<T>;
  using Codes = typename CodesOf<T>::type;
  constexpr int kLanes = D / V::n;
  constexpr int kRows = 32 / kLanes, kPasses = kPage / kRows;
  cudaGridDependencySynchronize();
  const uint32_t w = blockIdx.x * kCopyWarps + (threadIdx.x >> 5);
  if (w >= p.items) return;
  const int lane = threadIdx.x & 31, r0 = lane / kLanes, c0 = (lane % kLanes) * V::n;
  const Item t = item_of(p.r, p.p, w);
  const uint32_t live = t.id < 0 ? 0 : p.p.mask ? p.p.mask[t.id] : kFullMask;
  const int64_t block = (max(t.id, int64_t(0)) * p.p.hkv + t.h) * 2 + t.kv;
  const float scale = t.id < 0 ? 0.f : p.p.scales[block];
  const int8_t* codes = p.p.codes + block * kPage * D + c0;
  T* to = static_cast<T*>(t.kv ? p.v : p.k) + t.h * D + c0;
  const int64_t stride = t.kv ? p.v_stride : p.k_stride;
  Codes c[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int s = i * kRows + r0;
    c[i] = Codes{};
    if (s >= t.lo && s < t.hi && (live >> s & 1)) c[i] = *reinterpret_cast<const Codes*>(codes + s * D);
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int s = i * kRows + r0;
    if (s < t.lo || s >= t.hi) continue;
    const float by = live >> s & 1 ? scale : 0.f;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&c[i]);
    float f[V::n];
#pragma unroll
    for (int j = 0; j < V::n; ++j) f[j] = static_cast<float>(static_cast<int8_t>(w[j / 4] >> (8 * (j % 4)))) * by;
    *reinterpret_cast<int4*>(to + (t.token + s - t.lo) * stride) = V::pack(f);
  }
}

// ---- host side

// Fills the ranges [first, last) of each row; *tokens is their sum.
int check_rows(RowRange* r, int32_t rows, const int32_t* first, const int32_t* last, int32_t max_pages, int64_t* tokens) {
  *tokens = 0;
  r->rows = rows;
  r->page0[0] = 0;
  for (int i = 0; i < rows; ++i) {
    if (last[i] > max_pages * kPage) return report(TKV_ERR_INVALID_ARG, "row %d: more tokens than its max_pages hold", i);
    r->first[i] = first[i];
    r->last[i] = last[i];
    r->token0[i] = *tokens;
    *tokens += last[i] - first[i];
    r->page0[i + 1] = r->page0[i] + (last[i] > first[i] ? (last[i] + kPage - 1) / kPage - first[i] / kPage : 0);
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
  const int64_t items = static_cast<int64_t>(p.r.page0[rows]) * n_kv_heads * 2;
  if (items > INT32_MAX) return tkv_status(report(TKV_ERR_INVALID_ARG, "more than 2^31 blocks in one call"));
  p.items = static_cast<uint32_t>(items);
  const unsigned n = (p.items + kCopyWarps - 1) / kCopyWarps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void (*const kernel)(AppendQParams) = dtype == TKV_DTYPE_BF16 ? (head_dim == 64 ? append_quantized_kernel<__nv_bfloat16, 64> : append_quantized_kernel<__nv_bfloat16, 128>)
                                                         : (head_dim == 64 ? append_quantized_kernel<float, 64> : append_quantized_kernel<float, 128>);
  return tkv_status(launched("quantised append", launch_early(kernel, dim3(n), kCopyThreads, 0, s, 1, p)));
}

tkv_status tkv_read_quantized(int32_t rows, const int32_t* first, const int32_t* lens, int32_t n_kv_heads,
                              int32_t head_dim, int32_t dtype, const int8_t* pool, const float* scales,
                              int64_t pool_pages, const int32_t* page_table, int32_t max_pages,
                              const uint32_t* slot_mask, void* k, int64_t k_stride, void* v, int64_t v_stride,
                              tkv_stream stream) {
  if (rows < 1 || rows > kMaxBatch) return tkv_status(report(TKV_ERR_INVALID_ARG, "rows must be 1 to %d", kMaxBatch));
  ReadQParams p{};
  if (int st = check_dtype(dtype)) return tkv_status(st);
  if (int st = check_pool(&p.p, pool, scales, pool_pages, n_kv_heads, head_dim, page_table, max_pages, slot_mask))
    return tkv_status(st);
  if (!first || !lens) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  for (int i = 0; i < rows; ++i)
    if (first[i] < 0 || lens[i] < first[i]) return tkv_status(report(TKV_ERR_INVALID_ARG, "row %d: 0 <= first <= len", i));
  int64_t tokens;
  if (int st = check_rows(&p.r, rows, first, lens, max_pages, &tokens)) return tkv_status(st);
  if (tokens == 0) return TKV_OK;
  if (int st = check_tokens(dtype, n_kv_heads, head_dim, k, k_stride, v, v_stride)) return tkv_status(st);
  if (k == v) return tkv_status(report(TKV_ERR_INVALID_ARG, "k and v are the same"));
  p.k = k; p.v = v; p.k_stride = k_stride; p.v_stride = v_stride;
  const int64_t items = static_cast<int64_t>(p.r.page0[rows]) * n_kv_heads * 2;
  if (items > INT32_MAX) return tkv_status(report(TKV_ERR_INVALID_ARG, "more than 2^31 blocks in one call"));
  p.items = static_cast<uint32_t>(items);
  const unsigned n = (p.items + kCopyWarps - 1) / kCopyWarps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void (*const kernel)(ReadQParams) = dtype == TKV_DTYPE_BF16 ? (head_dim == 64 ? read_quantized_kernel<__nv_bfloat16, 64> : read_quantized_kernel<__nv_bfloat16, 128>)
                                                         : (head_dim == 64 ? read_quantized_kernel<float, 64> : read_quantized_kernel<float, 128>);
  return tkv_status(launched("quantised read", launch_early(kernel, dim3(n), kCopyThreads, 0, s, 1, p)));
}

}  // extern "C"
