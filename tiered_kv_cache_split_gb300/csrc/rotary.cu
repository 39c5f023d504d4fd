// Rotary positions: pair (a, b) of a head at position pos turns by the angle
// t = pos * f of its frequency f,
//   a' = scale (a cos t - b sin t),  b' = scale (b cos t + a sin t).
//
// The angle is formed in integers. A frequency is held as turns per position in
// 64-bit fixed point (step = f / 2 pi * 2^64), so pos * step mod 2^64 is the
// phase, exact however far the position: an angle in fp32 has lost all its
// digits at position 2^24, and fp64 is slow here. The two top bits of phase + 1/8
// turn pick the quadrant, the rest is an angle of at most an eighth of a turn
// that fp32 holds to 2^-27 half turns.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "elements.h"

namespace tkv {
namespace {

constexpr int kRotaryThreads = 256;
constexpr int kMaxHeadDim = 512;
constexpr int kTurns = 2048;      // sines and cosines a CTA holds
constexpr int kMaxTokens = 8;     // tokens of a CTA
constexpr int kCtaVectors = 1024; // vectors (half layout: pairs of them) of a CTA, at most
constexpr int kManyTokens = 152 * 6;  // a token for each of the CTAs that run at once

struct RotateParams {
  const void *q, *k;
  void *q_out, *k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;  // elements from one token to the next
  const uint64_t* steps;
  const void* positions;
  int64_t tokens;
  int32_t q_heads, k_heads, d, pairs;
  int32_t wide;         // positions are 64-bit
  int32_t interleaved;  // pairs are (2 i, 2 i + 1), else (i, i + pairs)
  int32_t inverse;
  int32_t per_cta;      // tokens of a CTA
  int32_t heads_cta;    // vectors: heads of a CTA
  float scale;
};

__device__ __forceinline__ float2 turn(const RotateParams& p, int64_t pos, int i) {
  uint64_t phase = static_cast<uint64_t>(pos) * p.steps[i];
  if (p.inverse) phase = 0 - phase;
  const uint32_t quadrant = static_cast<uint32_t>((phase + (uint64_t(1) << 61)) >> 62);
  const int64_t rest = static_cast<int64_t>(phase - (static_cast<uint64_t>(quadrant) << 62));
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-63f, &s, &c);
  const float x = quadrant & 1 ? s : c, y = quadrant & 1 ? c : s;
  return make_float2((quadrant == 1 || quadrant == 2 ? -x : x) * p.scale, (quadrant >= 2 ? -y : y) * p.scale);
}

__device__ __forceinline__ int64_t position(const RotateParams& p, int64_t token) {
  return p.wide ? static_cast<const int64_t*>(p.positions)[token] : static_cast<const int32_t*>(p.positions)[token];
}

// The sines and cosines of a CTA's tokens, formed once for all their heads. Of a
// vector's kGroup pairs the first ones of all vectors lie together, then the second
// ones: neighbouring threads then read neighbouring banks.
template <int kGroup>
__device__ __forceinline__ void form_turns(const RotateParams& p, int64_t token0, int tokens, float2* s_turn) {
  for (int w = threadIdx.x; w < tokens * p.pairs; w += kRotaryThreads) {
    const int token = w / p.pairs, i = w - token * p.pairs;
    s_turn[token * p.pairs + i % kGroup * (p.pairs / kGroup) + i / kGroup] = turn(p, position(p, token0 + token), i);
  }
}

// Rows of any alignment and pairs of any number: an element or a pair per thread. 8192 tokens
// of 40 heads at d 128 in bf16 take 123 us with rows off 16 bytes (vectors: 30) and 201 with 25
// pairs, whose heads are 103 items of work instead of 64.
template <typename T>
__global__ void __launch_bounds__(kRotaryThreads) rotate_kernel(const __grid_constant__ RotateParams p) {
  __shared__ float2 s_turn[kTurns];
  cudaGridDependencySynchronize();
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * p.per_cta;
  const int tokens = static_cast<int>(min(p.tokens - token0, static_cast<int64_t>(p.per_cta)));
  form_turns<1>(p, token0, tokens, s_turn);
  __syncthreads();
  const int work = p.d - p.pairs, heads = p.q_heads + p.k_heads;  // pairs, then elements that pass
  for (int w = threadIdx.x; w < tokens * heads * work; w += kRotaryThreads) {
    const int row = w / work, i = w - row * work, token = row / heads, head = row - token * heads;
    const bool is_q = head < p.q_heads;
    const int64_t at = static_cast<int64_t>(is_q ? head : head - p.q_heads) * p.d;
    const T* from = static_cast<const T*>(is_q ? p.q : p.k) + (token0 + token) * (is_q ? p.q_stride : p.k_stride) + at;
    T* to = static_cast<T*>(is_q ? p.q_out : p.k_out) + (token0 + token) * (is_q ? p.q_out_stride : p.k_out_stride) + at;
    if (i < p.pairs) {
      const int ia = p.interleaved ? 2 * i : i, ib = p.interleaved ? 2 * i + 1 : i + p.pairs;
      const float2 t = s_turn[token * p.pairs + i];
      const float a = to_float(from[ia]), b = to_float(from[ib]);
      put(to + ia, a * t.x - b * t.y);
      put(to + ib, b * t.x + a * t.y);
    } else {
      to[i + p.pairs] = from[i + p.pairs];
    }
  }
}

// Rows of whole 16-byte vectors. A thread keeps its place in the head (one vector
// of pairs, or the two that hold them, or one that passes) and goes through the heads
// of the CTA's tokens, 64 bytes on their way at a time; the first ones leave before
// the sines are formed. HBM bounds it: 8192 tokens of 40 heads at d 128 in bf16,
// 168 MB, take 30 us with inputs past the L2 (5.5 TB/s; 25 at the rate of a copy), and 27 in a
// row of calls on the same inputs, of which the L2 holds a part. CTAs of
// 1024 vectors: with 2048 the second wave is short of CTAs (32 us, and 25 for 22 at
// 1501 tokens of 64 heads in fp32), with 512 the sines weigh more (34 us).
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRotaryThreads) rotate_vectors_kernel(const __grid_constant__ RotateParams p) {
  using V = Vec<T>;
  constexpr int kAhead = kInterleaved ? 4 : 2;            // vectors (half layout: pairs of them) on their way
  constexpr int kGroup = kInterleaved ? V::n / 2 : V::n;  // pairs of a thread
  __shared__ float2 s_turn[kTurns];
  cudaGridDependencySynchronize();
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * p.per_cta;
  const int tokens = static_cast<int>(min(p.tokens - token0, static_cast<int64_t>(p.per_cta)));
  const int turning = (kInterleaved ? 2 * p.pairs : p.pairs) / V::n, items = turning + (p.d - 2 * p.pairs) / V::n;
  const int step = kRotaryThreads / items;         // heads in one go
  const int head0 = blockIdx.y * p.heads_cta, heads = min(p.heads_cta, p.q_heads + p.k_heads - head0);
  const int item = threadIdx.x % items;
  int head = threadIdx.x / items, token = threadIdx.x < step * items ? 0 : tokens;
  const bool turns = item < turning;
  const int at = turns ? item * V::n : 2 * p.pairs + (item - turning) * V::n;
  auto advance = [&] {
    while (head >= heads && token < tokens) head -= heads, ++token;
  };
  int4 x[kAhead], y[kAhead];
  T* to[kAhead];
  int of[kAhead];
  auto load = [&] {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      of[u] = token;
      if (token >= tokens) continue;
      const bool is_q = head0 + head < p.q_heads;
      const int64_t in_token = static_cast<int64_t>(is_q ? head0 + head : head0 + head - p.q_heads) * p.d + at;
      const T* from = static_cast<const T*>(is_q ? p.q : p.k) + (token0 + token) * (is_q ? p.q_stride : p.k_stride) + in_token;
      to[u] = static_cast<T*>(is_q ? p.q_out : p.k_out) + (token0 + token) * (is_q ? p.q_out_stride : p.k_out_stride) + in_token;
      x[u] = *reinterpret_cast<const int4*>(from);
      if (!kInterleaved && turns) y[u] = *reinterpret_cast<const int4*>(from + p.pairs);
      head += step;
      advance();
    }
  };
  advance();
  load();
  form_turns<kGroup>(p, token0, tokens, s_turn);
  __syncthreads();
  while (of[0] < tokens) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (of[u] >= tokens) break;
      const float2* t = s_turn + of[u] * p.pairs + item;
      float a[V::n], b[V::n];
      V::unpack(x[u], a);
      if (turns && kInterleaved) {
#pragma unroll
        for (int i = 0; i < V::n; i += 2) {
          const float2 c = t[i / 2 * turning];
          const float v = a[i], w = a[i + 1];
          a[i] = v * c.x - w * c.y;
          a[i + 1] = w * c.x + v * c.y;
        }
      } else if (turns) {
        V::unpack(y[u], b);
#pragma unroll
        for (int i = 0; i < V::n; ++i) {
          const float2 c = t[i * turning];
          const float v = a[i], w = b[i];
          a[i] = v * c.x - w * c.y;
          b[i] = w * c.x + v * c.y;
        }
        *reinterpret_cast<int4*>(to[u] + p.pairs) = V::pack(b);
      }
      *reinterpret_cast<int4*>(to[u]) = turns ? V::pack(a) : x[u];
    }
    load();
  }
}

template <typename T>
cudaError_t launch_rotate(const RotateParams& p, bool vectors, dim3 ctas, cudaStream_t s) {
  void (*const kernel)(RotateParams) = !vectors ? rotate_kernel<T> : p.interleaved ? rotate_vectors_kernel<T, true> : rotate_vectors_kernel<T, false>;
  return launch_early(kernel, ctas, kRotaryThreads, 0, s, 1, p);
}

}  // namespace
}  // namespace tkv

using namespace tkv;

extern "C" {

tkv_status tkv_rotary_steps(int32_t n, const double* inv_freq, uint64_t* steps) {
  if (n < 1 || n > kMaxHeadDim / 2) return tkv_status(report(TKV_ERR_INVALID_ARG, "n must be 1 to %d", kMaxHeadDim / 2));
  if (!inv_freq || !steps) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  for (int i = 0; i < n; ++i)
    if (!(std::fabs(inv_freq[i]) <= 0x1p32)) return tkv_status(report(TKV_ERR_INVALID_ARG, "inv_freq[%d] not finite or above 2^32", i));
  // 1 / 2 pi in two doubles
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  for (int i = 0; i < n; ++i) {
    const double x = std::fabs(inv_freq[i]), turns = x * kHi;
    const double rest = std::fma(x, kHi, -turns) + x * kLo;
    const double part = turns - std::floor(turns);  // exact
    const uint64_t step = static_cast<uint64_t>(part * 0x1p64) + static_cast<uint64_t>(std::llrint(rest * 0x1p64));
    steps[i] = inv_freq[i] < 0 ? 0 - step : step;
  }
  return TKV_OK;
}

tkv_status tkv_rotate(int64_t n_tokens, int32_t n_q_heads, int32_t n_k_heads, int32_t head_dim, int32_t rotary_dim,
                      int32_t dtype, int32_t interleaved, int32_t inverse, float scale, const uint64_t* steps,
                      const void* positions, int32_t position_bits, const void* q, int64_t q_stride, const void* k,
                      int64_t k_stride, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                      tkv_stream stream) {
  if (n_tokens < 0 || n_tokens > INT32_MAX) return tkv_status(report(TKV_ERR_INVALID_ARG, "n_tokens out of 0..2^31 - 1"));
  if (n_q_heads < 0 || n_k_heads < 0 || n_q_heads > 65535 || n_k_heads > 65535 || n_q_heads + n_k_heads == 0)
    return tkv_status(report(TKV_ERR_INVALID_ARG, "n_q_heads and n_k_heads must be 0 to 65535, one of them at least 1"));
  if (head_dim < 2 || head_dim > kMaxHeadDim) return tkv_status(report(TKV_ERR_INVALID_ARG, "head_dim must be 2 to %d", kMaxHeadDim));
  if (rotary_dim < 2 || rotary_dim > head_dim || rotary_dim % 2)
    return tkv_status(report(TKV_ERR_INVALID_ARG, "rotary_dim must be even, 2 to head_dim"));
  if (int st = check_dtype(dtype)) return tkv_status(st);
  if (position_bits != 32 && position_bits != 64) return tkv_status(report(TKV_ERR_INVALID_ARG, "position_bits must be 32 or 64"));
  if (!std::isfinite(scale)) return tkv_status(report(TKV_ERR_INVALID_ARG, "scale must be finite"));
  if (n_tokens == 0) return TKV_OK;
  if (!steps || !positions || (n_q_heads && (!q || !q_out)) || (n_k_heads && (!k || !k_out)))
    return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  const int esz = dtype == TKV_DTYPE_BF16 ? 2 : 4;
  if (misaligned(steps, 8) || misaligned(positions, position_bits / 8) || misaligned(q, esz) || misaligned(k, esz) ||
      misaligned(q_out, esz) || misaligned(k_out, esz))
    return tkv_status(report(TKV_ERR_INVALID_ARG, "a pointer is not aligned to its elements"));
  const int64_t qrow = static_cast<int64_t>(n_q_heads) * head_dim, krow = static_cast<int64_t>(n_k_heads) * head_dim;
  if (q_stride < qrow || q_out_stride < qrow || k_stride < krow || k_out_stride < krow ||
      (q_stride | q_out_stride | k_stride | k_out_stride) >> 36)
    return tkv_status(report(TKV_ERR_INVALID_ARG, "token strides must hold a token"));
  if ((n_q_heads && q == q_out && q_stride != q_out_stride) || (n_k_heads && k == k_out && k_stride != k_out_stride))
    return tkv_status(report(TKV_ERR_INVALID_ARG, "in place, the output's stride must be the input's"));
  if (n_q_heads && n_k_heads && q_out == k_out) return tkv_status(report(TKV_ERR_INVALID_ARG, "q_out and k_out are the same"));
  RotateParams p{};
  p.q = q; p.k = k; p.q_out = q_out; p.k_out = k_out;
  p.q_stride = q_stride; p.k_stride = k_stride; p.q_out_stride = q_out_stride; p.k_out_stride = k_out_stride;
  p.steps = steps;
  p.positions = positions;
  p.tokens = n_tokens;
  p.q_heads = n_q_heads; p.k_heads = n_k_heads; p.d = head_dim; p.pairs = rotary_dim / 2;
  p.wide = position_bits == 64;
  p.interleaved = interleaved != 0;
  p.inverse = inverse != 0;
  p.scale = scale;
  // 16-byte vectors: every row, half of the pairs and part that passes starts and ends on one
  const int unit = 16 / esz;
  const bool vectors = !misaligned(q, 16) && !misaligned(k, 16) && !misaligned(q_out, 16) && !misaligned(k_out, 16) &&
                       (q_stride | k_stride | q_out_stride | k_out_stride | head_dim) % unit == 0 &&
                       (interleaved ? rotary_dim : rotary_dim / 2) % unit == 0;
  const int heads = n_q_heads + n_k_heads;
  const int64_t row = (interleaved ? rotary_dim : rotary_dim / 2) / unit + (head_dim - rotary_dim) / unit;  // vectors (or pairs of them) of a head
  p.heads_cta = heads;
  if (vectors) {  // equal groups of heads
    const int64_t fit = std::clamp<int64_t>(kCtaVectors / row, 1, heads), groups = (heads + fit - 1) / fit;
    p.heads_cta = static_cast<int32_t>((heads + groups - 1) / groups);
  }
  const int64_t most = vectors ? std::max<int64_t>(1, kCtaVectors / (p.heads_cta * row)) : kMaxTokens;
  p.per_cta = static_cast<int32_t>(std::clamp<int64_t>(n_tokens / kManyTokens, 1, std::min<int64_t>(most, std::min(kMaxTokens, kTurns / p.pairs))));
  const dim3 ctas(static_cast<unsigned>((n_tokens + p.per_cta - 1) / p.per_cta), (heads + p.heads_cta - 1) / p.heads_cta);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return tkv_status(launched("rotate", dtype == TKV_DTYPE_BF16 ? launch_rotate<__nv_bfloat16>(p, vectors, ctas, s)
                                                               : launch_rotate<float>(p, vectors, ctas, s)));
}

}  // extern "C"
