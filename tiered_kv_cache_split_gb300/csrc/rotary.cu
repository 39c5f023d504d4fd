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
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "tkv.h"
#include "tkv_internal.h"

namespace tkv {
namespace {

constexpr int kRotaryThreads = 128;
constexpr int kMaxHeadDim = 512;

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

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* at, float x) { *at = x; }
__device__ __forceinline__ void put(__nv_bfloat16* at, float x) { *at = __float2bfloat16_rn(x); }

// One CTA per token: the sines and cosines of its pairs once, then all heads.
template <typename T>
__global__ void __launch_bounds__(kRotaryThreads) rotate_kernel(const __grid_constant__ RotateParams p) {
  __shared__ float2 s_turn[kMaxHeadDim / 2];
  for (int64_t token = blockIdx.x; token < p.tokens; token += gridDim.x) {
    const int64_t pos = position(p, token);
    __syncthreads();
    for (int i = threadIdx.x; i < p.pairs; i += kRotaryThreads) s_turn[i] = turn(p, pos, i);
    __syncthreads();
    const int work = p.d - p.pairs;  // pairs, then elements that pass
    for (int w = threadIdx.x; w < (p.q_heads + p.k_heads) * work; w += kRotaryThreads) {
      const int head = w / work, i = w % work;
      const bool is_q = head < p.q_heads;
      const int64_t at = static_cast<int64_t>(is_q ? head : head - p.q_heads) * p.d;
      const T* from = static_cast<const T*>(is_q ? p.q : p.k) + token * (is_q ? p.q_stride : p.k_stride) + at;
      T* to = static_cast<T*>(is_q ? p.q_out : p.k_out) + token * (is_q ? p.q_out_stride : p.k_out_stride) + at;
      if (i < p.pairs) {
        const int ia = p.interleaved ? 2 * i : i, ib = p.interleaved ? 2 * i + 1 : i + p.pairs;
        const float2 t = s_turn[i];
        const float a = to_float(from[ia]), b = to_float(from[ib]);
        put(to + ia, a * t.x - b * t.y);
        put(to + ib, b * t.x + a * t.y);
      } else {
        to[i + p.pairs] = from[i + p.pairs];
      }
    }
  }
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
  if (dtype != TKV_DTYPE_F32 && dtype != TKV_DTYPE_BF16) return tkv_status(report(TKV_ERR_INVALID_ARG, "dtype"));
  if (position_bits != 32 && position_bits != 64) return tkv_status(report(TKV_ERR_INVALID_ARG, "position_bits must be 32 or 64"));
  if (!std::isfinite(scale)) return tkv_status(report(TKV_ERR_INVALID_ARG, "scale must be finite"));
  if (n_tokens == 0) return TKV_OK;
  if (!steps || !positions || (n_q_heads && (!q || !q_out)) || (n_k_heads && (!k || !k_out)))
    return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  const int esz = dtype == TKV_DTYPE_BF16 ? 2 : 4;
  auto misaligned = [](const void* ptr, int to) { return reinterpret_cast<uintptr_t>(ptr) % to != 0; };
  if (misaligned(steps, 8) || misaligned(positions, position_bits / 8) || misaligned(q, esz) || misaligned(k, esz) ||
      misaligned(q_out, esz) || misaligned(k_out, esz))
    return tkv_status(report(TKV_ERR_INVALID_ARG, "a pointer is not aligned to its elements"));
  const int64_t qrow = static_cast<int64_t>(n_q_heads) * head_dim, krow = static_cast<int64_t>(n_k_heads) * head_dim;
  if (q_stride < qrow || q_out_stride < qrow || k_stride < krow || k_out_stride < krow ||
      (q_stride | q_out_stride | k_stride | k_out_stride) >> 36)
    return tkv_status(report(TKV_ERR_INVALID_ARG, "token strides must hold a token"));
  if ((n_q_heads && q == q_out && q_stride != q_out_stride) || (n_k_heads && k == k_out && k_stride != k_out_stride))
    return tkv_status(report(TKV_ERR_INVALID_ARG, "in place, the output's stride must be the input's"));
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
  const unsigned ctas = static_cast<unsigned>(std::min<int64_t>(n_tokens, 152 * 16));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == TKV_DTYPE_BF16) rotate_kernel<__nv_bfloat16><<<ctas, kRotaryThreads, 0, s>>>(p);
  else rotate_kernel<float><<<ctas, kRotaryThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TKV_OK : tkv_status(report(TKV_ERR_CUDA, "rotate launch failed: %s", cudaGetErrorString(e)));
}

}  // extern "C"
