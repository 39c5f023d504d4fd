// Prompt attention and shared-prefix decode attention: planning, the C ABI, the
// fp32 kernel and the merge of partials (see tile_attention.h for the terms).
//
// For a row with logits l_j = q . k_j log2(e) / sqrt(d) over its keys,
//   m = max l_j,  Z = sum 2^(l_j - m),  O = sum 2^(l_j - m) v_j,  out = O / Z,
// all of it in one pass over the keys: when a block raises m, Z and O are
// scaled by 2^(m_old - m_new). Partials of disjoint key ranges join the same
// way. A row without a key has m = -inf, Z = 0 and gives 0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "tile_attention.h"
#include "tkv.h"

namespace tkv {
namespace {

constexpr int kFmaThreads = 256;
constexpr int kFmaRows = 64;   // rows of a tile
constexpr int kMmaRows = 128;  // rows of a bf16 tile, two to a group
constexpr int kFmaKeys = 64;   // keys staged at once (half a key block)
constexpr int kMaxPromptKeys = 1 << 26;
// Longest key range of a unit (what a full page table holds). Its sums are
// sequential in fp32, and the tensor core's accumulator loses up to a step
// (2^-23 of it) at every addition of 8 or 16 keys into O: at most 2^-8 of a sum of
// 2^18 keys that agree in sign, half a step of bf16. Longer rows are joined from
// partials (one unit over 2^21 keys of a constant V gave results 2 % low; over 2^18
// they round to V). A unit stays under 10 ms, too.
constexpr int kMaxUnitKeys = 1 << 18;
constexpr int kSms = 152;      // SMs of a GB300: what the plan fills (results do not depend on the device)

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ bool finite1(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// fp32 FMA kernel: 64 rows x 64 keys at a time, 256 threads as 16 x 16, each
// with a 4 x 4 patch of S and 4 rows x D / 16 columns of O. The weights take the
// place of K in shared memory, so that two CTAs fit on an SM at d = 128 and one
// loads while the other computes; at 64 more would fit, but 128 registers a thread
// allow two. Bound by the FMA pipe and about as
// much by shared-memory reads: tensor cores would round fp32 operands. Two
// 1024-token prompts with 28 / 4 heads, d 128: 422 us, 35.7 TFLOP/s (half of the
// FMA pipe's 75).
template <int D>
__global__ void __launch_bounds__(kFmaThreads, 2) tile_fma_kernel(const __grid_constant__ TileParams p) {
  constexpr int LD = D + 4, LP = kFmaKeys + 4, C4 = D / 4, NC = D / 64;
  static_assert(kFmaRows * LP <= kFmaKeys * LD, "the weights fit where K was");
  extern __shared__ float4 smem4[];
  float* sq = reinterpret_cast<float*>(smem4);
  float* sk = sq + kFmaRows * LD;
  float* sv = sk + kFmaKeys * LD;
  float* sp = sk;  // weights, once S is done
  __shared__ int64_t s_page[kFmaKeys / kPage];   // page of each 16 keys of the stage, -1: none
  __shared__ uint32_t s_bits[kFmaKeys / kPage];  // its valid slots
  // keys that only some rows of the tile see and whose V row is not finite
  __shared__ uint32_t s_flag[kFmaRows / 32 + 1];

  const TileUnit t = tile_unit(p, blockIdx.x);
  const TileSeg& sg = p.seg[t.seg];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const float* q = static_cast<const float*>(p.q);
  const int G = p.G;

  for (int i = tid; i < kFmaRows * C4; i += kFmaThreads) {
    const int r = i / C4, c = i % C4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < t.rows) {
      const int row = t.row0 + r;
      x = load4(q + static_cast<int64_t>(sg.tok0 + row / G) * p.q_stride + (t.h * G + row % G) * D + c * 4);
    }
    store4(sq + r * LD + c * 4, x);
  }
  if (tid <= kFmaRows / 32) s_flag[tid] = 0;

  int lim[4];
  float m[4], z[4];
  float2 o2[4][NC * 2];  // columns 4 tx .. of each 64
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lim[i] = tile_row_limit(p, sg, t.row0 + min(ty * 4 + i, t.rows - 1));
    m[i] = -INFINITY;
    z[i] = 0.f;
#pragma unroll
    for (int c = 0; c < NC * 2; ++c) o2[i][c] = make_float2(0.f, 0.f);
  }
  const int lim_first = tile_row_limit(p, sg, t.row0);
  const int kend = min(t.j1 * kKeyBlock, tile_row_limit(p, sg, t.row0 + t.rows - 1));

  for (int k0 = t.j0 * kKeyBlock; k0 < kend; k0 += kFmaKeys) {
    __syncthreads();
    if (tid < kFmaKeys / kPage) {
      const int pg = k0 / kPage + tid;
      int64_t id = -1;
      uint32_t bits = 0;
      if (p.paged) {
        if (pg < sg.nkeys / kPage) {
          id = p.table[sg.key0 + pg];
          if (id < 0 || id >= p.pages) id = -1;
          if (id >= 0) bits = p.mask[id] & 0xffffu;
        }
      } else {
        const int left = sg.nkeys - pg * kPage;
        bits = left >= kPage ? 0xffffu : left > 0 ? (1u << left) - 1 : 0u;
      }
      s_page[tid] = id;
      s_bits[tid] = bits;
    }
    __syncthreads();
    for (int i = tid; i < kFmaKeys * C4; i += kFmaThreads) {
      const int kk = i / C4, c = i % C4;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
      if ((s_bits[kk / kPage] >> (kk % kPage)) & 1u) {
        if (p.paged) {
          const float* at = static_cast<const float*>(p.pool) + ((s_page[kk / kPage] * p.Hkv + t.h) * 2 * kPage + kk % kPage) * D + c * 4;
          a = load4(at);
          b = load4(at + kPage * D);
        } else {
          const int64_t tok = sg.key0 + k0 + kk;
          a = load4(static_cast<const float*>(p.k) + tok * p.k_stride + t.h * D + c * 4);
          b = load4(static_cast<const float*>(p.v) + tok * p.v_stride + t.h * D + c * 4);
        }
        const int part = k0 + kk - lim_first;  // >= 0: the tile's first row does not see this key
        if (part >= 0 && !(finite1(b.x) && finite1(b.y) && finite1(b.z) && finite1(b.w))) {
          // 0 * inf must not reach the rows that do not see the key: the rows that do get it below
          if (!finite1(b.x)) b.x = 0.f;
          if (!finite1(b.y)) b.y = 0.f;
          if (!finite1(b.z)) b.z = 0.f;
          if (!finite1(b.w)) b.w = 0.f;
          if (part < kFmaRows) atomicOr(&s_flag[part >> 5], 1u << (part & 31));
        }
      }
      store4(sk + kk * LD + c * 4, a);
      store4(sv + kk * LD + c * 4, b);
    }
    __syncthreads();
    float2 s2[4][4] = {};  // even and odd columns apart
#pragma unroll 4
    for (int c = 0; c < C4; ++c) {
      float4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = load4(sq + (ty * 4 + i) * LD + c * 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = load4(sk + (tx + 16 * j) * LD + c * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s2[i][j] = fma2(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), s2[i][j]);
          s2[i][j] = fma2(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), s2[i][j]);
        }
    }
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j].x + s2[i][j].y;
    __syncthreads();  // K is done with
    // key tx + 16 j is slot tx of page j of the stage
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool seen = ((s_bits[j] >> tx) & 1u) && k0 + 16 * j + tx < lim[i];
        s[i][j] = seen ? s[i][j] * p.qscale : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float mn = fmaxf(m[i], top);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[i] - base);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (sg.spill0 >= 0 && ty * 4 + i < t.rows && k0 + 16 * j + tx < sg.nkeys)
          p.spill[sg.spill0 + static_cast<int64_t>(t.h * G + (t.row0 + ty * 4 + i) % G) * sg.nkeys + k0 + 16 * j + tx] = s[i][j];
        const float e = exp2f(s[i][j] - base);
        sum += e;
        sp[(ty * 4 + i) * LP + tx + 16 * j] = e;
      }
#pragma unroll
      for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      z[i] = z[i] * f + sum;
#pragma unroll
      for (int c = 0; c < NC * 2; ++c) o2[i][c].x *= f, o2[i][c].y *= f;
    }
    __syncwarp();  // a row's weights are written and read by the same half warp
#pragma unroll 2
    for (int kk = 0; kk < kFmaKeys; kk += 4) {
      float e[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = load4(sp + (ty * 4 + i) * LP + kk);
        e[i][0] = x.x, e[i][1] = x.y, e[i][2] = x.z, e[i][3] = x.w;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float4 v[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) v[c] = load4(sv + (kk + u) * LD + c * 64 + tx * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float2 w = make_float2(e[i][u], e[i][u]);
            o2[i][c * 2] = fma2(w, make_float2(v[c].x, v[c].y), o2[i][c * 2]);
            o2[i][c * 2 + 1] = fma2(w, make_float2(v[c].z, v[c].w), o2[i][c * 2 + 1]);
          }
        }
      }
    }
  }
  float o[4][NC * 4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < NC * 2; ++c) o[i][c * 2] = o2[i][c].x, o[i][c * 2 + 1] = o2[i][c].y;
  __syncthreads();
  // the non-finite values of partly seen keys, for the rows that see them
  for (int part = 0; part < kFmaRows; ++part) {
    if (!((s_flag[part >> 5] >> (part & 31)) & 1u)) continue;
    const int64_t tok = sg.key0 + lim_first + part;
#pragma unroll
    for (int c = 0; c < NC * 4; ++c) {
      const int col = (c / 4) * 64 + tx * 4 + c % 4;
      const float x = static_cast<float>(static_cast<const float*>(p.v)[tok * p.v_stride + t.h * D + col]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lim_first + part < lim[i] && !finite1(x)) o[i][c] += x;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i, row = t.row0 + r;
    if (r >= t.rows) continue;
    if (sg.direct) {
      const float inv = z[i] > 0.f || z[i] != z[i] ? 1.f / z[i] : 0.f;
      float* at = static_cast<float*>(p.out) + static_cast<int64_t>(sg.tok0 + row / G) * p.out_stride + (t.h * G + row % G) * D + tx * 4;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        store4(at + c * 64, make_float4(o[i][c * 4] * inv, o[i][c * 4 + 1] * inv, o[i][c * 4 + 2] * inv, o[i][c * 4 + 3] * inv));
    } else {
      const int64_t pr = tile_part_row(p, sg, t.grp, t.h, t.split, 0) + r;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        store4(p.part_o + (pr - r) * D + ((c * 8 + tx / 2) * sg.part_rows + r) * 8 + (tx & 1) * 4, make_float4(o[i][c * 4], o[i][c * 4 + 1], o[i][c * 4 + 2], o[i][c * 4 + 3]));
      if (tx == 0) {
        p.part_m[pr] = m[i];
        p.part_z[pr] = z[i];
      }
    }
  }
}

// ---- merge: out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) Z_i over a row's
// partials. Four warps share a row's partials where a row has many (few rows,
// split far), else each takes a row. Bound by reading the partials, which the
// L2 mostly still holds; eight loads per lane are in flight. Sharing: one token
// with 32 heads behind 32767 keys 33.0 us for the call against 35.2 without; 64
// rows of 32 heads 126.8 with it against 125.2, hence the bound on rows.
// A second kind of CTA serves decode steps with alpha: 512 own slots of a
// (sequence, KV head), adding the softmax weights of their spilled logits
// summed over the G heads; it forms M and Z of the G heads for itself.
constexpr int kMergeThreads = 128;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kAlphaSlots = kMergeThreads * 4;
// Four warps share a row from this many partials, while rows are at most one wave of CTAs.
constexpr int kShareParts = 16, kShareRows = 152 * 8;

struct PartList {
  int64_t first[2], step[2];  // partial row i of a list is first + i * step
  int row[2], rows[2];        // the row in its tile, rows of a partial tile
  int n0, n;                  // partials of the first list, of both
  __device__ __forceinline__ int64_t at(int i) const { return i < n0 ? first[0] + i * step[0] : first[1] + (i - n0) * step[1]; }
};

template <bool kMma>
__device__ __forceinline__ void add_parts(PartList& l, int which, const TileParams& p, const TileSeg& s, int h, int row) {
  if (s.splits == 0) return;
  int n;
  l.rows[which] = s.part_rows;
  if (s.pair) {
    l.first[which] = tile_part_row(p, s, 0, h, 0, 0) + row;
    l.row[which] = row;
    l.step[which] = s.part_rows;
    n = s.splits * 2;
  } else {
    constexpr uint32_t kTile = kMma ? kMmaRows : kFmaRows, kPer = kMma ? 2 * kMmaRows : kFmaRows;
    const uint32_t r = row;
    l.row[which] = r % kTile;
    l.first[which] = tile_part_row(p, s, r / kPer, h, 0, r % kPer / kTile) + r % kTile;
    l.step[which] = static_cast<int64_t>(p.tpg) * s.part_rows;
    n = s.splits;
  }
  if (which == 0) l.n0 = n;
  l.n += n;
}

// The partials of query head h * G + g of the n-th token that has partials; *tok: that token.
template <bool kMma>
__device__ __forceinline__ PartList part_list(const TileParams& p, int n, int h, int g, int* tok) {
  PartList l{};
  *tok = n;
  if (p.paged) {  // segment 0 is the prefix of all tokens
    add_parts<kMma>(l, 0, p, p.seg[0], h, n * p.G + g);
    add_parts<kMma>(l, 1, p, p.seg[n + 1], h, g);
  } else {
    int own = 0;
    for (int i = 0, at = 0; i < p.nseg; ++i) {
      if (p.seg[i].direct) continue;
      if (n >= at && n < at + p.seg[i].ntok) own = i, *tok = p.seg[i].tok0 + n - at;
      at += p.seg[i].ntok;
    }
    add_parts<kMma>(l, 0, p, p.seg[own], h, (*tok - p.seg[own].tok0) * p.G + g);
  }
  return l;
}

// M (0 where there is no key) and Z of a row, by one warp in one pass. A partial
// whose logits are all NaN has m = -inf and Z NaN, which stays.
__device__ __forceinline__ float2 parts_sum(const TileParams& p, const PartList& l, const float* part_z, int lane) {
  float m = -INFINITY, z = 0.f;
  for (int i = lane; i < l.n; i += 32) {
    const float mi = p.part_m[l.at(i)], zi = part_z[l.at(i)], next = fmaxf(m, mi);
    if (next == -INFINITY) {
      z += zi;
      continue;
    }
    z = z * exp2f(m - next) + zi * exp2f(mi - next);
    m = next;
  }
  float M = m;
#pragma unroll
  for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  M = M == -INFINITY ? 0.f : M;
  z *= exp2f(m - M);
#pragma unroll
  for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
  return make_float2(M, z);
}
__device__ __forceinline__ float parts_inv(float z) { return z > 0.f || z != z ? 1.f / z : 0.f; }
// Weight of a logit; an empty slot (-inf) has none even where the row is NaN.
__device__ __forceinline__ float alpha_weight(float x, float m, float inv) { return x == -INFINITY ? 0.f : exp2f(x - m) * inv; }

template <typename T, int D, int kShare>
__global__ void __launch_bounds__(kMergeThreads) tile_merge_kernel(const __grid_constant__ TileParams p, uint32_t rows, int row_ctas) {
  constexpr int E = D / 32, kAhead = 8;
  __shared__ float s_acc[kMergeWarps][D], s_m[kMaxGroup], s_inv[kMaxGroup];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = p.G;
  cudaGridDependencySynchronize();
  if (static_cast<int>(blockIdx.x) < row_ctas) {
    const uint32_t row = blockIdx.x * (kMergeWarps / kShare) + warp / kShare, hq_all = p.Hq;
    const bool live = row < rows;
    float acc[E] = {}, z = 0.f;
    int tok = 0;
    const int hq = live ? row % hq_all : 0;
    if (live) {
      const uint32_t h = static_cast<uint32_t>(hq) / static_cast<uint32_t>(G);
      const PartList l = part_list<sizeof(T) == 2>(p, row / hq_all, h, hq - h * G, &tok);
      int64_t off[2];  // this lane's columns, from a partial row's number of elements
#pragma unroll
      for (int q = 0; q < 2; ++q)
        off[q] = (static_cast<int64_t>(lane * E / 8) * l.rows[q] + l.row[q]) * 8 + lane * E % 8 - static_cast<int64_t>(l.row[q]) * D;
      float v[kAhead][E];
      auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (i0 + i < l.n) {
            const float* at = p.part_o + l.at(i0 + i) * D + off[i0 + i >= l.n0];
            if constexpr (E == 4) {
              const float4 x = *reinterpret_cast<const float4*>(at);
              v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
            } else {
              const float2 x = *reinterpret_cast<const float2*>(at);
              v[i][0] = x.x, v[i][1] = x.y;
            }
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e) v[i][e] = 0.f;
          }
        }
      };
      int i0 = warp % kShare * kAhead;
      load(i0);  // on its way while M and Z are formed
      const float2 mz = parts_sum(p, l, p.part_z, lane);
      z = mz.y;
      while (i0 < l.n) {
        const float w = lane < kAhead && i0 + lane < l.n ? exp2f(p.part_m[l.at(i0 + lane)] - mz.x) : 0.f;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(wi, v[i][e], acc[e]);
        }
        i0 += kShare * kAhead;
        if (i0 < l.n) load(i0);
      }
    }
    if constexpr (kShare > 1) {
      if (warp > 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
      }
      __syncthreads();
      if (warp > 0) return;
      for (int o = 1; o < kMergeWarps; ++o) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += s_acc[o][lane * E + e];
      }
    }
    if (!live) return;
    const float inv = parts_inv(z);
    T* at = static_cast<T*>(p.out) + static_cast<int64_t>(tok) * p.out_stride + hq * D + lane * E;
    if constexpr (sizeof(T) == 2 && E == 4) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv), b = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
      *reinterpret_cast<uint2*>(at) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) at[e] = static_cast<T>(acc[e] * inv);
    }
    return;
  }
  // alpha
  const int per = (static_cast<int>(gridDim.x) - row_ctas) / (static_cast<int>(rows / static_cast<uint32_t>(p.Hq)) * p.Hkv);  // CTAs of a (sequence, KV head)
  const int item = blockIdx.x - row_ctas, tok = item / per / p.Hkv, h = item / per % p.Hkv;
  const TileSeg& so = p.seg[tok + 1];
  const int i = item % per * kAlphaSlots + threadIdx.x * 4;
  if (item % per * kAlphaSlots >= so.nkeys) return;
  for (int g = warp; g < G; g += kMergeWarps) {
    int same;
    const float2 mz = parts_sum(p, part_list<sizeof(T) == 2>(p, tok, h, g, &same), p.part_ze, lane);
    if (lane == 0) {
      s_m[g] = mz.x;
      s_inv[g] = parts_inv(mz.y);
    }
  }
  __syncthreads();
  if (i >= so.nkeys) return;
  const float* l = p.spill + so.spill0 + static_cast<int64_t>(h) * G * so.nkeys + i;
  float4* at = reinterpret_cast<float4*>(p.alpha + (static_cast<int64_t>(tok) * p.Hkv + h) * p.alpha_stride_h + p.alpha_first + i);
  const float4 before = *at;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);  // of the heads first: what was there may be much larger, and is rounded once
#pragma unroll 4
  for (int g = 0; g < G; ++g) {
    const float4 x = *reinterpret_cast<const float4*>(l + static_cast<int64_t>(g) * so.nkeys);
    sum.x += alpha_weight(x.x, s_m[g], s_inv[g]);
    sum.y += alpha_weight(x.y, s_m[g], s_inv[g]);
    sum.z += alpha_weight(x.z, s_m[g], s_inv[g]);
    sum.w += alpha_weight(x.w, s_m[g], s_inv[g]);
  }
  *at = make_float4(before.x + sum.x, before.y + sum.y, before.z + sum.z, before.w + sum.w);
}

// ---- planning (host)

struct TilePlan {
  int64_t part_rows, spill;  // partial rows, spilled floats
  int64_t exact_rows;        // partial rows with a Z of unrounded weights (bf16 with alpha: all of them, else none)
  int64_t units;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct TileShape {
  int rows, tpg;     // rows of a tile, tiles of a row group
  int slots;         // units the device runs at once
  int unit_cost;     // fixed time of a unit, in key blocks (a block: 64 KB of K and V at d = 128)
};
// bf16: one CTA per SM; a unit's end takes about 2 us, a block about 1.5 us.
// fp32: two 64-row CTAs per SM, whose blocks take several times as long.
TileShape tile_shape(int dtype) {
  if (dtype == TKV_DTYPE_BF16) return {kMmaRows, 2, kSms, 2};
  return {kFmaRows, 1, 2 * kSms, 1};
}

struct SegWork {
  int64_t groups, most, blocks;  // row groups; key blocks of the longest; of all of them
};
SegWork seg_work(const TileParams& p, const TileSeg& s, const TileShape& ts) {
  SegWork w{0, 0, 0};
  if (s.ntok == 0 || (s.nkeys == 0 && p.paged)) return w;
  const int64_t per = static_cast<int64_t>(ts.rows) * ts.tpg, rows = static_cast<int64_t>(s.ntok) * p.G;
  w.groups = ceil_div(rows, per);
  w.most = ceil_div(s.nkeys, kKeyBlock);
  // a causal segment's groups see from see0 to all of its keys, evenly spread
  w.blocks = p.causal ? ceil_div(w.groups * (s.see0 + s.nkeys), 2 * kKeyBlock) : w.groups * w.most;
  return w;
}

// What a unit costs beside its blocks, in blocks: the fixed part (half of it for
// a tile of few rows), and its partial rows written and read again where keys are split.
double unit_cost(const TileShape& ts, int64_t rows, bool split) {
  const int64_t most = static_cast<int64_t>(ts.rows) * ts.tpg;
  return ts.unit_cost * (rows <= ts.rows ? 0.5 : 1.0) + (split ? static_cast<double>(std::min(rows, most)) / 96 : 0.0);
}

// Segments whose ranges are cut to one length, the last taking the rest: the rest
// fills the places that whole waves leave (512 tokens behind 15872 cached, 64
// units of 128 blocks on 152 SMs: ranges of 57, 57 and 14 against two of 64, 114 us
// against 121). Even ranges where the rows of a group see very different numbers of
// keys, or keys are few.
bool leads(const TileParams& p, int i) {
  return p.causal ? p.seg[i].see0 >= p.seg[i].nkeys / 2 : p.paged && i == 0;
}

// A segment whose keys are not split, in a call where others are: its units write
// the output themselves (a 2048-token prompt beside one token behind 32768 keys,
// 28 / 4 heads: 78 -> 46 us), unless its rows are one tile, which a pair finishes
// sooner by way of partials.
bool whole_is_direct(const TileParams& p, const TileSeg& s, const TileShape& ts) {
  return !p.paged && (ts.tpg == 1 || static_cast<int64_t>(s.ntok) * p.G > ts.rows);
}

// Key blocks per unit. Units are handed out longest first to `slots` places, so
// the time is about the larger of what one place gets on average and of the
// waves the longest kind of unit makes. Rows alone leave a decode step, or a
// short piece of a prompt, with a few long units: then keys are split, and the
// candidate with the shortest time wins. More than four waves are split only where a
// unit would pass kMaxUnitKeys.
int64_t blocks_per_unit(const TileParams& p, const SegWork* w, const TileShape& ts) {
  int64_t whole = 0, most = 1, blocks = 0;
  struct Live {
    int64_t units;         // with keys whole
    double whole, split;   // what a unit costs beside its blocks
    uint32_t most;
    bool lead, direct;     // direct: writes the output where its keys are whole
  } live[kMaxSegs];
  int nlive = 0;
  for (int i = 0; i < p.nseg; ++i) {
    if (!w[i].groups) continue;
    whole += w[i].groups * p.Hkv;
    most = std::max(most, w[i].most);
    blocks += w[i].blocks * p.Hkv;
    const int64_t rows = static_cast<int64_t>(p.seg[i].ntok) * p.G;
    live[nlive++] = {w[i].groups * p.Hkv, unit_cost(ts, rows, false), unit_cost(ts, rows, true), static_cast<uint32_t>(w[i].most), leads(p, i),
                     whole_is_direct(p, p.seg[i], ts)};
  }
  const int64_t uncut = most;
  most = std::min<int64_t>(most, kMaxUnitKeys / kKeyBlock);
  if (whole >= 4 * ts.slots) return most;
  // candidates: keys whole, and around what each place gets if all is even
  const int64_t even = std::max<int64_t>(1, ceil_div(blocks, ts.slots));
  int64_t best = most;
  double best_time = 1e300;
  constexpr int kSixteenths[] = {8, 12, 16, 17, 18, 20, 24, 32, 48, 64};
  int64_t last = 0;
  for (int c = -1; c < 10; ++c) {
    const int64_t per = c < 0 ? most : std::max<int64_t>(1, even * kSixteenths[c] / 16);
    if (per > most || per == last) continue;
    last = per;
    const bool split = p.paged || per < uncut;
    double work = static_cast<double>(blocks), longest = 0, rest = 0;
    int64_t n_longest = 0, n_rest = 0;
    for (int i = 0; i < nlive; ++i) {
      const Live& l = live[i];
      const double cost = split && !(l.direct && l.most <= per) ? l.split : l.whole;
      double time = static_cast<double>(l.most) + cost;
      int64_t units = l.units, n = units;
      if (l.most > per) {
        const uint32_t cut = static_cast<uint32_t>(per), parts = (l.most + cut - 1) / cut, left = l.most % cut;
        units *= parts;
        if (l.lead && left) {
          n = units - l.units;
          time = static_cast<double>(cut) + cost;
          if (!p.paged) rest = std::max(rest, static_cast<double>(left) + cost), n_rest += l.units;
        } else {
          n = units;
          time = static_cast<double>((l.most + parts - 1) / parts) + cost;
        }
      }
      work += cost * units;
      if (time > longest * 1.01) longest = time, n_longest = n;
      else if (time > longest * 0.99) n_longest += n;
    }
    double time = std::max(work / ts.slots, longest * ceil_div(n_longest, ts.slots));
    if (n_rest && n_longest < ts.slots)  // the rests run beside the one wave, in rounds of their own
      time = std::max(time, std::min(rest * ceil_div(n_rest, ts.slots - n_longest), longest + rest));
    if (!p.paged && split) time += ts.unit_cost;  // the merge
    if (time < best_time * 0.999) {
      best_time = time;
      best = per;
    }
  }
  return best;
}

// Cuts the segments (tok0, ntok, nkeys, see0 set) into units.
TilePlan plan_units(TileParams& p, int dtype, bool want_alpha) {
  const TileShape ts = tile_shape(dtype);
  TilePlan out{};
  SegWork work[kMaxSegs];
  p.tile_rows = ts.rows;
  p.tpg = ts.tpg;
  bool split = p.paged;
  for (int i = 0; i < p.nseg; ++i) work[i] = seg_work(p, p.seg[i], ts);
  const int64_t per = blocks_per_unit(p, work, ts);
  for (int i = 0; i < p.nseg; ++i) split |= work[i].groups && work[i].most > per;
  p.merge_tokens = p.paged ? p.seg[0].ntok : 0;
  int live = 0;
  for (int i = 0; i < p.nseg; ++i) {
    p.seg[i].splits = work[i].groups ? (split ? static_cast<int32_t>(std::max<int64_t>(1, ceil_div(work[i].most, per))) : 1) : 0;
    p.seg[i].lead = p.seg[i].splits > 1 && leads(p, i) ? static_cast<int32_t>(per) : 0;
    live += work[i].groups > 0;
  }
  struct Length {
    int64_t blocks, groups;
    TileParams::Band band;
  } bands[kMaxBands];
  p.nbands = 0;
  for (int i = 0; i < p.nseg; ++i) {
    const int64_t groups = work[i].groups;
    if (!groups) continue;
    const int64_t cut = p.causal ? std::min<int64_t>(groups, kMaxBands / live / 2) : 1, rows = static_cast<int64_t>(ts.rows) * ts.tpg;
    const int32_t splits = p.seg[i].splits, lead = p.seg[i].lead;
    for (int64_t j = 0; j < cut; ++j) {
      const int64_t top = groups - 1 - groups * j / cut, count = top - (groups - 1 - groups * (j + 1) / cut);
      const int64_t seen = p.causal ? std::min<int64_t>(p.seg[i].nkeys, p.seg[i].see0 + ((top + 1) * rows - 1) / p.G + 1) : p.seg[i].nkeys;
      const int64_t nb = ceil_div(seen, kKeyBlock);
      if (lead) {
        bands[p.nbands++] = {std::min<int64_t>(nb, lead), count, {0, static_cast<int32_t>(top), i, 0, splits - 1}};
        bands[p.nbands++] = {std::max<int64_t>(0, nb - static_cast<int64_t>(splits - 1) * lead), count, {0, static_cast<int32_t>(top), i, splits - 1, 1}};
      } else {
        bands[p.nbands++] = {ceil_div(nb, splits), count, {0, static_cast<int32_t>(top), i, 0, splits}};
      }
    }
  }
  std::sort(bands, bands + p.nbands, [](const Length& a, const Length& b) {
    if (a.blocks != b.blocks) return a.blocks > b.blocks;
    if (a.band.seg != b.band.seg) return a.band.seg < b.band.seg;
    return a.band.top != b.band.top ? a.band.top > b.band.top : a.band.split0 < b.band.split0;
  });
  for (int i = 0; i < p.nbands; ++i) {
    p.band[i] = bands[i].band;
    p.band[i].first_unit = static_cast<int32_t>(std::min<int64_t>(out.units, INT32_MAX));
    out.units += bands[i].groups * p.Hkv * bands[i].band.splits;
  }
  for (int i = 0; i < p.nseg; ++i) {
    TileSeg& s = p.seg[i];
    s.part0 = out.part_rows;
    s.spill0 = -1;
    s.groups = s.part_rows = s.pair = s.direct = 0;
    if (!work[i].groups) continue;
    s.groups = static_cast<int32_t>(work[i].groups);
    const int64_t rows = static_cast<int64_t>(s.ntok) * p.G;
    s.direct = s.splits == 1 && (!split || whole_is_direct(p, s, ts));
    s.pair = !s.direct && ts.tpg == 2 && rows <= ts.rows;
    s.part_rows = static_cast<int32_t>(std::min<int64_t>(ts.rows, rows));
    if (!s.direct) {
      out.part_rows += static_cast<int64_t>(s.groups) * p.Hkv * s.splits * ts.tpg * s.part_rows;
      if (!p.paged) p.merge_tokens += s.ntok;
    }
    if (want_alpha && p.paged && i > 0) {
      s.spill0 = out.spill;
      out.spill += static_cast<int64_t>(s.nkeys) * p.Hq;
    }
  }
  // the units write it for every partial, the prefix's too, whether or not a sequence has slots of its own
  out.exact_rows = want_alpha && dtype == TKV_DTYPE_BF16 ? out.part_rows : 0;
  return out;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

struct TileScratch {
  size_t o_m, o_z, o_ze, o_spill, bytes;
};
TileScratch tile_scratch(const TilePlan& pl, int D) {
  const size_t column = align256(static_cast<size_t>(pl.part_rows) * 4);
  TileScratch s;
  s.o_m = align256(static_cast<size_t>(pl.part_rows) * D * 4);
  s.o_z = s.o_m + column;
  s.o_ze = s.o_z + column;
  s.o_spill = s.o_ze + align256(static_cast<size_t>(pl.exact_rows) * 4);
  s.bytes = s.o_spill + align256(static_cast<size_t>(pl.spill) * 4);
  return s;
}

int check_heads(int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype) {
  if (Hkv < 1 || Hq < 1 || Hkv > 65535 || Hq % Hkv || Hq / Hkv > kMaxGroup)
    return report(TKV_ERR_INVALID_ARG, "n_q_heads must be 1 to %d times n_kv_heads", kMaxGroup);
  if (D != 64 && D != 128) return report(TKV_ERR_INVALID_ARG, "head_dim must be 64 or 128");
  if (dtype != TKV_DTYPE_F32 && dtype != TKV_DTYPE_BF16) return report(TKV_ERR_INVALID_ARG, "kv_dtype");
  return TKV_OK;
}

// A call runs in rounds, nearly always one. A sequence of more than kMaxUnitKeys
// keys has its keys split however many rows there are, and partials of all its rows
// at once could be larger than the cache (70 GB for 2^20 tokens of 32 heads, d 128):
// each round takes as many tokens of such sequences as make four waves of tiles,
// and the rounds share the scratch.
int plan_prompt(TileParams& p, TilePlan* plan, int32_t batch, const int32_t* q_lens, const int32_t* k_lens, int32_t Hq,
                int32_t Hkv, int32_t D, int32_t dtype, int round, int* rounds, int64_t* tokens, int64_t* keys) {
  if (batch < 1 || batch > kMaxBatch) return report(TKV_ERR_INVALID_ARG, "batch must be 1 to %d", kMaxBatch);
  if (int st = check_heads(Hq, Hkv, D, dtype)) return st;
  if (!q_lens || !k_lens) return report(TKV_ERR_INVALID_ARG, "null pointer");
  p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv;
  p.causal = 1;
  p.nseg = batch;
  p.qscale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
  const TileShape ts = tile_shape(dtype);
  int64_t taking_turns = 0;
  for (int i = 0; i < batch; ++i) taking_turns += k_lens[i] > kMaxUnitKeys;
  const int64_t round_tokens = ceil_div(int64_t(4) * ts.slots * ts.rows * ts.tpg, Hq * std::max<int64_t>(1, taking_turns));  // of each
  int64_t tq = 0, tk = 0;
  *rounds = 1;
  for (int i = 0; i < batch; ++i) {
    if (q_lens[i] < 0 || k_lens[i] < q_lens[i]) return report(TKV_ERR_INVALID_ARG, "sequence %d: 0 <= q_len <= k_len", i);
    if (k_lens[i] > kMaxPromptKeys) return report(TKV_ERR_INVALID_ARG, "sequence %d: k_len above 2^26", i);
    int64_t first = round > 0 ? q_lens[i] : 0, last = q_lens[i];  // the tokens taken now
    if (k_lens[i] > kMaxUnitKeys) {
      first = std::min(last, round * round_tokens);
      last = std::min(last, first + round_tokens);
      *rounds = std::max(*rounds, static_cast<int>(ceil_div(q_lens[i], round_tokens)));
    }
    p.seg[i].tok0 = static_cast<int32_t>(tq + first);
    p.seg[i].ntok = static_cast<int32_t>(last - first);
    p.seg[i].key0 = tk;
    p.seg[i].see0 = static_cast<int32_t>(k_lens[i] - q_lens[i] + first);
    p.seg[i].nkeys = p.seg[i].see0 + p.seg[i].ntok;
    tq += q_lens[i];
    tk += k_lens[i];
    if (tq * p.G > INT32_MAX || tk > INT32_MAX - 2 * kKeyBlock)
      return report(TKV_ERR_INVALID_ARG, "more than 2^31 rows or keys in one call");
  }
  *tokens = tq;
  *keys = tk;
  *plan = plan_units(p, dtype, false);
  if (plan->units > INT32_MAX) return report(TKV_ERR_INVALID_ARG, "more than 2^31 units of work in one call");
  p.units = static_cast<int32_t>(plan->units);
  return TKV_OK;
}

int plan_shared(TileParams& p, TilePlan* plan, int32_t batch, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype,
                const int32_t* page_counts, int32_t max_pages, int32_t shared_pages, int want_alpha) {
  if (batch < 1 || batch > kMaxBatch) return report(TKV_ERR_INVALID_ARG, "batch must be 1 to %d", kMaxBatch);
  if (int st = check_heads(Hq, Hkv, D, dtype)) return st;
  if (max_pages < 1 || max_pages > kMaxSeqPages) return report(TKV_ERR_INVALID_ARG, "max_pages must be 1 to %d", kMaxSeqPages);
  if (!page_counts) return report(TKV_ERR_INVALID_ARG, "null pointer");
  if (shared_pages < 0 || shared_pages > max_pages) return report(TKV_ERR_INVALID_ARG, "shared_pages out of 0..max_pages");
  p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv;
  p.paged = 1;
  p.nseg = batch + 1;
  p.qscale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
  p.seg[0].ntok = batch;
  p.seg[0].nkeys = shared_pages * kPage;
  for (int b = 0; b < batch; ++b) {
    if (page_counts[b] < shared_pages || page_counts[b] > max_pages)
      return report(TKV_ERR_INVALID_ARG, "page_counts[%d] out of shared_pages..max_pages", b);
    TileSeg& s = p.seg[b + 1];
    s.tok0 = b;
    s.ntok = 1;
    s.key0 = static_cast<int64_t>(b) * max_pages + shared_pages;
    s.nkeys = (page_counts[b] - shared_pages) * kPage;
  }
  *plan = plan_units(p, dtype, want_alpha != 0);
  if (plan->units > INT32_MAX) return report(TKV_ERR_INVALID_ARG, "more than 2^31 units of work in one call");
  p.units = static_cast<int32_t>(plan->units);
  return TKV_OK;
}

template <int D>
cudaError_t launch_fma(const TileParams& p, cudaStream_t s) {
  constexpr int bytes = (kFmaRows + 2 * kFmaKeys) * (D + 4) * 4;
  static SharedMemoryOptIn opt_in;
  const cudaError_t e = opt_in.once(reinterpret_cast<const void*>(tile_fma_kernel<D>), bytes);
  if (e != cudaSuccess) return e;
  tile_fma_kernel<D><<<static_cast<unsigned>(p.units), kFmaThreads, bytes, s>>>(p);
  return cudaGetLastError();
}

// The merge may start while the units' kernel ends; it waits for it before it reads.
template <typename T, int D>
cudaError_t launch_merge(const TileParams& p, cudaStream_t s) {
  int parts = 0, slots = 0;  // most partials of a row, most own slots of a sequence
  for (int i = 0; i < p.nseg; ++i) {
    const int n = p.seg[i].splits * (p.seg[i].pair ? 2 : 1) + (p.paged && i > 0 ? p.seg[0].splits * (p.seg[0].pair ? 2 : 1) : 0);
    parts = std::max(parts, n);
    if (p.paged && i > 0) slots = std::max(slots, p.seg[i].nkeys);
  }
  const int64_t tokens = p.merge_tokens, rows = tokens * p.Hq;
  const bool share = parts >= kShareParts && rows <= kShareRows;
  const int64_t row_ctas = share ? rows : ceil_div(rows, kMergeWarps);
  const int64_t alpha_ctas = p.alpha ? tokens * p.Hkv * ceil_div(slots, kAlphaSlots) : 0;
  if (rows > INT32_MAX || row_ctas + alpha_ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(row_ctas + alpha_ctas));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.units > 0 ? 1 : 0;
  return share ? cudaLaunchKernelEx(&cfg, tile_merge_kernel<T, D, kMergeWarps>, p, static_cast<uint32_t>(rows), static_cast<int>(row_ctas))
               : cudaLaunchKernelEx(&cfg, tile_merge_kernel<T, D, 1>, p, static_cast<uint32_t>(rows), static_cast<int>(row_ctas));
}

template <typename T>
cudaError_t launch_tiles(const TileParams& p, int D, int64_t keys, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p.units > 0) {
    if (sizeof(T) == 2) e = launch_tile_mma(p, D, keys, s);
    else e = D == 64 ? launch_fma<64>(p, s) : launch_fma<128>(p, s);
    if (e != cudaSuccess) return e;
  }
  if (p.merge_tokens > 0) e = D == 64 ? launch_merge<T, 64>(p, s) : launch_merge<T, 128>(p, s);
  return e;
}

cudaError_t launch_dtype(const TileParams& p, int dtype, int D, int64_t keys, cudaStream_t s) {
  return dtype == TKV_DTYPE_BF16 ? launch_tiles<__nv_bfloat16>(p, D, keys, s) : launch_tiles<float>(p, D, keys, s);
}

thread_local uint64_t g_stall_limit_ns = 0;  // tkv_test_stall_next_tiles

void set_waits(TileParams& p, int32_t dtype) {
  p.wait_limit_ns = 2000000000ull;
  p.stall = 0;
  if (g_stall_limit_ns && dtype == TKV_DTYPE_BF16) {
    p.wait_limit_ns = g_stall_limit_ns;
    p.stall = 1;
    g_stall_limit_ns = 0;
  }
}

// Words that waits raise in calls without a status word of their own: one per
// device, in mapped host memory, so that a later call finds one raised without
// waiting for the device. Made by the first call, which may be captured.
constexpr int kWordDevices = 64;
std::mutex g_words_mu;
int32_t* g_words = nullptr;

int device_word(int32_t** word) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev >= kWordDevices) return report(TKV_ERR_INVALID_ARG, "device index above %d", kWordDevices - 1);
  std::lock_guard<std::mutex> lock(g_words_mu);
  if (e == cudaSuccess && !g_words) {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // of this thread, for the allocation
    void* made = nullptr;
    e = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e == cudaSuccess) {
      e = cudaHostAlloc(&made, kWordDevices * sizeof(int32_t), cudaHostAllocPortable | cudaHostAllocMapped);
      const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
      if (e == cudaSuccess) e = back;
    }
    if (e == cudaSuccess) {
      g_words = static_cast<int32_t*>(made);
      std::fill(g_words, g_words + kWordDevices, 0);
    }
  }
  if (e != cudaSuccess) return report(TKV_ERR_CUDA, "status word of the device: %s", cudaGetErrorString(e));
  *word = g_words + dev;
  return TKV_OK;
}

// TKV_ERR_TIMEOUT, once, if an earlier call's wait on the current device raised its word.
int raised(int32_t* word) {
  if (__atomic_load_n(word, __ATOMIC_RELAXED) == 0) return TKV_OK;
  __atomic_store_n(word, 0, __ATOMIC_RELAXED);
  return report(TKV_ERR_TIMEOUT, "a bounded device wait of an earlier attention call gave up: rows of its output are not valid");
}

// The word for a call's waits: the caller's, or the device's.
int bind_status(TileParams& p, int32_t* status) {
  int32_t* word;
  if (int st = device_word(&word)) return st;
  if (int st = raised(word)) return st;
  p.status = status ? status : word;
  return TKV_OK;
}

bool misaligned(const void* ptr, size_t to) { return reinterpret_cast<uintptr_t>(ptr) % to != 0; }

int bind_scratch(TileParams& p, const TilePlan& plan, int D, void* scratch, size_t bytes) {
  const TileScratch s = tile_scratch(plan, D);
  if (s.bytes == 0) return TKV_OK;
  if (!scratch) return report(TKV_ERR_INVALID_ARG, "null scratch: need %zu bytes", s.bytes);
  if (bytes < s.bytes) return report(TKV_ERR_CAPACITY, "scratch too small: need %zu bytes", s.bytes);
  if (misaligned(scratch, 256)) return report(TKV_ERR_INVALID_ARG, "scratch not 256-byte aligned");
  char* at = static_cast<char*>(scratch);
  p.part_o = reinterpret_cast<float*>(at);
  p.part_m = reinterpret_cast<float*>(at + s.o_m);
  p.part_z = reinterpret_cast<float*>(at + s.o_z);
  p.part_ze = plan.exact_rows ? reinterpret_cast<float*>(at + s.o_ze) : p.part_z;
  p.spill = reinterpret_cast<float*>(at + s.o_spill);
  return TKV_OK;
}

}  // namespace
}  // namespace tkv

using namespace tkv;

extern "C" {

tkv_status tkv_prompt_attention_scratch_size(int32_t batch, const int32_t* q_lens, const int32_t* k_lens,
                                             int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t kv_dtype,
                                             size_t* scratch_bytes) {
  if (!scratch_bytes) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  TileParams p{};
  TilePlan plan;
  int64_t tq, tk;
  int rounds = 1;
  size_t most = 0;
  for (int round = 0; round < rounds; ++round) {
    if (int st = plan_prompt(p, &plan, batch, q_lens, k_lens, n_q_heads, n_kv_heads, head_dim, kv_dtype, round, &rounds, &tq, &tk))
      return tkv_status(st);
    most = std::max(most, tile_scratch(plan, head_dim).bytes);
  }
  *scratch_bytes = most;
  return TKV_OK;
}

tkv_status tkv_prompt_attention(int32_t batch, const int32_t* q_lens, const int32_t* k_lens, int32_t n_q_heads,
                                int32_t n_kv_heads, int32_t head_dim, int32_t kv_dtype, const void* q, int64_t q_stride,
                                const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* out,
                                int64_t out_stride, void* scratch, size_t scratch_bytes, int32_t* status,
                                tkv_stream stream) {
  TileParams p{};
  TilePlan plan;
  int64_t tq, tk;
  int rounds;
  auto plan_round = [&](int round) {
    return plan_prompt(p, &plan, batch, q_lens, k_lens, n_q_heads, n_kv_heads, head_dim, kv_dtype, round, &rounds, &tq, &tk);
  };
  if (int st = plan_round(0)) return tkv_status(st);
  if (tq == 0) return TKV_OK;
  if (!q || !k || !v || !out) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  const int64_t unit = kv_dtype == TKV_DTYPE_BF16 ? 8 : 4;  // elements of 16 bytes
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(out, 16))
    return tkv_status(report(TKV_ERR_INVALID_ARG, "q, k, v and out must be 16-byte aligned"));
  const int64_t qrow = static_cast<int64_t>(n_q_heads) * head_dim, krow = static_cast<int64_t>(n_kv_heads) * head_dim;
  if (q_stride < qrow || out_stride < qrow || k_stride < krow || v_stride < krow || q_stride % unit || out_stride % unit ||
      k_stride % unit || v_stride % unit || (q_stride | out_stride | k_stride | v_stride) >> 36)
    return tkv_status(report(TKV_ERR_INVALID_ARG, "token strides must hold a token and be multiples of 16 bytes"));
  // planned from the end: nothing is launched unless the scratch is enough for all of it
  for (int round = rounds - 1; round >= 0; --round) {
    if (rounds > 1)
      if (int st = plan_round(round)) return tkv_status(st);
    if (int st = bind_scratch(p, plan, head_dim, scratch, scratch_bytes)) return tkv_status(st);
  }
  if (int st = bind_status(p, status)) return tkv_status(st);
  for (int round = 0; round < rounds; ++round) {
    if (round > 0) {
      if (int st = plan_round(round)) return tkv_status(st);
      if (int st = bind_scratch(p, plan, head_dim, scratch, scratch_bytes)) return tkv_status(st);
    }
    p.q = q; p.q_stride = q_stride;
    p.k = k; p.k_stride = k_stride;
    p.v = v; p.v_stride = v_stride;
    p.out = out; p.out_stride = out_stride;
    p.out_sectors = !misaligned(out, 32) && out_stride % (2 * unit) == 0;
    set_waits(p, kv_dtype);
    const cudaError_t e = launch_dtype(p, kv_dtype, head_dim, tk, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return tkv_status(report(TKV_ERR_CUDA, "prompt attention launch failed: %s", cudaGetErrorString(e)));
  }
  return TKV_OK;
}

tkv_status tkv_attention_synchronize(tkv_stream stream) {
  const cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return tkv_status(report(TKV_ERR_CUDA, "cudaStreamSynchronize failed: %s", cudaGetErrorString(e)));
  int32_t* word;
  if (int st = device_word(&word)) return tkv_status(st);
  return tkv_status(raised(word));
}

tkv_status tkv_test_stall_next_tiles(uint64_t wait_limit_ns) {
  if (wait_limit_ns < 1000000ull || wait_limit_ns > 2000000000ull)
    return tkv_status(report(TKV_ERR_INVALID_ARG, "wait limit out of 1 ms .. 2 s"));
  g_stall_limit_ns = wait_limit_ns;
  return TKV_OK;
}

tkv_status tkv_shared_prefix_attention_scratch_size(int32_t batch, int32_t n_q_heads, int32_t n_kv_heads,
                                                    int32_t head_dim, int32_t kv_dtype, const int32_t* page_counts,
                                                    int32_t max_pages, int32_t shared_pages, int32_t want_alpha,
                                                    size_t* scratch_bytes) {
  if (!scratch_bytes) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  TileParams p{};
  TilePlan plan;
  if (int st = plan_shared(p, &plan, batch, n_q_heads, n_kv_heads, head_dim, kv_dtype, page_counts, max_pages, shared_pages,
                           want_alpha))
    return tkv_status(st);
  *scratch_bytes = tile_scratch(plan, head_dim).bytes;
  return TKV_OK;
}

tkv_status tkv_shared_prefix_attention(int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                       int32_t kv_dtype, const void* q, const void* pool, int64_t pool_pages,
                                       const int32_t* page_table, const uint32_t* slot_mask, const int32_t* page_counts,
                                       int32_t max_pages, int32_t shared_pages, void* out, float* alpha_sum,
                                       void* scratch, size_t scratch_bytes, int32_t* status, tkv_stream stream) {
  TileParams p{};
  TilePlan plan;
  if (int st = plan_shared(p, &plan, batch, n_q_heads, n_kv_heads, head_dim, kv_dtype, page_counts, max_pages, shared_pages,
                           alpha_sum != nullptr))
    return tkv_status(st);
  if (!q || !pool || !page_table || !slot_mask || !out) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  if (pool_pages < 1 || pool_pages > (int64_t(1) << 29) / n_kv_heads)
    return tkv_status(report(TKV_ERR_INVALID_ARG, "pool_pages x n_kv_heads must be 1 to 2^29"));
  if (misaligned(q, 16) || misaligned(pool, 16) || misaligned(out, 16) || misaligned(alpha_sum, 16))
    return tkv_status(report(TKV_ERR_INVALID_ARG, "q, pool, out and alpha_sum must be 16-byte aligned"));
  if (int st = bind_scratch(p, plan, head_dim, scratch, scratch_bytes)) return tkv_status(st);
  p.q = q; p.q_stride = static_cast<int64_t>(n_q_heads) * head_dim;
  p.out = out; p.out_stride = p.q_stride;
  p.out_sectors = !misaligned(out, 32);
  p.pool = pool;
  p.pages = pool_pages;
  p.table = page_table;
  p.mask = slot_mask;
  p.alpha = alpha_sum;
  p.alpha_stride_h = static_cast<int64_t>(max_pages) * kPage;
  p.alpha_first = static_cast<int64_t>(shared_pages) * kPage;
  if (int st = bind_status(p, status)) return tkv_status(st);
  set_waits(p, kv_dtype);
  const cudaError_t e = launch_dtype(p, kv_dtype, head_dim, 0, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess)
    return tkv_status(report(TKV_ERR_CUDA, "shared-prefix attention launch failed: %s", cudaGetErrorString(e)));
  return TKV_OK;
}

}  // extern "C"
