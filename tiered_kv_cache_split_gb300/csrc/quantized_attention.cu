// Decode attention over a paged cache held in 8 bits (quantized.h): one query
// token per sequence, the G query heads of a KV head together, so that a code is
// read once.
//
// HBM bounds it: 2 D code bytes and half a byte of scales per token and KV head.
// The G heads are too few for tcgen05 (its smallest M is 64, and S would go
// through TMEM for every 16 keys), so the products run on mma.sync m16n8k16 with
// the codes as the 16-row operand and the heads as the 8 columns:
//   S^T [16 keys][8] = K codes [16][D] x Q^T,   O^T [D][8] += V^T codes x P^T.
// Codes are exact in fp16 (a byte put under the exponent of 1024 by a byte
// permute, 1152 taken off), so nothing is lost on that side. A column holds:
//   bf16  a query head, scaled by a power of two to at most 2 (exact in fp16
//         but for elements 2^-14 below the row's largest);
//   fp32  one of two fp16 parts of a head, hi and (x - hi) * 2^11, next to each
//         other: both lie in the same thread, and their sum has 22 bits.
// The softmax weights go into the second product the same way. Logits, maxima, sums and
// accumulators are fp32.
//
// The scale of K multiplies a page's logits. That of V multiplies its weights: a
// weight is 2^(l + k + 13 - r) f with V's scale f 2^k, and r a running maximum
// of l + k of its own, so that pages whose scales are far apart lose nothing in
// fp16 (weights down to 2^-38 of the largest count). Z sums 2^(l - m) as always.
// Both references rise only when a logit passes them by more than 1 (a vote per
// page), so the shuffles and the rescaling are rare.
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "quantized.h"
#include "tile_attention.h"  // SharedMemoryOptIn

namespace tkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnitPages = 384;     // most pages of a unit: what its shared memory describes
constexpr int kMergeThreads = 128;
constexpr int kAlphaSlots = 1024;   // slots of an alpha CTA
constexpr int kSms = 152;
constexpr float kNegInf = -INFINITY;
constexpr float kWeightBits = 13.f; // weights are at most 2^15: reference lag and f below 2 each

template <typename T> struct Columns;  // heads of an 8-column tile, and columns of a head
template <> struct Columns<__nv_bfloat16> { static constexpr int heads = 8, parts = 1; };
template <> struct Columns<float> { static constexpr int heads = 4, parts = 2; };

struct AttendParams {
  PoolRef p;
  const void* q;
  void* out;
  float* alpha;             // [B][Hkv][max_pages * 16], or null
  float* part_o;            // [chunk][Hq][D]
  float4* part_m;           // [chunk][Hq]: maximum, V's reference, sum
  float* spill;             // [page of the call][Hkv][16][columns of heads], logits in base 2
  int32_t B, Hq, G, groups; // groups: head groups of a KV head, each a unit of its own
  int32_t max_pages;
  int32_t units;
  float qscale;             // log2(e) / sqrt(D)
  int32_t count[kMaxBatch];            // pages
  int32_t order[kMaxBatch];            // sequences by decreasing pages per unit
  int32_t order_first[kMaxBatch + 1];  // prefix sums of their chunks in that order
  int32_t chunk0[kMaxBatch + 1];       // prefix sums of the chunks by sequence
  int32_t page0[kMaxBatch + 1];        // prefix sums of the pages
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^x in two halves, for x where one would leave fp32's normal range
__device__ __forceinline__ float times_ex2(float v, float x) {
  const float h = exp2f(0.5f * x);
  return v * h * h;
}
__device__ __forceinline__ float finite_or_nan(float x) { return fabsf(x) < INFINITY ? x : NAN; }
__device__ __forceinline__ void put4(float* at, float4 x) { *reinterpret_cast<float4*>(at) = x; }
__device__ __forceinline__ void put4(__nv_bfloat16* at, float4 x) {
  __nv_bfloat162 v[2] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(x.z, x.w)};
  *reinterpret_cast<uint2*>(at) = *reinterpret_cast<const uint2*>(v);
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// two code bytes (biased by 128) of x as fp16 codes
template <int kSelect>
__device__ __forceinline__ uint32_t codes2(uint32_t x) {
  const uint32_t y = __byte_perm(x, 0x64646464u, kSelect);  // 1024 + byte
  const uint32_t bias = 0x64806480u;                        // 1152
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&y), *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&h);
}
constexpr int kLow = 0x4140, kHigh = 0x4342;

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;"); }
template <int N> __device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// What a unit keeps of a page: id (-1: none of its slots counts), valid slots and
// the power k of V's scale, K's scale in the logits' units, and V's scale as f in f 2^k.
__device__ __forceinline__ int4 page_info(const AttendParams& p, int b, int page, int h) {
  const int32_t id = p.p.table[b * p.p.table_stride + page];
  if (id < 0 || id >= p.p.pages) return make_int4(-1, 0, 0, 0);
  const uint32_t live = p.p.mask[id] & kFullMask;
  if (!live) return make_int4(-1, 0, 0, 0);
  const float2 s = *reinterpret_cast<const float2*>(p.p.scales + (static_cast<int64_t>(id) * p.p.hkv + h) * 2);
  float f = finite_or_nan(s.y);
  int k = -126;                                  // of 0 and NaN: no reference rises for them
  if (f > 0.f) {
    const bool small = f < 0x1p-100f;
    const uint32_t bits = __float_as_uint(small ? f * 0x1p40f : f);
    k = static_cast<int>(bits >> 23) - 127 - (small ? 40 : 0);
    f = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
  }
  return make_int4(id, static_cast<int>(live | static_cast<uint32_t>(k + 256) << 16), __float_as_int(finite_or_nan(s.x) * p.qscale),
                   __float_as_int(f));
}

template <int D>
struct Ring {
  static constexpr int page_bytes = 2 * kPage * D;                    // a head's K and V codes
  static constexpr int stages = D == 128 ? 3 : 6;                     // 12 KB per warp
  static constexpr int bytes = kWarps * stages * page_bytes;
};

template <typename T, int D, int NT>
struct Smem {
  static constexpr int heads = Columns<T>::heads * NT;
  static constexpr int out_row = D + 4;                               // floats; rows start in different banks
  static constexpr int merge_bytes = kWarps * heads * out_row * 4;
  static constexpr int o_info = Ring<D>::bytes > merge_bytes ? Ring<D>::bytes : merge_bytes;
  static constexpr int o_stat = o_info + kUnitPages * 16;
  static constexpr int bytes = o_stat + kWarps * heads * 16;
};

// Where the 16-byte chunk c of row r of a slot lies (rows 0 .. 15 are K's, 16 .. 31
// V's): rows are whole 128-byte lines on the way in, and the fragments' reads
// (below) touch every bank group once.
template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {
  if (D == 128) return r * 128 + (r < kPage ? c ^ (r & 1) << 2 : c ^ (r & 6)) * 16;
  const int u = (r & 1) * 4 + c;                                      // chunk of a pair of rows
  return (r >> 1) * 128 + (r < kPage ? u : u ^ (r & 6)) * 16;
}

// The copies of one page by one warp: 512 bytes in a row each.
template <int D>
__device__ __forceinline__ void copy_page(uint32_t to, const int8_t* block, int lane) {
  constexpr int kRowChunks = D / 16;
#pragma unroll
  for (int i = 0; i < 2 * kPage * D / 512; ++i) {
    const int at = i * 32 + lane;
    copy16(to + chunk_at<D>(at / kRowChunks, at % kRowChunks), block + at * 16);
  }
}

// A CTA per unit: pages j0 .. j1 of a sequence, a KV head and a group of its
// query heads. Page j goes to warp j % 4, which keeps 2 (D 64: 5) pages on their
// way besides the one it reads; no warp waits for another before the end.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 3) attend_quantized_kernel(const __grid_constant__ AttendParams p) {
  using S = Smem<T, D, NT>;
  using R = Ring<D>;
  constexpr int kHeads = Columns<T>::heads, kParts = Columns<T>::parts;
  constexpr int kOwn = 2 / kParts;                 // heads of a thread's column pair
  constexpr int kTiles = D / 16;
  constexpr int kChunks = D / 64;                  // 16-byte pieces of a key row per thread
  extern __shared__ __align__(128) char smem[];
  int4* s_info = reinterpret_cast<int4*>(smem + S::o_info);
  float4* s_stat = reinterpret_cast<float4*>(smem + S::o_stat);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  // the unit
  const int per_chunk = p.p.hkv * p.groups;
  const int rank = blockIdx.x / per_chunk, rest = blockIdx.x % per_chunk;
  const int h = rest / p.groups, group = rest % p.groups;
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.order_first[mid] <= rank) lo = mid; else hi = mid - 1;
  }
  const int b = p.order[lo], chunk = rank - p.order_first[lo], chunks = p.order_first[lo + 1] - p.order_first[lo];
  const int each = p.count[b] / chunks, longer = p.count[b] % chunks;
  const int j0 = chunk * each + min(chunk, longer), n = each + (chunk < longer);
  for (int i = tid; i < n; i += kThreads) s_info[i] = page_info(p, b, j0 + i, h);

  // queries: fragments of Q^T, and the power of two taken out of each head
  const int head0 = h * p.G + group * S::heads;    // first head of the group
  const int nheads = min(S::heads, p.G - group * S::heads);
  uint32_t qf[NT][kChunks * 4][2];
  float qpow[NT][kOwn];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int head = nt * kHeads + g / kParts, part = g % kParts;
    float x[kChunks * 16], top = 0.f;
    const T* q = static_cast<const T*>(p.q) + (static_cast<int64_t>(b) * p.Hq + head0 + head) * D + t * 16;
#pragma unroll
    for (int i = 0; i < kChunks * 16; i += Vec<T>::n)
      Vec<T>::unpack(head < nheads ? *reinterpret_cast<const int4*>(q + (i >> 4) * 64 + (i & 15)) : make_int4(0, 0, 0, 0), x + i);
#pragma unroll
    for (int i = 0; i < kChunks * 16; ++i) top = fmaxf(top, fabsf(x[i]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -126);
    const float down0 = __uint_as_float(static_cast<uint32_t>(127 - e / 2) << 23), down1 = __uint_as_float(static_cast<uint32_t>(127 - (e - e / 2)) << 23);
#pragma unroll
    for (int i = 0; i < kChunks * 16; i += 2) {
      float y[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        y[j] = x[i + j] * down0 * down1;
        if (kParts == 2 && part == 1) y[j] = (y[j] - __half2float(__float2half_rn(y[j]))) * 2048.f;
      }
      qf[nt][i >> 2][(i >> 1) & 1] = half2_bits(y[0], y[1]);
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int of = __shfl_sync(0xffffffffu, e, (2 * t + i) * 4);
      qpow[nt][i] = __uint_as_float(static_cast<uint32_t>(of + 127) << 23);  // infinity for a row that holds one
    }
  }

  float o[NT][kTiles][4] = {};
  float m[NT][kOwn], r[NT][kOwn], z[NT][kOwn];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < kOwn; ++i) m[nt][i] = r[nt][i] = kNegInf, z[nt][i] = 0.f;
  __syncthreads();

  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * R::stages * R::page_bytes;
  const int mine = n > warp ? (n - warp + kWarps - 1) / kWarps : 0;
  auto start = [&](int i) {                        // the copies of this warp's page i, if there is one
    if (i < mine) {
      const int id = s_info[warp + i * kWarps].x;
      if (id >= 0)
        copy_page<D>(ring + (i % R::stages) * R::page_bytes, p.p.codes + (static_cast<int64_t>(id) * p.p.hkv + h) * R::page_bytes, lane);
    }
    commit();
  };
  float* spill = p.spill ? p.spill + ((static_cast<int64_t>(p.page0[b] + j0) * p.p.hkv + h) * kPage * p.groups) * S::heads + group * S::heads : nullptr;
  const int64_t spill_page = static_cast<int64_t>(p.p.hkv) * kPage * p.groups * S::heads;
  const int spill_slot = p.groups * S::heads;
#pragma unroll
  for (int i = 0; i < R::stages - 1; ++i) start(i);
  for (int i = 0; i < mine; ++i) {
    wait_copies<R::stages - 2>();
    __syncwarp();                                  // page i is here for all lanes, and page i - 1 is read
    start(i + R::stages - 1);
    const int page = warp + i * kWarps;
    const int4 info = s_info[page];
    const uint32_t live = info.y & kFullMask;
    if (info.x < 0) {                              // an empty page: nothing was copied
      if (spill) {
        float* at = spill + page * spill_page;
        for (int w = lane; w < kPage * S::heads; w += 32) at[(w / S::heads) * spill_slot + w % S::heads] = kNegInf;
      }
      continue;
    }
    const char* slot = smem + (warp * R::stages + i % R::stages) * R::page_bytes;
    // S^T = K Q^T
    float s[NT][4] = {};
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const uint4 a = *reinterpret_cast<const uint4*>(slot + chunk_at<D>(g, c * 4 + t));
      const uint4 d = *reinterpret_cast<const uint4*>(slot + chunk_at<D>(g + 8, c * 4 + t));
      const uint32_t av[4] = {a.x, a.y, a.z, a.w}, dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x = av[w] ^ 0x80808080u, y = dv[w] ^ 0x80808080u;
        const uint32_t a0 = codes2<kLow>(x), a1 = codes2<kLow>(y), a2 = codes2<kHigh>(x), a3 = codes2<kHigh>(y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma(s[nt], a0, a1, a2, a3, qf[nt][c * 4 + w][0], qf[nt][c * 4 + w][1]);
      }
    }
    // logits (base 2) of keys g and g + 8
    const float sk = __int_as_float(info.z), f = __int_as_float(info.w);
    const float k = static_cast<float>((info.y >> 16) - 256);
    const bool live0 = live >> g & 1, live1 = live >> (g + 8) & 1;
    float l[NT][kOwn][2];
    bool rise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (kParts == 2) {
        s[nt][0] += s[nt][1] * 0x1p-11f;
        s[nt][2] += s[nt][3] * 0x1p-11f;
      }
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        l[nt][j][0] = live0 ? s[nt][j] * sk * qpow[nt][j] : kNegInf;
        l[nt][j][1] = live1 ? s[nt][2 + j] * sk * qpow[nt][j] : kNegInf;
        const float top = fmaxf(l[nt][j][0], l[nt][j][1]);
        rise |= top > m[nt][j] + 1.f || top + k > r[nt][j] + 1.f;
      }
      if (spill) {
        float* at = spill + page * spill_page + g * spill_slot + nt * kHeads + t * kOwn;
        if (kOwn == 2) {
          *reinterpret_cast<float2*>(at) = make_float2(l[nt][0][0], l[nt][kOwn - 1][0]);
          *reinterpret_cast<float2*>(at + 8 * spill_slot) = make_float2(l[nt][0][1], l[nt][kOwn - 1][1]);
        } else {
          at[0] = l[nt][0][0];
          at[8 * spill_slot] = l[nt][0][1];
        }
      }
    }
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float keep[2];
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          float top = fmaxf(l[nt][j][0], l[nt][j][1]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          const float m1 = fmaxf(m[nt][j], top), r1 = fmaxf(r[nt][j], top + k);
          z[nt][j] *= m1 == kNegInf ? 1.f : ex2(m[nt][j] - m1);
          keep[j] = r1 == kNegInf ? 1.f : ex2(r[nt][j] - r1);
          if (kOwn == 1) keep[1] = keep[0];
          m[nt][j] = m1;
          r[nt][j] = r1;
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          o[nt][i][0] *= keep[0], o[nt][i][2] *= keep[0];
          o[nt][i][1] *= keep[1], o[nt][i][3] *= keep[1];
        }
      }
    }
    // weights, and P^T as the second product takes it
    uint32_t pf[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float w[2][2];
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        const float mz = m[nt][j] == kNegInf ? 0.f : m[nt][j], ro = r[nt][j] == kNegInf ? 0.f : k + kWeightBits - r[nt][j];
        z[nt][j] += ex2(l[nt][j][0] - mz) + ex2(l[nt][j][1] - mz);
        w[0][j] = live0 ? ex2(l[nt][j][0] + ro) * f : 0.f;
        w[1][j] = live1 ? ex2(l[nt][j][1] + ro) * f : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (kParts == 2) w[i][1] = (w[i][0] - __half2float(__float2half_rn(w[i][0]))) * 2048.f;
        pf[nt][i] = transposed(half2_bits(w[i][0], w[i][1]));
      }
    }
    // O^T += V^T P^T: V's rows of four tokens, 16 (D 64: 8) of their codes
    uint32_t v[4][D / 32];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = kPage + 2 * t + (c & 1) + (c >> 1) * 8;
      if (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(slot + chunk_at<D>(row, g));
        v[c][0] = x.x, v[c][1] = x.y, v[c][D / 32 - 2] = x.z, v[c][D / 32 - 1] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(slot + chunk_at<D>(row, g >> 1) + (g & 1) * 8);
        v[c][0] = x.x, v[c][1] = x.y;
      }
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int pick = half ? 0x7362 : 0x5140;   // codes 2, 3 or 0, 1 of both tokens
        const uint32_t x = __byte_perm(v[0][w], v[1][w], pick) ^ 0x80808080u, y = __byte_perm(v[2][w], v[3][w], pick) ^ 0x80808080u;
        const uint32_t a0 = codes2<kLow>(x), a1 = codes2<kHigh>(x), a2 = codes2<kLow>(y), a3 = codes2<kHigh>(y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma(o[nt][w * 2 + half], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
      }
    }
  }
  wait_copies<0>();
  __syncthreads();                                 // the ring becomes the merge's

  // join the four warps
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) z[nt][j] += __shfl_xor_sync(0xffffffffu, z[nt][j], d);
      if (g == 0) s_stat[warp * S::heads + nt * kHeads + t * kOwn + j] = make_float4(m[nt][j], r[nt][j], z[nt][j], 0.f);
    }
  __syncthreads();
  float* s_out = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const int head = nt * kHeads + t * kOwn + j;
      float top = kNegInf;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_stat[w * S::heads + head].y);
      const float keep = r[nt][j] == kNegInf ? (z[nt][j] == z[nt][j] ? 0.f : NAN) : ex2(r[nt][j] - top);
      float* row = s_out + (warp * S::heads + head) * S::out_row + g * (D / 8);
#pragma unroll
      for (int i = 0; i < kTiles; i += 2) {
        float4 x;
        if (kParts == 2) {
          x = make_float4(o[nt][i][0] + o[nt][i][1] * 0x1p-11f, o[nt][i][2] + o[nt][i][3] * 0x1p-11f,
                          o[nt][i + 1][0] + o[nt][i + 1][1] * 0x1p-11f, o[nt][i + 1][2] + o[nt][i + 1][3] * 0x1p-11f);
        } else {
          x = make_float4(o[nt][i][j], o[nt][i][2 + j], o[nt][i + 1][j], o[nt][i + 1][2 + j]);
        }
        *reinterpret_cast<float4*>(row + i * 2) = make_float4(x.x * keep, x.y * keep, x.z * keep, x.w * keep);
      }
    }
  __syncthreads();
  const int64_t part = static_cast<int64_t>(p.chunk0[b] + chunk) * p.Hq + head0;
  for (int i = tid; i < nheads * (D / 4); i += kThreads) {
    const int head = i / (D / 4), d = i % (D / 4) * 4;
    float top = kNegInf, ref = kNegInf, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 st = s_stat[w * S::heads + head];
      top = fmaxf(top, st.x);
      ref = fmaxf(ref, st.y);
    }
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 st = s_stat[w * S::heads + head];
      sum += st.x == kNegInf ? st.z : st.z * ex2(st.x - top);
      const float4 y = *reinterpret_cast<const float4*>(s_out + (w * S::heads + head) * S::out_row + d);
      x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    if (p.part_m && d == 0) p.part_m[part + head] = make_float4(top, ref, sum, 0.f);
    if (chunks == 1) {
      const float by = sum == 0.f ? 0.f : 1.f / sum, e = sum == 0.f ? 0.f : ref - top - kWeightBits;
      put4(static_cast<T*>(p.out) + (static_cast<int64_t>(b) * p.Hq + head0 + head) * D + d,
           make_float4(times_ex2(x.x * by, e), times_ex2(x.y * by, e), times_ex2(x.z * by, e), times_ex2(x.w * by, e)));
    } else {
      *reinterpret_cast<float4*>(p.part_o + (part + head) * D + d) = x;
    }
  }
}

// Joins the chunks of a row: the first B * Hq CTAs a query head each, four
// warps taking every fourth chunk. The others (alpha) take 1024 slots of a
// sequence and KV head: the maximum and sum of each query head from its chunks,
// then the weights of the slots from their logits.
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) merge_quantized_kernel(const __grid_constant__ AttendParams p, int rows, int columns) {
  constexpr int E = D / 32;
  __shared__ float s_x[4][D];
  __shared__ float2 s_head[64];
  cudaGridDependencySynchronize();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (static_cast<int>(blockIdx.x) < rows) {
    const int b = blockIdx.x / p.Hq, hq = blockIdx.x % p.Hq;
    const int c0 = p.chunk0[b], chunks = p.chunk0[b + 1] - c0;
    T* out = static_cast<T*>(p.out) + static_cast<int64_t>(blockIdx.x) * D;
    if (chunks == 1) return;                       // written by its unit
    float m = kNegInf, r = kNegInf, z = 0.f;
    for (int c = lane; c < chunks; c += 32) {
      const float4 st = p.part_m[static_cast<int64_t>(c0 + c) * p.Hq + hq];
      m = fmaxf(m, st.x);
      r = fmaxf(r, st.y);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, d));
    }
    for (int c = lane; c < chunks; c += 32) {
      const float4 st = p.part_m[static_cast<int64_t>(c0 + c) * p.Hq + hq];
      z += st.x == kNegInf ? st.z : st.z * ex2(st.x - m);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
    float x[E] = {};
    for (int c = warp; c < chunks; c += 4) {
      const int64_t row = static_cast<int64_t>(c0 + c) * p.Hq + hq;
      const float ref = p.part_m[row].y, keep = ref == kNegInf ? 1.f : ex2(ref - r);
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] += p.part_o[row * D + i * 32 + lane] * keep;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) s_x[warp][i * 32 + lane] = x[i];
    __syncthreads();
    const float by = z == 0.f ? 0.f : 1.f / z, e = z == 0.f ? 0.f : r - m - kWeightBits;
    if (tid < D / 4) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float4 a = *reinterpret_cast<const float4*>(&s_x[w][tid * 4]);
        y.x += a.x, y.y += a.y, y.z += a.z, y.w += a.w;
      }
      put4(out + tid * 4, make_float4(times_ex2(y.x * by, e), times_ex2(y.y * by, e), times_ex2(y.z * by, e), times_ex2(y.w * by, e)));
    }
    return;
  }
  // alpha
  const int most = (p.max_pages * kPage + kAlphaSlots - 1) / kAlphaSlots;
  int at = blockIdx.x - rows;
  const int piece = at % most;
  at /= most;
  const int h = at % p.p.hkv, b = at / p.p.hkv;
  const int slots = p.count[b] * kPage, first = piece * kAlphaSlots;
  if (first >= slots) return;
  const int c0 = p.chunk0[b], chunks = p.chunk0[b + 1] - c0;
  for (int i = warp; i < p.G; i += 4) {
    const int hq = h * p.G + i;
    float m = kNegInf, z = 0.f;
    for (int c = lane; c < chunks; c += 32) m = fmaxf(m, p.part_m[static_cast<int64_t>(c0 + c) * p.Hq + hq].x);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    for (int c = lane; c < chunks; c += 32) {
      const float4 st = p.part_m[static_cast<int64_t>(c0 + c) * p.Hq + hq];
      z += st.x == kNegInf ? st.z : st.z * ex2(st.x - m);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
    if (lane == 0) s_head[i] = make_float2(m, z == 0.f ? 0.f : 1.f / z);
  }
  __syncthreads();
  float* alpha = p.alpha + (static_cast<int64_t>(b) * p.p.hkv + h) * p.max_pages * kPage;
  for (int i = first + tid; i < min(slots, first + kAlphaSlots); i += kMergeThreads) {
    const float* l = p.spill + ((static_cast<int64_t>(p.page0[b] + i / kPage) * p.p.hkv + h) * kPage + i % kPage) * columns;
    float sum = 0.f;
    bool any = false;
    for (int j = 0; j < p.G; ++j) {
      const float x = l[j];
      if (x == kNegInf) continue;
      any = true;
      sum += ex2(x - s_head[j].x) * s_head[j].y;
    }
    if (any) alpha[i] += sum;
  }
}

// ---- host side

struct Plan {
  int nt;                     // column tiles of a unit
  int heads;                  // of a unit
  bool merge;                 // some sequence has several chunks
  size_t o_m, o_spill, bytes; // scratch
};

int plan_attend(AttendParams* p, Plan* plan, int32_t batch, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype,
                const int32_t* page_counts, int32_t max_pages, bool want_alpha) {
  if (batch < 1 || batch > kMaxBatch) return report(TKV_ERR_INVALID_ARG, "batch must be 1 to %d", kMaxBatch);
  if (Hkv < 1 || Hq < 1 || Hkv > 65535 || Hq % Hkv || Hq / Hkv > 64)
    return report(TKV_ERR_INVALID_ARG, "n_q_heads must be 1 to 64 times n_kv_heads");
  if (D != 64 && D != 128) return report(TKV_ERR_INVALID_ARG, "head_dim must be 64 or 128");
  if (int st = check_dtype(dtype)) return st;
  if (max_pages < 1 || max_pages > kMaxSeqPages) return report(TKV_ERR_INVALID_ARG, "max_pages must be 1 to %d", kMaxSeqPages);
  if (!page_counts) return report(TKV_ERR_INVALID_ARG, "null pointer");
  const int tile = dtype == TKV_DTYPE_BF16 ? Columns<__nv_bfloat16>::heads : Columns<float>::heads;
  p->B = batch; p->Hq = Hq; p->G = Hq / Hkv; p->max_pages = max_pages;
  p->qscale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
  plan->nt = p->G > tile ? 2 : 1;
  plan->heads = tile * plan->nt;
  p->groups = (p->G + plan->heads - 1) / plan->heads;
  int most = 0;
  p->page0[0] = 0;
  for (int b = 0; b < batch; ++b) {
    const int n = page_counts[b];
    if (n < 0 || n > max_pages) return report(TKV_ERR_INVALID_ARG, "page_counts[%d] out of 0..max_pages", b);
    p->count[b] = n;
    p->page0[b + 1] = p->page0[b] + n;
    most = std::max(most, n);
  }
  // Pages per unit: the shortest estimated time, in pages' time of one of the CTAs
  // that run at once; a unit's start and end cost about as much as kUnitCost pages,
  // the launch that joins chunks kMergeCost.
  constexpr double kUnitCost = 7, kMergeCost = 7;
  const int64_t per_chunk = static_cast<int64_t>(Hkv) * p->groups, slots = kSms * (plan->nt == 1 ? 4 : 3);
  int best = std::min(std::max(most, 1), kUnitPages);
  double best_time = 1e300;
  for (int parts = 1; parts <= kMaxSeqPages; parts = parts < 8 ? parts + 1 : parts + parts / 8) {
    const int per = (most + parts - 1) / parts;
    if (per > kUnitPages) continue;
    if (per < 4) break;
    int64_t units = 0;
    for (int b = 0; b < batch; ++b) units += (p->count[b] + per - 1) / per;
    units *= per_chunk;
    const double work = static_cast<double>(p->page0[batch]) * per_chunk + kUnitCost * units;
    const double longest = per + kUnitCost;
    double time = units <= slots ? longest : std::max(longest, work / slots + 0.5 * longest);
    if (parts > 1) time += kMergeCost;
    if (time < best_time) best_time = time, best = per;
  }
  int chunks[kMaxBatch];
  int64_t total = 0;
  plan->merge = false;
  p->chunk0[0] = 0;
  for (int b = 0; b < batch; ++b) {
    chunks[b] = std::max(1, (p->count[b] + best - 1) / best);
    plan->merge |= chunks[b] > 1;
    total += chunks[b];
    p->chunk0[b + 1] = static_cast<int32_t>(total);
    p->order[b] = b;
  }
  std::sort(p->order, p->order + batch, [&](int a, int b) {
    const int64_t x = static_cast<int64_t>(p->count[a]) * chunks[b], y = static_cast<int64_t>(p->count[b]) * chunks[a];
    return x != y ? x > y : a < b;
  });
  p->order_first[0] = 0;
  for (int i = 0; i < batch; ++i) p->order_first[i + 1] = p->order_first[i] + chunks[p->order[i]];
  if (total * per_chunk > INT32_MAX) return report(TKV_ERR_INVALID_ARG, "more than 2^31 units of work in one call");
  p->units = static_cast<int32_t>(total * per_chunk);
  auto align = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = static_cast<size_t>(total) * Hq;
  plan->o_m = plan->merge ? align(rows * D * 4) : 0;
  plan->o_spill = plan->o_m + (plan->merge || want_alpha ? align(rows * 16) : 0);
  plan->bytes = plan->o_spill + (want_alpha ? align(static_cast<size_t>(p->page0[batch]) * Hkv * kPage * p->groups * plan->heads * 4) : 0);
  return TKV_OK;
}

template <typename T, int D, int NT>
cudaError_t launch_units(const AttendParams& p, cudaStream_t s) {
  constexpr int bytes = Smem<T, D, NT>::bytes;
  static SharedMemoryOptIn opt_in;
  const cudaError_t e = opt_in.once(reinterpret_cast<const void*>(attend_quantized_kernel<T, D, NT>), bytes);
  if (e != cudaSuccess) return e;
  attend_quantized_kernel<T, D, NT><<<static_cast<unsigned>(p.units), kThreads, bytes, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_attend(const AttendParams& p, const Plan& plan, cudaStream_t s) {
  cudaError_t e = plan.nt == 1 ? launch_units<T, D, 1>(p, s) : launch_units<T, D, 2>(p, s);
  if (e != cudaSuccess || !(plan.merge || p.alpha)) return e;
  const int64_t rows = plan.merge ? static_cast<int64_t>(p.B) * p.Hq : 0;
  const int64_t pieces = p.alpha ? static_cast<int64_t>(p.B) * p.p.hkv * ((p.max_pages * kPage + kAlphaSlots - 1) / kAlphaSlots) : 0;
  if (rows + pieces > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows + pieces));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_quantized_kernel<T, D>, p, static_cast<int>(rows), p.groups * plan.heads);
}

}  // namespace
}  // namespace tkv

using namespace tkv;

extern "C" {

tkv_status tkv_quantized_attention_scratch_size(int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                                int32_t dtype, const int32_t* page_counts, int32_t max_pages,
                                                int32_t want_alpha, size_t* scratch_bytes) {
  if (!scratch_bytes) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  AttendParams p{};
  Plan plan;
  if (int st = plan_attend(&p, &plan, batch, n_q_heads, n_kv_heads, head_dim, dtype, page_counts, max_pages, want_alpha != 0))
    return tkv_status(st);
  *scratch_bytes = plan.bytes;
  return TKV_OK;
}

tkv_status tkv_quantized_attention(int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t dtype,
                                   const void* q, const int8_t* pool, const float* scales, int64_t pool_pages,
                                   const int32_t* page_table, const uint32_t* slot_mask, const int32_t* page_counts,
                                   int32_t max_pages, void* out, float* alpha_sum, void* scratch, size_t scratch_bytes,
                                   tkv_stream stream) {
  AttendParams p{};
  Plan plan;
  if (int st = plan_attend(&p, &plan, batch, n_q_heads, n_kv_heads, head_dim, dtype, page_counts, max_pages, alpha_sum != nullptr))
    return tkv_status(st);
  if (int st = check_pool(&p.p, pool, scales, pool_pages, n_kv_heads, head_dim, page_table, max_pages, slot_mask)) return tkv_status(st);
  if (!q || !out || !slot_mask) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  if (misaligned(q, 16) || misaligned(out, 16) || misaligned(alpha_sum, 16))
    return tkv_status(report(TKV_ERR_INVALID_ARG, "q, out and alpha_sum must be 16-byte aligned"));
  if (plan.bytes) {
    if (!scratch) return tkv_status(report(TKV_ERR_INVALID_ARG, "null scratch: need %zu bytes", plan.bytes));
    if (scratch_bytes < plan.bytes) return tkv_status(report(TKV_ERR_CAPACITY, "scratch too small: need %zu bytes", plan.bytes));
    if (misaligned(scratch, 256)) return tkv_status(report(TKV_ERR_INVALID_ARG, "scratch not 256-byte aligned"));
  }
  char* at = static_cast<char*>(scratch);
  p.q = q; p.out = out; p.alpha = alpha_sum;
  p.part_o = plan.merge ? reinterpret_cast<float*>(at) : nullptr;
  p.part_m = plan.merge || alpha_sum ? reinterpret_cast<float4*>(at + plan.o_m) : nullptr;
  p.spill = alpha_sum ? reinterpret_cast<float*>(at + plan.o_spill) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == TKV_DTYPE_BF16) e = head_dim == 64 ? launch_attend<__nv_bfloat16, 64>(p, plan, s) : launch_attend<__nv_bfloat16, 128>(p, plan, s);
  else e = head_dim == 64 ? launch_attend<float, 64>(p, plan, s) : launch_attend<float, 128>(p, plan, s);
  return tkv_status(launched("quantised attention", e));
}

}  // extern "C"
