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
// weight is 2^((l - m) + (k + 13 - r)) f with V's scale f 2^k, m the running
// maximum of the logits and r one of (l - m) + k, so that pages whose scales are
// far apart neither overflow fp16 nor crowd at its lower end: a row's weights, V's
// scale among them, count down to 2^-38 of its largest (fp32: 2^-49, in two parts), with
// all their bits from 2^-27 on, and are 0 below in every element. Z
// sums 2^(l - m) as always. r is relative to m: a reference of l + k itself would lose k
// to rounding from |l| = 2^24 on, and the output its scale. Both references rise only when
// a logit passes them by more than 1 (a vote per page), so the shuffles and the
// rescaling are rare.
//
// 4 x 131072 tokens of 8 KV heads at d 128 (1.07 GB) take 166 us, 6.5 TB/s (a copy: 6.8);
// the tensor pipe is 17 % busy and the issue slots 61 %. The benchmark's batch (152 MB, 32
// sequences) takes 35 us without alpha and 42 with it, of which 5 are the start, when every CTA's
// table, page and scale reads queue up, 2 the uneven end and 3 the joining launch. In fp32: 165, 42
// and 48. Two column tiles (9 to 16 heads per KV head, fp32 5 to 8) at d 128 fill their 168
// registers and spill 8 bytes (fp32 40) outside the loop over pages: 222 us (fp32 198) for 1.07 GB.
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "quantized.h"
#include "tile_attention.h"  // SharedMemoryOptIn

namespace tkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kWindow = 384;        // pages that shared memory describes at a time
constexpr int kSegmentCost = 8;     // pages' time of a piece's start and end
constexpr int kLeastPages = 16;     // pages of a CTA's stretch, at least
constexpr int kMaxCluster = 8;      // CTAs of a cluster
constexpr int kClusterPages = 8;    // pages of each, at least
constexpr int kJoinPages = 24;      // pages' time of the launch that joins partials: 3 us
constexpr int kWholePages = 40;     // pages of segments that are not cut however many there are
constexpr int kAlphaPages = 64;     // line: pages of a segment up to which its one CTA forms alpha itself
constexpr int kMergeWarps = 4;
constexpr int kMergeThreads = kMergeWarps * 32;
constexpr int kAlphaSlots = 512;    // slots of an alpha CTA at a time
constexpr int kMaxColumns = 72;     // 64 heads per KV head in groups of 8 or 16, and what a load of 8 reads past them
constexpr int kSms = 152;
constexpr int kAlphaWave = kSms * 6;  // alpha CTAs that run at once
constexpr int kMaxShared = 232448;    // bytes of a CTA, and of an SM (of which each CTA takes 1 KB more)
constexpr int kSmShared = 233472;
constexpr float kNegInf = -INFINITY;
constexpr float kWeightBits = 13.f; // weights are at most 2^15: reference lag and f below 2 each

template <typename T> struct Columns;  // heads of an 8-column tile, and columns of a head
template <> struct Columns<__nv_bfloat16> { static constexpr int heads = 8, parts = 1; };
template <> struct Columns<float> { static constexpr int heads = 4, parts = 2; };

// How a call is cut. A SEGMENT is the pages of a sequence for one KV head and one
// group of its query heads.
//   Clusters: each segment is a cluster of 1 to 8 CTAs, whose results meet in shared
//   memory: one launch and no partials, for segments short enough for it.
//   The line: the segments lie one behind the other, each with kSegmentCost pages' room
//   ahead of its pages for its start and end, and CTA k takes the stretch
//   [k, k + 1) * share: all CTAs run at once and read the same number of pages. (Units of
//   72 pages in several waves took 191 us where this takes 168, 4 x 131072 tokens of 8
//   heads: every start waits out the queue that the running CTAs fill.)
// A PIECE is what a CTA has of a segment. On the line a piece that is not all of it
// leaves a partial, of which a CTA has two at most: one that goes on from the CTA before
// (2 k), and one that starts here (2 k + 1); a second launch joins them.
struct AttendParams {
  PoolRef p;
  const void* q;
  void* out;
  float* alpha;             // [B][Hkv][max_pages * 16], or null
  float* part_o;            // [2 * CTAs][heads of a unit][D]
  float4* part_m;           // [2 * CTAs][heads of a unit]: maximum, V's reference above it, sum
  float2* stats;            // [B][Hq] maximum and sum of rows written whole, for alpha
  float* spill;             // [page of the call][Hkv][16][columns], logits in base 2; null: in shared memory
  int32_t keep;             // logits are kept, for alpha
  int32_t columns;          // query heads of a KV head, filled up to 4 (several groups: to whole ones)
  int32_t B, Hq, G, groups; // groups: head groups of a KV head
  int32_t max_pages;
  int32_t ctas, cluster;    // cluster: CTAs of a segment, 0: stretches of the line
  int32_t share, total;
  float qscale;             // log2(e) / sqrt(D)
  int32_t count[kMaxBatch];     // pages
  int32_t order[kMaxBatch];     // clusters: sequences, longest first
  int32_t base[kMaxBatch + 1];  // where the segments of a sequence start on the line
  int32_t page0[kMaxBatch + 1]; // prefix sums of the pages
  int32_t alpha_slots;            // slots of an alpha CTA
  int32_t alpha0[kMaxBatch + 1];  // prefix sums of the alpha CTAs of a KV head
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// v 2^x, in two halves where 2^x alone would leave fp32's normal range
__device__ __forceinline__ float times_ex2(float v, float x) {
  if (fabsf(x) <= 120.f) return v * exp2f(x);
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
// a += b, rounded to nearest. The tensor core cuts what it adds to an accumulator: over
// 862 pages of constant V sums came out 2e-5 low, over 6896 1.6e-4.
__device__ __forceinline__ void add4(float (&a)[4], const float (&b)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    unsigned long long x, y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a[i]), "f"(a[i + 1]));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b[i]), "f"(b[i + 1]));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(y));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a[i]), "=f"(a[i + 1]) : "l"(x));
  }
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

__device__ __forceinline__ void copy16(uint32_t to, const void* from, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "l"(policy) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;"); }
template <int N> __device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A slot's weights, summed over the heads, from their logits and each head's (maximum,
// 1 / sum), which are (0, 0) for columns without a head and for rows without a weight.
struct AlphaSum {
  float value = 0.f;
  bool any = false;  // a valid slot
  __device__ __forceinline__ void add(const float4& l, const float2* head) {
    const float x[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float w = ex2(x[i] - head[i].x) * head[i].y;
      const bool valid = x[i] != kNegInf;
      value += valid ? w : 0.f;  // a NaN of the row stays out of its empty slots
      any |= valid;
    }
  }
};
// The joint maximum of n statistics (maximum, V's reference above it, sum), and V's reference above that.
struct Peak {
  float top, ref;
};
template <int n, typename Stat>
__device__ __forceinline__ Peak peak_of(Stat stat) {
  Peak p = {kNegInf, kNegInf};
#pragma unroll
  for (int i = 0; i < n; ++i) p.top = fmaxf(p.top, stat(i).x);
#pragma unroll
  for (int i = 0; i < n; ++i) p.ref = fmaxf(p.ref, (stat(i).x - p.top) + stat(i).y);  // -inf or NaN of one without a maximum
  return p;
}
__device__ __forceinline__ float2 alpha_head(float top, float sum) { return sum == 0.f ? make_float2(0.f, 0.f) : make_float2(top, 1.f / sum); }

// Four elements of a row's output from its sum of weighted V, in the units of its reference.
template <typename T>
__device__ __forceinline__ void put_row(T* at, const float4& x, float ref, float sum) {
  const float by = sum == 0.f ? 0.f : 1.f / sum, e = sum == 0.f ? 0.f : ref - kWeightBits;
  put4(at, make_float4(times_ex2(x.x * by, e), times_ex2(x.y * by, e), times_ex2(x.z * by, e), times_ex2(x.w * by, e)));
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// 16 bytes of another CTA's shared memory, at this CTA's address of them
__device__ __forceinline__ float4 load_cluster(uint32_t at, int cta) {
  uint32_t there;
  float4 x;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(cta));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(there) : "memory");
  return x;
}

// What a unit keeps of a page: id (-1: none of its slots counts), valid slots and
// the power k of V's scale, K's scale, and V's scale as f in f 2^k
// (1 <= |f| < 2, of the scale's sign).
__device__ __forceinline__ int4 page_info(const AttendParams& p, int32_t id, int h) {
  if (id < 0 || id >= p.p.pages) return make_int4(-1, 0, 0, 0);
  const uint32_t live = p.p.mask[id] & kFullMask;
  if (!live) return make_int4(-1, 0, 0, 0);
  const float2 s = *reinterpret_cast<const float2*>(p.p.scales + (static_cast<int64_t>(id) * p.p.hkv + h) * 2);
  float f = finite_or_nan(s.y);
  int k = -126;                                  // of 0 and NaN: no reference rises for them
  if (fabsf(f) > 0.f) {
    const bool small = fabsf(f) < 0x1p-100f;
    const uint32_t bits = __float_as_uint(small ? f * 0x1p40f : f);
    k = static_cast<int>(bits >> 23 & 0xffu) - 127 - (small ? 40 : 0);
    f = __uint_as_float((bits & 0x807fffffu) | 0x3f800000u);
  }
  return make_int4(id, static_cast<int>(live | static_cast<uint32_t>(k + 256) << 16), __float_as_int(finite_or_nan(s.x)),
                   __float_as_int(f));
}

template <int D>
struct Ring {
  static constexpr int page_bytes = 2 * kPage * D;                    // a head's K and V codes
  // 8 KB per warp. More in flight only lengthens the queues, and with them each
  // start and the spread of the ends: with 12 KB the same call took 179 us, not 168.
  static constexpr int stages = D == 128 ? 2 : 4;
  static constexpr int bytes = kWarps * stages * page_bytes;
};

template <typename T, int D, int NT>
struct Smem {
  static constexpr int heads = Columns<T>::heads * NT;
  static constexpr int out_row = D + 4;                               // floats; rows start in different banks
  static constexpr int merge_bytes = kWarps * heads * out_row * 4;
  static constexpr int o_info = Ring<D>::bytes > merge_bytes ? Ring<D>::bytes : merge_bytes;
  static constexpr int o_stat = o_info + kWindow * 16;
  static constexpr int o_head = o_stat + kWarps * heads * 16;
  static constexpr int o_piece = o_head + heads * 8;
  static constexpr int bytes = o_piece + heads * 16;
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
__device__ __forceinline__ void copy_page(uint32_t to, const int8_t* block, int lane, uint64_t policy) {
  constexpr int kRowChunks = D / 16;
#pragma unroll
  for (int i = 0; i < 2 * kPage * D / 512; ++i) {
    const int at = i * 32 + lane;
    copy16(to + chunk_at<D>(at / kRowChunks, at % kRowChunks), block + at * 16, policy);
  }
}

// Page j of a piece goes to warp j % 4, which keeps one (D 64: 3) on its way
// besides the one it reads; no warp waits for another before the end of a piece.
// The first copies need the page ids only, so they leave before the masks, scales
// and queries are here.
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
  float2* s_head = reinterpret_cast<float2*>(smem + S::o_head);
  float4* s_piece = reinterpret_cast<float4*>(smem + S::o_piece);
  float* s_spill = reinterpret_cast<float*>(smem + S::bytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  cudaGridDependencySynchronize();
  const int segments = p.p.hkv * p.groups;         // of a sequence
  int b = 0, pos = 0, end = 1;                     // the CTA's stretch
  const int rank = p.cluster ? blockIdx.x % p.cluster : 0;
  if (p.cluster) {
    b = p.order[blockIdx.x / p.cluster / segments];
  } else {
    pos = blockIdx.x * p.share;
    end = min(pos + p.share, p.total);
    int hi = p.B - 1;
    while (b < hi) {
      const int mid = (b + hi + 1) >> 1;
      if (p.base[mid] <= pos) b = mid; else hi = mid - 1;
    }
  }
  // codes are read once: their lines leave the L2 before the logits and partials (41 us for the
  // benchmark's batch with alpha, 45 without this)
  uint64_t policy;
  if (p.groups == 1) asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  else asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));  // the other groups read them too
  bool later = false;                              // not the first window: shared memory may be in use
  while (pos < end) {
    int segment, lo = 0, hi = p.count[b], stop = end;  // pages lo .. hi - 1 of it
    const int n = hi;
    bool last = false;                             // the stretch goes on with the next sequence
    if (p.cluster) {
      segment = blockIdx.x / p.cluster % segments;
      lo = n * rank / p.cluster;
      hi = n * (rank + 1) / p.cluster;
    } else {
      const int span = n + kSegmentCost;
      segment = (pos - p.base[b]) / span;
      const int from = p.base[b] + segment * span;
      stop = min(end, from + span);
      last = stop == p.base[b + 1];
      lo = max(pos - from - kSegmentCost, 0);
      hi = max(stop - from - kSegmentCost, 0);
      if (hi <= lo && !(n == 0 && pos == from)) {  // room ahead of the pages only
        pos = stop;
        b += last;
        continue;
      }
    }
    const int h = segment / p.groups, group = segment % p.groups;
    const int head0 = h * p.G + group * S::heads;  // first head of the group
    const int nheads = min(S::heads, p.G - group * S::heads);
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * R::stages * R::page_bytes;
    const int32_t* row = p.p.table + b * p.p.table_stride;

    uint32_t qf[NT][kChunks * 4][2];
    float qpow[NT][kOwn];
    float o[NT][kTiles][4];
    float m[NT][kOwn], r[NT][kOwn], z[NT][kOwn];
    for (int w0 = lo;; w0 += kWindow) {
      const int count = min(kWindow, hi - w0), mine = count > warp ? (count - warp + kWarps - 1) / kWarps : 0;
      auto copy = [&](int i, int id) {
        if (id >= 0 && id < p.p.pages)
          copy_page<D>(ring + (i % R::stages) * R::page_bytes, p.p.codes + (static_cast<int64_t>(id) * p.p.hkv + h) * R::page_bytes, lane, policy);
        commit();
      };
      auto start = [&](int i) { copy(i, i < mine ? s_info[warp + i * kWarps].x : -1); };
      int32_t first[R::stages - 1], ids[kWindow / kThreads];
#pragma unroll
      for (int i = 0; i < R::stages - 1; ++i) first[i] = i < mine ? row[w0 + warp + i * kWarps] : -1;
#pragma unroll
      for (int i = 0; i < kWindow / kThreads; ++i) ids[i] = tid + i * kThreads < count ? row[w0 + tid + i * kThreads] : -1;
      if (later) __syncthreads();                  // what the last window or piece left is read
      later = true;
#pragma unroll
      for (int i = 0; i < R::stages - 1; ++i) copy(i, first[i]);
#pragma unroll
      for (int i = 0; i < kWindow / kThreads; ++i)
        if (tid + i * kThreads < count) s_info[tid + i * kThreads] = page_info(p, ids[i], h);
      if (w0 == lo) {
        // queries: fragments of Q^T, and the power of two taken out of each head
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
              if (kParts == 2 && part == 1) {
                const float rest = y[j] - __half2float(__float2half_rn(y[j]));
                y[j] = rest == rest ? rest * 2048.f : 0.f;  // of an infinity or NaN the first part says it all
              }
            }
            qf[nt][i >> 2][(i >> 1) & 1] = half2_bits(y[0], y[1]);
          }
#pragma unroll
          for (int i = 0; i < kOwn; ++i) {
            const int of = __shfl_sync(0xffffffffu, e, (2 * t + i) * 4);
            qpow[nt][i] = __uint_as_float(static_cast<uint32_t>(of + 127) << 23) * p.qscale;  // infinity for a row that holds one
            m[nt][i] = kNegInf;
            r[nt][i] = z[nt][i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < kTiles; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
        }
      }
      __syncthreads();
      float* spill = p.spill ? p.spill + (static_cast<int64_t>(p.page0[b] + w0) * p.p.hkv + h) * kPage * p.columns + group * S::heads
                             : s_spill + (w0 - lo) * kPage * p.columns;
      const int64_t spill_page = static_cast<int64_t>(p.spill ? p.p.hkv : 1) * kPage * p.columns;
      const int own = min(S::heads, p.columns - group * S::heads);  // columns of the group
      for (int i = 0; i < mine; ++i) {
        wait_copies<R::stages - 2>();
        __syncwarp();                                  // page i is here for all lanes, and page i - 1 is read
        start(i + R::stages - 1);
        const int page = warp + i * kWarps;
        const int4 info = s_info[page];
        const uint32_t live = info.y & kFullMask;
        if (info.x < 0) {                              // an empty page: nothing was copied
          if (p.keep) {
            float* at = spill + page * spill_page;
            for (int w = lane; w < kPage * S::heads; w += 32)
              if (w % S::heads < own) at[(w / S::heads) * p.columns + w % S::heads] = kNegInf;
          }
          continue;
        }
        const char* slot = smem + (warp * R::stages + i % R::stages) * R::page_bytes;
        // S^T = K Q^T, as two sums: shorter chains, and half as many cut additions in each
        float s[NT][4] = {}, s1[NT][4] = {};
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
            for (int nt = 0; nt < NT; ++nt) mma(w & 1 ? s1[nt] : s[nt], a0, a1, a2, a3, qf[nt][c * 4 + w][0], qf[nt][c * 4 + w][1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) add4(s[nt], s1[nt]);
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
            // the factor below 1 first: no product leaves fp32's range but where the logit does, or is off by 2^-22
            const bool up = qpow[nt][j] > 1.f;
            const float first = up ? sk : qpow[nt][j], second = up ? qpow[nt][j] : sk;
            l[nt][j][0] = live0 ? s[nt][j] * first * second : kNegInf;
            l[nt][j][1] = live1 ? s[nt][2 + j] * first * second : kNegInf;
            const float over = fmaxf(l[nt][j][0], l[nt][j][1]) - m[nt][j];
            rise |= over > 1.f || over + k > r[nt][j] + 1.f;
          }
          if (p.keep && nt * kHeads + t * kOwn < own) {
            float* at = spill + page * spill_page + g * p.columns + nt * kHeads + t * kOwn;
            if (kOwn == 2) {
              *reinterpret_cast<float2*>(at) = make_float2(l[nt][0][0], l[nt][kOwn - 1][0]);
              *reinterpret_cast<float2*>(at + 8 * p.columns) = make_float2(l[nt][0][1], l[nt][kOwn - 1][1]);
            } else {
              at[0] = l[nt][0][0];
              at[8 * p.columns] = l[nt][0][1];
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
              const float m1 = fmaxf(m[nt][j], top);
              keep[j] = 1.f;
              if (m1 != kNegInf) {
                const float fall = m[nt][j] - m1, r1 = fmaxf(r[nt][j] + fall, (top - m1) + k);
                z[nt][j] *= ex2(fall);
                keep[j] = ex2(fall + (r[nt][j] - r1));
                m[nt][j] = m1;
                r[nt][j] = r1;
              }
              if (kOwn == 1) keep[1] = keep[0];
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
            const float mz = m[nt][j] == kNegInf ? 0.f : m[nt][j], ro = k + kWeightBits - r[nt][j];
            const float x0 = l[nt][j][0] - mz, x1 = l[nt][j][1] - mz;
            z[nt][j] += ex2(x0) + ex2(x1);
            w[0][j] = live0 ? ex2(x0 + ro) * f : 0.f;
            w[1][j] = live1 ? ex2(x1 + ro) * f : 0.f;
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
            for (int nt = 0; nt < NT; ++nt) {
              float c[4] = {};
              mma(c, a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
              add4(o[nt][w * 2 + half], c);
            }
          }
        }
      }
      if (w0 + kWindow >= hi) break;
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
        const Peak at = peak_of<kWarps>([&](int w) { return s_stat[w * S::heads + head]; });
        const float keep = m[nt][j] == kNegInf ? (z[nt][j] == z[nt][j] ? 0.f : NAN) : ex2((m[nt][j] - at.top) + (r[nt][j] - at.ref));
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
    const bool all = p.cluster || (lo == 0 && hi == n), alone = p.cluster <= 1;
    const int64_t part = (2 * static_cast<int64_t>(blockIdx.x) + (lo == 0)) * S::heads;
    const int64_t row0 = static_cast<int64_t>(b) * p.Hq + head0;
    for (int i = tid; i < nheads * (D / 4); i += kThreads) {
      const int head = i / (D / 4), d = i % (D / 4) * 4;
      const Peak of = peak_of<kWarps>([&](int w) { return s_stat[w * S::heads + head]; });
      float sum = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 st = s_stat[w * S::heads + head];
        sum += st.x == kNegInf ? st.z : st.z * ex2(st.x - of.top);
        const float4 y = *reinterpret_cast<const float4*>(s_out + (w * S::heads + head) * S::out_row + d);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      if (!alone) {                                // for the cluster, in the first warp's place
        *reinterpret_cast<float4*>(s_out + head * S::out_row + d) = x;
        if (d == 0) s_piece[head] = make_float4(of.top, of.ref, sum, 0.f);
      } else if (all) {
        put_row(static_cast<T*>(p.out) + (row0 + head) * D + d, x, of.ref, sum);
        if (p.keep && d == 0) {
          if (p.stats) p.stats[row0 + head] = make_float2(of.top, sum);
          s_head[head] = alpha_head(of.top, sum);
        }
      } else {
        if (d == 0) p.part_m[part + head] = make_float4(of.top, of.ref, sum, 0.f);
        *reinterpret_cast<float4*>(p.part_o + (part + head) * D + d) = x;
      }
    }
    if (p.keep && tid >= nheads && tid < S::heads) s_head[tid] = make_float2(0.f, 0.f);
    if (!alone) {
      // each CTA joins its share of the rows, and for alpha the sums of all heads
      cluster_arrive();
      cluster_wait();
      const uint32_t pieces = static_cast<uint32_t>(__cvta_generic_to_shared(s_piece)), outs = static_cast<uint32_t>(__cvta_generic_to_shared(s_out));
      float4 st[kMaxCluster];
      float take[kMaxCluster];
      Peak of;
      float sum;
      auto join_head = [&](int head) {
        sum = 0.f;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) st[c] = c < p.cluster ? load_cluster(pieces + head * 16, c) : make_float4(kNegInf, 0.f, 0.f, 0.f);
        of = peak_of<kMaxCluster>([&](int c) { return st[c]; });
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          sum += st[c].x == kNegInf ? st[c].z : st[c].z * ex2(st[c].x - of.top);
          take[c] = st[c].x == kNegInf ? 1.f : ex2((st[c].x - of.top) + (st[c].y - of.ref));
        }
      };
      for (int i = rank * kThreads + tid; i < nheads * (D / 4); i += p.cluster * kThreads) {
        const int head = i / (D / 4), d = i % (D / 4) * 4;
        join_head(head);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          if (c >= p.cluster) break;
          const float4 y = load_cluster(outs + (head * S::out_row + d) * 4, c);
          x.x += y.x * take[c], x.y += y.y * take[c], x.z += y.z * take[c], x.w += y.w * take[c];
        }
        put_row(static_cast<T*>(p.out) + (row0 + head) * D + d, x, of.ref, sum);
      }
      if (p.alpha && tid < nheads) {
        join_head(tid);
        s_head[tid] = alpha_head(of.top, sum);
      }
      cluster_arrive();                            // the others' shared memory is read
    }
    if (p.alpha && all && p.groups == 1 && (p.cluster || n <= kAlphaPages)) {
      __syncthreads();
      const float* l = p.spill ? p.spill + (static_cast<int64_t>(p.page0[b]) * p.p.hkv + h) * kPage * p.columns : s_spill - lo * kPage * p.columns;
      const int64_t page = static_cast<int64_t>(p.spill ? p.p.hkv : 1) * kPage;
      float* alpha = p.alpha + (static_cast<int64_t>(b) * p.p.hkv + h) * p.max_pages * kPage;
#pragma unroll 4
      for (int i = lo * kPage + tid; i < hi * kPage; i += kThreads) {
        const float* at = l + ((i / kPage) * page + i % kPage) * p.columns;
        AlphaSum sum;
#pragma unroll
        for (int j = 0; j < S::heads; j += 4)
          if (j < p.columns) sum.add(*reinterpret_cast<const float4*>(at + j), s_head + j);
        if (sum.any) alpha[i] += sum.value;
      }
    }
    if (!alone) cluster_wait();
    pos = stop;
    b += last;
  }
}

// The partials of a segment: CTAs first .. last have a piece of it, and all of it
// if they are the same.
struct Pieces {
  int first, last;
  __device__ int64_t row(int cta, int heads) const { return (2 * static_cast<int64_t>(cta) + (cta == first)) * heads; }
};
__device__ __forceinline__ Pieces pieces_of(const AttendParams& p, int b, int segment) {
  if (p.count[b] == 0) return {0, 0};
  const int from = p.base[b] + segment * (p.count[b] + kSegmentCost) + kSegmentCost;
  return {from / p.share, (from + p.count[b] - 1) / p.share};
}

// (m, z) and (m1, z1) joined
__device__ __forceinline__ void join(float& m, float& z, float m1, float z1) {
  const float top = fmaxf(m, m1);
  z = (m == kNegInf ? z : z * ex2(m - top)) + (m1 == kNegInf ? z1 : z1 * ex2(m1 - top));
  m = top;
}

// The last B * Hq CTAs join the pieces of a query head each, a warp every fourth
// piece. The others (alpha) take alpha_slots slots of a sequence and KV head: the
// maximum and sum of each query head, then the slots' weights from their logits,
// which are on their way meanwhile.
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) merge_quantized_kernel(const __grid_constant__ AttendParams p, int heads) {
  constexpr int E = D / 32;
  __shared__ float s_x[kMergeWarps][D];
  __shared__ float4 s_st[kMergeWarps];
  __shared__ float2 s_head[kMaxColumns];
  cudaGridDependencySynchronize();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int parts = p.alpha ? p.alpha0[p.B] * p.p.hkv : 0;
  if (static_cast<int>(blockIdx.x) >= parts) {
    const int row_out = blockIdx.x - parts, b = row_out / p.Hq, hq = row_out % p.Hq, h = hq / p.G, head = hq % p.G;
    const Pieces pc = pieces_of(p, b, h * p.groups + head / heads);
    if (pc.first == pc.last) return;               // written by its CTA
    float m = kNegInf, r = 0.f, z = 0.f, x[E] = {};
#pragma unroll 4
    for (int c = pc.first + warp; c <= pc.last; c += kMergeWarps) {
      const int64_t row = pc.row(c, heads) + head % heads;
      const float4 st = p.part_m[row];
      float y[E];
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = p.part_o[row * D + lane * E + i];
      const float m0 = m;
      join(m, z, st.x, st.z);
      const float ref = fmaxf((m0 - m) + r, (st.x - m) + st.y);
      const float keep = m0 == kNegInf ? 1.f : ex2((m0 - m) + (r - ref)), take = st.x == kNegInf ? 1.f : ex2((st.x - m) + (st.y - ref));
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = x[i] * keep + y[i] * take;
      r = m == kNegInf ? 0.f : ref;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) s_x[warp][lane * E + i] = x[i];
    if (lane == 0) s_st[warp] = make_float4(m, r, z, 0.f);
    __syncthreads();
    if (tid < D / 4) {
      m = kNegInf;
      z = 0.f;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) join(m, z, s_st[w].x, s_st[w].z);
      const Peak of = peak_of<kMergeWarps>([&](int w) { return s_st[w]; });
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        const float4 a = *reinterpret_cast<const float4*>(&s_x[w][tid * 4]);
        const float take = s_st[w].x == kNegInf ? 1.f : ex2((s_st[w].x - of.top) + (s_st[w].y - of.ref));
        y.x += a.x * take, y.y += a.y * take, y.z += a.z * take, y.w += a.w * take;
      }
      put_row(static_cast<T*>(p.out) + static_cast<int64_t>(row_out) * D + tid * 4, y, of.ref, z);
    }
    return;
  }
  // alpha
  constexpr int kSlots = kAlphaSlots / kMergeThreads;  // of a thread
  const int h = blockIdx.x % p.p.hkv, at = blockIdx.x / p.p.hkv;
  int b = 0, last = p.B - 1;
  while (b < last) {
    const int mid = (b + last + 1) >> 1;
    if (p.alpha0[mid] <= at) b = mid; else last = mid - 1;
  }
  int first = (at - p.alpha0[b]) * p.alpha_slots + tid;
  const int slots = min(p.count[b] * kPage, first - tid + p.alpha_slots);
  if (p.groups == 1 && p.count[b] <= kAlphaPages) {
    const Pieces pc = pieces_of(p, b, h);
    if (pc.first == pc.last) return;               // formed by its CTA
  }
  const int columns = p.columns;
  float4 l[kSlots][2];
  float* alpha = p.alpha + (static_cast<int64_t>(b) * p.p.hkv + h) * p.max_pages * kPage;
  float before[kSlots];
  auto load = [&](int j) {                         // logits of heads j .. j + 7
#pragma unroll
    for (int k = 0; k < kSlots; ++k)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        l[k][v] = make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
        const int i = first + k * kMergeThreads;
        if (i < slots && j + 4 * v < columns)
          l[k][v] = *reinterpret_cast<const float4*>(
              p.spill + ((static_cast<int64_t>(p.page0[b] + i / kPage) * p.p.hkv + h) * kPage + i % kPage) * columns + j + 4 * v);
      }
  };
  auto load_first = [&] {
#pragma unroll
    for (int k = 0; k < kSlots; ++k) before[k] = first + k * kMergeThreads < slots ? alpha[first + k * kMergeThreads] : 0.f;
    load(0);
  };
  load_first();
  if (tid >= p.G && tid < kMaxColumns) s_head[tid] = make_float2(0.f, 0.f);
  for (int i = tid / 8; i < p.G; i += kMergeThreads / 8) {  // eight lanes per head
    const uint32_t lanes = 0xffu << (lane & 24);
    const Pieces pc = pieces_of(p, b, h * p.groups + i / heads);
    float m = kNegInf, z = 0.f;
    if (pc.first == pc.last) {
      const float2 st = p.stats[static_cast<int64_t>(b) * p.Hq + h * p.G + i];
      m = st.x, z = st.y;
    } else {
#pragma unroll 4
      for (int c = pc.first + lane % 8; c <= pc.last; c += 8) {
        const float4 st = p.part_m[pc.row(c, heads) + i % heads];
        join(m, z, st.x, st.z);
      }
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) join(m, z, __shfl_xor_sync(lanes, m, d), __shfl_xor_sync(lanes, z, d));
    }
    if (lane % 8 == 0) s_head[i] = alpha_head(m, z);
  }
  __syncthreads();
  while (first < slots) {
    AlphaSum sum[kSlots];
    for (int j = 0; j < p.G; j += 8) {
      if (j) load(j);
#pragma unroll
      for (int k = 0; k < kSlots; ++k)
#pragma unroll
        for (int v = 0; v < 2; ++v) sum[k].add(l[k][v], s_head + j + 4 * v);
    }
#pragma unroll
    for (int k = 0; k < kSlots; ++k)
      if (sum[k].any) alpha[first + k * kMergeThreads] = before[k] + sum[k].value;
    first += kAlphaSlots;
    load_first();
  }
}

// ---- host side

struct Plan {
  int nt;      // column tiles of a unit
  int heads;   // of a unit
  int shared;  // bytes of shared memory for logits
  size_t o_m, o_stats, o_spill, bytes;  // scratch
};

template <int D>
int smem_bytes(int dtype, int nt) {
  if (dtype == TKV_DTYPE_BF16) return nt == 1 ? Smem<__nv_bfloat16, D, 1>::bytes : Smem<__nv_bfloat16, D, 2>::bytes;
  return nt == 1 ? Smem<float, D, 1>::bytes : Smem<float, D, 2>::bytes;
}

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
  p->columns = p->groups == 1 ? (p->G + 3) / 4 * 4 : p->groups * plan->heads;
  int most = 0;
  p->page0[0] = 0;
  for (int b = 0; b < batch; ++b) {
    const int n = page_counts[b];
    if (n < 0 || n > max_pages) return report(TKV_ERR_INVALID_ARG, "page_counts[%d] out of 0..max_pages", b);
    p->count[b] = n;
    p->page0[b + 1] = p->page0[b] + n;
    most = std::max(most, n);
  }
  const int64_t segments = static_cast<int64_t>(Hkv) * p->groups, slots = kSms * (plan->nt == 1 ? 4 : 3);
  const int64_t total = segments * (p->page0[batch] + static_cast<int64_t>(batch) * kSegmentCost);
  if (total > (int64_t(1) << 30)) return report(TKV_ERR_INVALID_ARG, "more than 2^30 pages and heads in one call");
  p->total = static_cast<int32_t>(total);
  p->share = static_cast<int32_t>(std::max<int64_t>((total + slots - 1) / slots, kSegmentCost + kLeastPages));
  // Clusters save the partials and the launch that joins them, worth kJoinPages pages of a
  // CTA's time, and lose where their CTAs get more pages than the line's (us with alpha, line
  // and clusters): 8 rows of 2000 tokens, 4 KV heads, 16.4 and 14.4; 64 of 1000, 8, 37 and 31; one of 8192,
  // 8, 15 and 24; the benchmark's batch 43 and 46. More segments than CTAs run at once would leave the last
  // wave short: then only if they are short too.
  int c = 1;
  while (c < kMaxCluster && segments * batch * c * 2 <= slots && most >= 2 * c * kClusterPages) c *= 2;
  const bool clusters = segments * batch <= slots ? (most + c - 1) / c <= p->share + kJoinPages : most <= kWholePages;
  p->cluster = p->groups == 1 && clusters ? c : 0;  // alpha takes the sums of all heads: one group
  // alpha CTAs of one wave, so that the heads' pieces are joined by few of them (64 rows of 4000 tokens,
  // 8 KV heads: 107 us, 110 with 512 slots each)
  const int64_t all_slots = static_cast<int64_t>(p->page0[batch]) * kPage * Hkv;
  p->alpha_slots = static_cast<int32_t>(std::min<int64_t>((all_slots / kAlphaWave + kAlphaSlots - 1) / kAlphaSlots, 64)) * kAlphaSlots;
  p->alpha_slots = std::max(p->alpha_slots, kAlphaSlots);
  p->alpha0[0] = 0;
  for (int b = 0; b < batch; ++b)
    p->alpha0[b + 1] = p->alpha0[b] + (p->cluster ? 0 : (p->count[b] * kPage + p->alpha_slots - 1) / p->alpha_slots);
  if (p->cluster) {
    p->ctas = static_cast<int32_t>(segments * batch * p->cluster);
    for (int b = 0; b < batch; ++b) p->order[b] = b;
    std::sort(p->order, p->order + batch, [&](int a, int b) { return p->count[a] != p->count[b] ? p->count[a] > p->count[b] : a < b; });
  } else {
    p->ctas = static_cast<int32_t>((total + p->share - 1) / p->share);
    p->base[0] = 0;
    for (int b = 0; b < batch; ++b) p->base[b + 1] = p->base[b] + static_cast<int32_t>(segments) * (p->count[b] + kSegmentCost);
  }
  auto align = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = p->cluster ? 0 : 2 * static_cast<size_t>(p->ctas) * plan->heads;
  plan->o_m = align(rows * D * 4);
  plan->o_stats = plan->o_m + align(rows * 16);
  plan->o_spill = plan->o_stats + (want_alpha && !p->cluster ? align(static_cast<size_t>(batch) * Hq * 8) : 0);
  plan->bytes = plan->o_spill;
  plan->shared = 0;
  if (want_alpha) {
    // logits stay in the clusters' shared memory where all CTAs still run at once with it
    const int64_t need = static_cast<int64_t>((most + c - 1) / c) * kPage * p->columns * 4;
    const int64_t cta = need + (D == 64 ? smem_bytes<64>(dtype, plan->nt) : smem_bytes<128>(dtype, plan->nt));
    if (p->cluster && cta <= kMaxShared && p->ctas <= kSms * (kSmShared / (cta + 1024))) plan->shared = static_cast<int>(need);
    else plan->bytes += align(static_cast<size_t>(p->page0[batch]) * Hkv * kPage * p->columns * 4);
  }
  return TKV_OK;
}

template <typename T, int D, int NT>
cudaError_t launch_units(const AttendParams& p, int shared, cudaStream_t s) {
  const int bytes = Smem<T, D, NT>::bytes + shared;
  static SharedMemoryOptIn opt_in;
  const cudaError_t e = opt_in.once(reinterpret_cast<const void*>(attend_quantized_kernel<T, D, NT>), kMaxShared);
  if (e != cudaSuccess) return e;
  return launch_early(attend_quantized_kernel<T, D, NT>, dim3(p.ctas), kThreads, bytes, s, std::max(p.cluster, 1), p);
}

template <typename T, int D>
cudaError_t launch_attend(const AttendParams& p, const Plan& plan, cudaStream_t s) {
  cudaError_t e = plan.nt == 1 ? launch_units<T, D, 1>(p, plan.shared, s) : launch_units<T, D, 2>(p, plan.shared, s);
  const int64_t rows = p.cluster ? 0 : static_cast<int64_t>(p.B) * p.Hq;
  const int64_t parts = p.alpha ? static_cast<int64_t>(p.alpha0[p.B]) * p.p.hkv : 0;
  if (e != cudaSuccess || rows + parts == 0) return e;
  return launch_early(merge_quantized_kernel<T, D>, dim3(static_cast<unsigned>(rows + parts)), kMergeThreads, 0, s, 1, p, plan.heads);
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
  p.part_o = reinterpret_cast<float*>(at);
  p.part_m = reinterpret_cast<float4*>(at + plan.o_m);
  p.keep = alpha_sum != nullptr;
  p.stats = alpha_sum && !p.cluster ? reinterpret_cast<float2*>(at + plan.o_stats) : nullptr;
  p.spill = alpha_sum && !plan.shared ? reinterpret_cast<float*>(at + plan.o_spill) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == TKV_DTYPE_BF16) e = head_dim == 64 ? launch_attend<__nv_bfloat16, 64>(p, plan, s) : launch_attend<__nv_bfloat16, 128>(p, plan, s);
  else e = head_dim == 64 ? launch_attend<float, 64>(p, plan, s) : launch_attend<float, 128>(p, plan, s);
  return tkv_status(launched("quantised attention", e));
}

}  // extern "C"
