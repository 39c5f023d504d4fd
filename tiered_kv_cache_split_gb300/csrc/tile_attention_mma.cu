// bf16 tiled attention on the 5th-generation tensor cores (terms and plan:
// tile_attention.h; the mathematics: tile_attention.cu).
//
// One CTA per SM runs unit after unit: up to 256 rows as two tiles of 128
// against a stream of 128-key blocks, each in two halves of 64. Twelve warps:
//   0-3, 4-7  softmax of tile 0 / 1: one thread per row (TMEM lane), so row
//             maxima and sums need no exchange between threads; they also load
//             the tile's Q and write its result
//   8         producer: takes units and publishes them to the other warps; TMA of
//             K and V blocks into a ring of shared-memory slots, running ahead
//             into the next unit
//   9, 10     issue tcgen05.mma for tile 0 / 1: S = Q K^T from shared memory,
//             O += P V with P read from TMEM. The tensor core takes few MMAs
//             ahead, so a lone issuer's waits would idle it: with two, one waits
//             while the other's MMAs run
//   11        helper: cleans V blocks (below)
// TMEM holds, per tile, S of two halves (2 x 64 fp32 columns) and O (D
// columns); P (bf16) overwrites the S it came from. S of the next half is
// computed while the softmax works on this one, so a softmax warp finds its
// next S ready; the next unit's first two are computed while the last O is
// written out. A segment of at most 128 rows that is split anyway (a decode
// step) runs as a PAIR: both tiles hold the same rows, tile t takes half t of
// every block, and each has a partial of its own (four chains of 8 tokens behind
// 8192: 18.8 us, against 20.6 with one tile idle; long splits, bound by HBM,
// take the same time either way).
//
// Measured (d 128; GB300, where a copy reaches 6.8 TB/s and a library product
// 1.89 PFLOP/s): a causal prompt of 8192 tokens with 32 / 8 heads 358 us, 1.54
// PFLOP/s, 81 % of that product's rate; the tensor pipe is busy in 66 % of an SM's
// active cycles (all of them would be 2.37 PFLOP/s at the 1.90 GHz it ran at) and
// waits for the softmax in the rest; 64 decode rows over a shared 131072-token prefix
// 119 us, 4.8 TB/s with the pipe busy in 54 %; 8 decode rows over 15360 tokens with
// 32 KV heads 60 us, 5.2 TB/s, bound by HBM and the last wave of units.
//
// The grid has a CTA per unit; a running CTA takes the units of CTAs that have
// not started (cluster launch control), so units are handed out in grid order,
// longest first, without a counter in memory, and a unit's start-up overlaps
// the end of the one before.
//
// Running maximum: O is rescaled only when a row's maximum has risen by more
// than kRise (base 2) over the one its weights refer to, or at the first key. A
// weight is 2^(l - reference - kRise): 2^-kRise for the reference itself and at
// most 1 for what may follow before a rescaling, so O stays below the sum of |V|
// whatever the size of V. O and Z always refer to the same maximum, and a
// weight's relative error does not depend on its size; those 2^-106 of the
// largest or smaller count as 0. With a rise of 8 one half in six was rescaled,
// at about 1500 cycles each (prompt of 8192, normal queries).
//
// The weights are rounded to bf16 (half a step 2^-8 each) because the MMA takes
// P and V in one type. Z sums the rounded weights, in fp32: where few keys carry
// a row, their errors then leave the quotient (0.0018 off the 64-bit result in
// the 2-norm, against 0.0023 with Z of the unrounded ones; output rounding alone
// is 0.0016), for 2 % of the time of a prompt of 8192 (351 us with the unrounded
// ones). alpha is made of unrounded weights: calls that ask for it keep their sum
// too.
//
// 0 * NaN must not reach O: the V rows of holes are zeroed in shared memory, and
// keys past a sequence's end or that only some rows see have their non-finite V
// values taken out there; those are added at the end to the rows that see them.
// The helper warp does this between a V block's arrival and its product, and
// passes on blocks that need nothing.
//
// Every wait is bounded: on running out it raises the CTA's abort flag and the
// caller's status word; each role then leaves its loop, the copies and MMAs in
// flight are awaited (bounded too) and TMEM is given back.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "tile_attention.h"

namespace tkv {
namespace {

constexpr int kRows = 128;
constexpr int kThreads = 384;
constexpr int kProducer = 8, kIssuer = 9, kHelper = 11;  // warps; one issuer per tile
constexpr int kHalf = 64;                  // keys of one S
constexpr int kBlockPages = kKeyBlock / kPage;
constexpr int kBox = 128 * 128;            // a box: 128 rows of 64 bf16 columns, 128-byte swizzled
constexpr float kRise = 20.f;              // of a row's maximum, in base 2, that rescales O: weights are 1 at most with it
constexpr int kBatch = 4;                  // blocks whose page ids are fetched together
constexpr int kUnits = 4;                  // units the producer may be ahead of the slowest warp
constexpr int kBatches = 8;                // batches the id ring holds: the producer is at most kUnits units and a
                                           // ring of slots (a batch or two) ahead of the softmax

template <int D>
struct Cfg {
  static constexpr int boxes = D / 64, tile = boxes * kBox;  // bytes of a Q, K or V tile
  // what Q leaves of 227 KB (four slots, with room to stage the output, ran 10 %
  // slower); at D = 64 eight slots are about as many bytes
  static constexpr int slots = D == 128 ? 5 : 8;
  static constexpr int o_ring = 2 * tile, o_shared = o_ring + slots * tile;
  __host__ __device__ static constexpr uint32_t col_o(int t) { return 256 + t * D; }
};

// What the warps need to know of a unit.
struct Work {
  int unit;           // -1: no more units
  int seg, h, grp, split, row0, rows;
  int pair, ahead;
  int block0, n;      // first key block, blocks
  int ns[2];          // halves each tile works on: a causal tile 0 may end before tile 1
  int pad[3];
};

// Barriers of alternate halves come in pairs: a parity wait tells two phases
// apart, and up to two halves of a tile are under way.
struct Shared {
  uint64_t full[8], empty[8], s_full[2][2], p_full[2][2], o_prev[2], o_last[2], q_full[2], drain[2];
  uint64_t v_clean[8];  // of the V blocks in turn: the helper gives back every slot, so at most 8 lie between it and an issuer
  uint64_t flags_full[2 * kUnits];  // of the units in turn: a warp is at most kUnits + 1 units behind
  uint64_t ids[kBatches], work_full[kUnits], work_empty[kUnits], response_full;
  alignas(16) uint4 response;
  alignas(16) Work work[kUnits];
  uint32_t tmem;
  int abort;
  alignas(16) uint32_t flag[2 * kUnits][8];  // per unit: partly seen keys with non-finite V values
  int32_t id[kBatches * 32];                 // page ids of recent blocks, -1: none
  alignas(16) uint16_t mask[kBatches * 32];  // their slot masks
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __noinline__ bool mbar_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  const uint64_t t0 = global_ns();
  for (uint32_t it = 1; it < (1u << 30); ++it) {
    if (mbar_try(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (abort && *abort) return false;
      if (global_ns() - t0 > limit_ns) break;
    }
  }
  if (abort) *abort = 1;
  return false;
}
// Waits for phase `parity`; false once the CTA aborts or the limit has passed
// (abort null: a wait of the abort path itself).
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  if (mbar_try(bar, parity)) return true;
  return mbar_wait_slow(bar, parity, abort, limit_ns);
}

// The same for a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, limit_ns));
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// Shared-memory matrix descriptor: 128-byte swizzle. lead: bytes between
// 64-column groups of an MN-major operand; stride: bytes between groups of 8 rows.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fff) | static_cast<uint64_t>(lead >> 4) << 16 |
         static_cast<uint64_t>(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// kind::f16 instruction descriptor: bf16 operands, fp32 accumulator, M = 128.
__host__ __device__ constexpr uint32_t instr_desc(int n, bool b_mn_major) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn_major ? 1u << 16 : 0u) | static_cast<uint32_t>(n >> 3) << 17 | (kRows >> 4) << 24;
}
// The issuing warp runs its loop with all lanes, so that descriptors stay in
// uniform registers; `leader` (one elected lane) predicates the instructions.
__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t is;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(is));
  return is;
}
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
      : "memory");
}
// Arrives on bar once the MMAs issued so far by the leader are done.
__device__ __forceinline__ void mma_commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.u32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define TKV_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define TKV_W8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])
// 32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : TKV_R8(r, 0), TKV_R8(r, 8), TKV_R8(r, 16), TKV_R8(r, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : TKV_R8(r, 0), TKV_R8(r, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::TKV_W8(r, 0),
      TKV_W8(r, 8), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::TKV_W8(r, 0),
      TKV_W8(r, 8), TKV_W8(r, 16), TKV_W8(r, 24), "r"(addr)
      : "memory");
}

// 16 bytes to shared memory
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// 32 bytes to global memory, in one access where `whole` says the address is a multiple of 32
__device__ __forceinline__ void store32(void* at, const uint32_t* v, int whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), TKV_W8(v, 0) : "memory");
  } else {
    reinterpret_cast<uint4*>(at)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(at)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// The larger magnitudes of two pairs of bf16 values; NaN wins.
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b & 0x7fff7fffu));
  return r;
}
// Zeroes the non-finite ones of two bf16 values; whether there was one.
__device__ __forceinline__ bool strip(uint32_t& w) {
  const bool lo = (w & 0x7f80u) == 0x7f80u, hi = (w & 0x7f800000u) == 0x7f800000u;
  if (lo) w &= 0xffff0000u;
  if (hi) w &= 0x0000ffffu;
  return lo || hi;
}

// Asks for the unit of a CTA that has not started; 16 bytes arrive at `to`.
__device__ __forceinline__ void request_unit(uint4* to, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(smem_u32(to)),
               "r"(smem_u32(bar))
               : "memory");
}
// The unit in a response, or -1.
__device__ __forceinline__ int response_unit(const uint4* at) {
  uint32_t got, x = 0;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 r;\n ld.shared.b128 r, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(at))
      : "memory");
  return got ? static_cast<int>(x) : -1;
}

__device__ __forceinline__ Work unit_work(const TileParams& p, int unit) {
  const TileUnit u = tile_unit(p, unit);
  const TileSeg& sg = p.seg[u.seg];
  Work w;
  w.unit = unit;
  w.seg = u.seg; w.h = u.h; w.grp = u.grp; w.split = u.split; w.row0 = u.row0; w.rows = u.rows;
  w.pair = sg.pair;
  w.ahead = w.pair ? 2 : 1;  // two halves per tile
  w.block0 = u.j0;
  w.n = u.j1 - u.j0;
  auto halves = [&](int row) {  // that row `row` sees, from block0
    return min(2 * w.n, max(0, (tile_row_limit(p, sg, row) + kHalf - 1) / kHalf - 2 * w.block0));
  };
  const int all = halves(u.row0 + u.rows - 1);
  if (w.pair) {
    w.ns[0] = (all + 1) / 2;
    w.ns[1] = all / 2;
  } else {
    w.ns[0] = u.rows > kRows ? halves(u.row0 + kRows - 1) : all;
    w.ns[1] = u.rows > kRows ? all : 0;
  }
  return w;
}

// Adds the non-finite V values of flagged keys (partly seen by the unit) to 16
// columns of a row that sees keys below lim. half: of every block the tile takes
// this half alone, -1: both. A pair's other tile adds those of the other half: a
// row may see no key of this one, and its partial's weight is 0 then.
__device__ __noinline__ void add_flagged(const TileParams& p, const uint32_t* flag, int lim_first, int lim, int half, int64_t key0,
                                         int col, uint32_t* o) {
  for (int w = 0; w < 8; ++w)
    for (uint32_t left = flag[w]; left; left &= left - 1) {
      const int key = lim_first + w * 32 + __ffs(left) - 1;
      if (key >= lim || (half >= 0 && key / kHalf % 2 != half)) continue;
      const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + (key0 + key) * p.v_stride + col;
      for (int e = 0; e < 16; ++e) {
        const float x = __bfloat162float(v[e]);
        if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
      }
    }
}

template <int D, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
    tile_mma_kernel(const __grid_constant__ TileParams p, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem + C::o_shared);
  const uint32_t s_q = smem_u32(smem), s_ring = s_q + C::o_ring;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  volatile int* abort = &sh.abort;
  const uint64_t limit = p.wait_limit_ns;

  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < C::slots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 3);  // both issuers and the helper
    }
    for (int t = 0; t < 2; ++t) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sh.s_full[t][b], 1);
        mbar_init(&sh.p_full[t][b], 4);
      }
      mbar_init(&sh.o_prev[t], 1);
      mbar_init(&sh.o_last[t], 1);
      mbar_init(&sh.q_full[t], 4);
      mbar_init(&sh.drain[t], 1);
    }
    mbar_init(&sh.response_full, 1);
    for (int i = 0; i < 8; ++i) mbar_init(&sh.v_clean[i], 1);
    for (int i = 0; i < 2 * kUnits; ++i) mbar_init(&sh.flags_full[i], 1);
    for (int i = 0; i < kBatches; ++i) mbar_init(&sh.ids[i], 1);
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&sh.work_full[i], 1);
      mbar_init(&sh.work_empty[i], kThreads / 32 - 1);  // every warp but the producer
    }
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy();
  }
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k) : "memory");
    if (!kPaged) asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v) : "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  // the set-up above may overlap the end of the kernel ahead on the stream
  cudaGridDependencySynchronize();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);

  // The CTA's k-th unit as the producer published it; unit -1 at the end or on an abort.
  auto next_work = [&](int k) {
    const int r = k % kUnits;
    Work w;
    w.unit = -1;
    if (!warp_wait(&sh.work_full[r], (k / kUnits) & 1, abort, limit)) return w;
    w = sh.work[r];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.work_empty[r]);
    return w;
  };

  if (warp == kProducer) {
    int pos = 0, batches = 0;
    int asked = -1;  // a request not answered yet
    for (int k = 0, unit = blockIdx.x;; ++k) {
      const int r = k % kUnits;
      if (k >= kUnits && !warp_wait(&sh.work_empty[r], (k / kUnits - 1) & 1, abort, limit)) break;
      Work w;
      w.unit = -1;
      if (unit >= 0) w = unit_work(p, unit);
      if (lane == 0) {
        sh.work[r] = w;
        mbar_arrive(&sh.work_full[r]);
      }
      if (unit < 0) break;
      const TileSeg& sg = p.seg[w.seg];
      // page ids and masks, a batch ahead of their use
      int32_t id_next = -1, id_after = -1;
      uint32_t mask_next = 0;
      const int npages = sg.nkeys / kPage, page0 = w.block0 * kBlockPages;
      auto fetch_id = [&](int batch) {
        const int pg = page0 + batch * 32 + lane;
        if (batch * kBatch >= w.n || pg >= npages) return -1;
        const int32_t id = p.table[sg.key0 + pg];
        return id < 0 || id >= p.pages ? -1 : id;
      };
      auto fetch_mask = [&](int32_t id) { return id < 0 ? 0u : p.mask[id] & 0xffffu; };
      if (kPaged) {
        id_next = fetch_id(0);
        id_after = fetch_id(1);
        mask_next = fetch_mask(id_next);
      }
      auto load = [&](int i, bool is_v) {
        if (kPaged && !is_v && i % kBatch == 0) {
          const int b = (batches + i / kBatch) % kBatches, at = b * 32 + lane;
          sh.id[at] = id_next;
          sh.mask[at] = static_cast<uint16_t>(mask_next);
          id_next = id_after;
          mask_next = fetch_mask(id_next);
          id_after = fetch_id(i / kBatch + 2);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.ids[b]);
        }
        const int slot = pos % C::slots, round = pos / C::slots;
        if (round > 0 && !warp_wait(&sh.empty[slot], (round - 1) & 1, abort, limit)) return false;
        ++pos;
        const uint32_t dst = s_ring + slot * C::tile;
        if (p.stall && unit == 0 && i == 0 && !is_v) return true;  // the waits on this slot run out
        if (lane == 0) mbar_expect(&sh.full[slot], C::tile);
        __syncwarp();
        if (kPaged) {
          const int pg = lane % kBlockPages, c = lane / kBlockPages;
          if (c < C::boxes) {
            const int32_t id = sh.id[(batches + i / kBatch) % kBatches * 32 + i % kBatch * kBlockPages + pg];
            const int64_t z = id < 0 ? p.pages * p.Hkv * 2 : (static_cast<int64_t>(id) * p.Hkv + w.h) * 2 + is_v;
            tma_3d(dst + c * kBox + pg * (kPage * 128), &map_k, c * 64, 0, static_cast<int>(z), &sh.full[slot]);
          }
        } else if (lane < C::boxes) {
          tma_3d(dst + lane * kBox, is_v ? &map_v : &map_k, lane * 64, w.h, static_cast<int>(sg.key0) + (w.block0 + i) * kKeyBlock,
                 &sh.full[slot]);
        }
        return true;
      };
      bool ok = true;
      for (int i = 0; ok && i < min(w.ahead, w.n); ++i) ok = load(i, false);
      for (int i = 0; ok && i < w.n; ++i) {
        ok = load(i, true);
        if (ok && i + w.ahead < w.n) ok = load(i + w.ahead, false);
      }
      if (!ok) break;
      batches += (w.n + kBatch - 1) / kBatch;
      // Ask for the next unit only now, with this one's last blocks on their way: a
      // unit claimed earlier would wait behind this one while another SM runs dry
      // (69 -> 59 us on a decode step of 128 long units and 256 short ones).
      if (lane == 0) {
        fence_proxy();
        mbar_expect(&sh.response_full, 16);
        request_unit(&sh.response, &sh.response_full);
      }
      __syncwarp();
      asked = k;
      if (!warp_wait(&sh.response_full, k & 1, abort, limit)) break;
      unit = __shfl_sync(0xffffffffu, response_unit(&sh.response), 0);
      asked = -1;
    }
    // the arrivals on the last slots come before this shared memory is another CTA's
    for (int q = max(0, pos - C::slots); q < pos; ++q)
      if (!warp_wait(&sh.empty[q % C::slots], (q / C::slots) & 1, abort, limit)) break;
    // an aborted CTA lets what is in flight land before it ends
    if (__any_sync(0xffffffffu, *abort)) {
      if (asked >= 0) warp_wait(&sh.response_full, asked & 1, nullptr, limit);
      for (int q = max(0, pos - C::slots); q < pos; ++q) warp_wait(&sh.full[q % C::slots], (q / C::slots) & 1, nullptr, limit);
    }
  } else if (warp == kIssuer || warp == kIssuer + 1) {
    const uint32_t leader = elect_leader();
    const int t = warp - kIssuer;
    constexpr uint32_t kIdescS = instr_desc(kHalf, false), kIdescO = instr_desc(D, true);
    const uint64_t desc_q = smem_desc(s_q + t * C::tile, 16, 1024);
    const uint32_t t_s = tmem + t * 2 * kHalf, t_o = tmem + C::col_o(t);
    int g0 = 0, blocks = 0, used = 0;  // halves of this tile, V blocks and units of this tile so far
    int slot = 0, slot_phase = 0;      // the ring slot to take next
    // Both issuers take every ring slot in turn and give it back, one that does
    // not use it as soon as it is full.
    auto take = [&](int* at) {
      *at = slot;
      const bool ready = warp_wait(&sh.full[slot], slot_phase, abort, limit);
      if (++slot == C::slots) {
        slot = 0;
        slot_phase ^= 1;
      }
      return ready;
    };
    auto take_v = [&](int* at) {
      const int i = blocks++;
      return take(at) && warp_wait(&sh.v_clean[i & 7], (i >> 3) & 1, abort, limit);
    };
    auto release = [&](int at) { mma_commit(leader, &sh.empty[at]); };
    // S of the tile's g-th half = Q K^T over one half of the K block
    auto qk = [&](int g, int at, int half) {
      const uint64_t b = smem_desc(s_ring + at * C::tile + half * (kHalf * 128), 16, 1024);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = ((k / 4) * kBox + (k % 4) * 32) >> 4;
        mma_ss(leader, t_s + (g & 1) * kHalf, desc_q + off, b + off, kIdescS, k > 0);
      }
      mma_commit(leader, &sh.s_full[t][g & 1]);
    };
    // O (+)= P V for the unit's h-th half of this tile
    auto pv = [&](int h, int at, int half, int mine) {
      const int g = g0 + h;
      if (!warp_wait(&sh.p_full[t][g & 1], (g >> 1) & 1, abort, limit)) return false;
      fence_after();
      const uint64_t b = smem_desc(s_ring + at * C::tile + half * (kHalf * 128), kBox, 1024);
#pragma unroll
      for (int k = 0; k < kHalf / 16; ++k)
        mma_ts(leader, t_o, t_s + (g & 1) * kHalf + k * 8, b + k * (2048 >> 4), kIdescO, h > 0 || k > 0);
      if (h == mine - 2) mma_commit(leader, &sh.o_prev[t]);
      if (h == mine - 1) mma_commit(leader, &sh.o_last[t]);
      return true;
    };
    for (int k = 0;; ++k) {
      const Work w = next_work(k);
      if (w.unit < 0) break;
      const int mine = w.ns[t];
      // a tile without rows or keys in this unit leaves the barriers of Q, S, P and O alone
      if (mine > 0) {
        if (!warp_wait(&sh.q_full[t], used++ & 1, abort, limit)) break;
        fence_after();
      }
      bool ok = true;
      if (w.pair) {
        for (int i = 0, at; i < min(2, w.n); ++i) {
          if (!(ok = take(&at))) break;
          if (i < mine) qk(g0 + i, at, t);
          release(at);
        }
        for (int i = 0, at; ok && i < w.n; ++i) {
          if (!(ok = take_v(&at))) break;
          if (i < mine && !(ok = pv(i, at, t, mine))) break;
          release(at);
          if (i + 2 < w.n) {
            if (!(ok = take(&at))) break;
            if (i + 2 < mine) qk(g0 + i + 2, at, t);
            release(at);
          }
        }
      } else {
        int at_k, at_v;
        auto qk_half = [&](int h, int half) {
          if (h < mine) qk(g0 + h, at_k, half);
        };
        if (w.n > 0) {
          if (!take(&at_k)) break;
          qk_half(0, 0);
          qk_half(1, 1);
          release(at_k);
        }
        for (int i = 0; i < w.n; ++i) {
          const int h = 2 * i;
          if (!(ok = take_v(&at_v))) break;
          if (h < mine && !(ok = pv(h, at_v, 0, mine))) break;
          if (i + 1 < w.n) {
            if (!(ok = take(&at_k))) break;
            qk_half(h + 2, 0);
          }
          if (h + 1 < mine && !(ok = pv(h + 1, at_v, 1, mine))) break;
          release(at_v);
          if (i + 1 < w.n) {
            qk_half(h + 3, 1);
            release(at_k);
          }
        }
      }
      if (!ok) break;
      g0 += mine;
    }
    if (__any_sync(0xffffffffu, *abort)) {
      mma_commit(leader, &sh.drain[t]);
      warp_wait(&sh.drain[t], 0, nullptr, limit);
    }
  } else if (warp == kHelper) {
    // Takes every ring slot in turn, K blocks too, and gives it back: a parity wait
    // on a slot is right only for who has seen its phase before and is not lapped.
    int slot = 0, slot_phase = 0, vb = 0, batches = 0;
    auto ready = [&] { return warp_wait(&sh.full[slot], slot_phase, abort, limit); };
    auto release = [&] {
      if (lane == 0) mbar_arrive(&sh.empty[slot]);
      if (++slot == C::slots) {
        slot = 0;
        slot_phase ^= 1;
      }
    };
    auto pass_k = [&] {
      if (!ready()) return false;
      release();
      return true;
    };
    for (int k = 0;; ++k) {
      const Work w = next_work(k);
      if (w.unit < 0) break;
      const TileSeg& sg = p.seg[w.seg];
      const int lim_first = tile_row_limit(p, sg, w.row0), lim_last = tile_row_limit(p, sg, w.row0 + w.rows - 1);
      uint32_t* flag = sh.flag[k % (2 * kUnits)];
      if (lane < 8) flag[lane] = 0;
      __syncwarp();
      bool ok = true;
      for (int i = 0; ok && i < min(w.ahead, w.n); ++i) ok = pass_k();
      for (int i = 0; ok && i < w.n; ++i, ++vb) {
        if (!(ok = ready())) break;
        const int k0 = (w.block0 + i) * kKeyBlock;
        if (kPaged) {
          const int b = batches + i / kBatch;
          if (!(ok = warp_wait(&sh.ids[b % kBatches], (b / kBatches) & 1, abort, limit))) break;
          const int at0 = b % kBatches * 32 + i % kBatch * kBlockPages;
          const uint16_t* mask = &sh.mask[at0];
          // two lanes per key, half of its columns each
          for (int pg = 0; pg < kBlockPages; ++pg) {
            if (mask[pg] == 0xffffu || sh.id[at0 + pg] < 0) continue;  // a page that is not there arrived as zeros
            const int key = pg * kPage + (lane >> 1);
            if ((mask[pg] >> (lane >> 1)) & 1u) continue;
            char* v = smem + C::o_ring + slot * C::tile + key * 128;
#pragma unroll 4
            for (int e = 0; e < D / 16; ++e) {
              const int c = (lane & 1) * (D / 16) + e;
              *reinterpret_cast<uint4*>(v + (c >> 3) * kBox + (((c + key) & 7) << 4)) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy();
        } else if (k0 + kKeyBlock > lim_first) {
          for (int key = max(0, lim_first - k0) + (lane >> 1); key < kKeyBlock; key += 16) {
            char* v = smem + C::o_ring + slot * C::tile + key * 128;
            uint32_t top[2] = {0, 0};  // largest magnitudes; NaN stays
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
              const int c = (lane & 1) * (D / 16) + e;
              const uint4 x = *reinterpret_cast<const uint4*>(v + (c >> 3) * kBox + (((c + key) & 7) << 4));
              top[0] = max_abs(max_abs(top[0], x.x), x.y);
              top[1] = max_abs(max_abs(top[1], x.z), x.w);
            }
            top[0] = max_abs(top[0], top[1]);
            if (!strip(top[0])) continue;
#pragma unroll 1
            for (int e = 0; e < D / 16; ++e) {
              const int c = (lane & 1) * (D / 16) + e;
              uint4* x = reinterpret_cast<uint4*>(v + (c >> 3) * kBox + (((c + key) & 7) << 4));
              strip(x->x), strip(x->y), strip(x->z), strip(x->w);
            }
            const int part = k0 + key - lim_first;
            if (k0 + key < lim_last) atomicOr(&flag[part >> 5], 1u << (part & 31));
          }
          fence_proxy();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.v_clean[vb & 7]);
        release();
        if (i + w.ahead < w.n) ok = pass_k();
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(&sh.flags_full[k % (2 * kUnits)]);
      batches += (w.n + kBatch - 1) / kBatch;
    }
  } else {
    const int t = warp >> 2, r = tid & 127, wq = warp & 3;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq) << 21);
    const uint32_t t_s = lane_base + t * 2 * kHalf, t_o = lane_base + C::col_o(t);
    const int G = p.G;
    const uint32_t gmul = (65535 + G) / G;  // (x * gmul) >> 16 = x / G for x < 320, G <= 64
    const float qs = p.qscale;
    // Q rows of a unit into the tile's shared memory, swizzled; rows past the end
    // keep what is there: a row's S, P and O depend on its own Q alone
    auto load_q = [&](const Work& w) {
      if (w.unit < 0) return;
      const TileSeg& sg = p.seg[w.seg];
      const int first = w.pair ? 0 : t * kRows, rows = min(kRows, w.rows - first);
      const int tok_base = sg.tok0 + w.row0 / G, g_base = w.row0 % G + first;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + w.h * G * D;
      constexpr int kChunks = D / 8;
      const int c = r % kChunks;
      const uint32_t dst = s_q + t * C::tile + (c >> 3) * kBox;
#pragma unroll 4
      for (int rr = r / kChunks; rr < rows; rr += kRows / kChunks) {
        const int x = g_base + rr, tok = (x * gmul) >> 16;
        cp_async16(dst + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), q + static_cast<int64_t>(tok_base + tok) * p.q_stride + (x - tok * G) * D + c * 8);
      }
    };
    int g0 = 0, batches = 0, used = 0, used2 = 0;  // used2: units with two halves or more
    Work w = next_work(0);
    load_q(w);
    for (int k = 0; w.unit >= 0; ++k) {
      const TileSeg& sg = p.seg[w.seg];
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy();
      __syncwarp();
      if (lane == 0 && w.ns[t] > 0) mbar_arrive(&sh.q_full[t]);
      const int first = w.pair ? 0 : t * kRows;  // the tile's first row in the unit
      const int rows = min(kRows, w.rows - first), mine = w.ns[t];
      const int row = w.row0 + first + min(r, max(rows - 1, 0));
      const bool valid = r < rows, active = wq * 32 < rows;  // active: the warp has rows at all
      const int lim = tile_row_limit(p, sg, row);
      const int lim_warp = __shfl_sync(0xffffffffu, lim, 0);  // limits rise with the row
      float ref = -INFINITY;           // maximum the weights refer to (unscaled logits)
      float z = 0.f, z_exact = 0.f;    // sums of the weights: rounded, not rounded
      bool ok = true;
      for (int h = 0; h < mine; ++h) {
        const int i = w.pair ? h : h >> 1, half = w.pair ? t : h & 1, g = g0 + h, buf = g & 1;
        const int k0 = (w.block0 + i) * kKeyBlock + half * kHalf;
        uint32_t live[2] = {~0u, ~0u};
        if (kPaged) {
          const int b = batches + i / kBatch;
          if (!(ok = warp_wait(&sh.ids[b % kBatches], (b / kBatches) & 1, abort, limit))) break;
          const uint2 x = *reinterpret_cast<const uint2*>(&sh.mask[b % kBatches * 32 + i % kBatch * kBlockPages + half * (kBlockPages / 2)]);
          live[0] = x.x;
          live[1] = x.y;
        }
        const bool holes = kPaged && (live[0] & live[1]) != ~0u;
        const bool cut = !kPaged && k0 + kHalf > lim_warp;

        if (!(ok = warp_wait(&sh.s_full[t][buf], (g >> 1) & 1, abort, limit))) break;
        fence_after();
        if (active) {
          uint32_t s[kHalf];
          tmem_ld32(t_s + buf * kHalf, s);
          tmem_ld32(t_s + buf * kHalf + 32, s + 32);
          wait_ld();
          if (cut) {
            const int m = lim - k0;
#pragma unroll
            for (int c = 0; c < kHalf; ++c) s[c] = c < m ? s[c] : 0xff800000u;
          }
          if (holes) {
#pragma unroll
            for (int c = 0; c < kHalf; ++c) s[c] = (live[c / 32] >> (c % 32)) & 1u ? s[c] : 0xff800000u;
          }
          if (kPaged && sg.spill0 >= 0 && valid) {
            float4* at = reinterpret_cast<float4*>(p.spill + sg.spill0 + static_cast<int64_t>(w.h * G + row % G) * sg.nkeys + k0);
#pragma unroll
            for (int c = 0; c < kHalf / 4; ++c)
              if (k0 + c * 4 < sg.nkeys)
                at[c] = make_float4(__uint_as_float(s[c * 4]) * qs, __uint_as_float(s[c * 4 + 1]) * qs,
                                    __uint_as_float(s[c * 4 + 2]) * qs, __uint_as_float(s[c * 4 + 3]) * qs);
          }
          float top[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) top[c] = max3(__uint_as_float(s[c]), __uint_as_float(s[c + 4]), __uint_as_float(s[c + 8]));
#pragma unroll
          for (int c = 12; c < 60; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) top[e] = max3(top[e], __uint_as_float(s[c + e]), __uint_as_float(s[c + 4 + e]));
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], __uint_as_float(s[60 + e]));
          const float next = fmaxf(max3(ref, top[0], top[1]), fmaxf(top[2], top[3]));
          if (__any_sync(0xffffffffu, valid && (next - ref) * qs > kRise)) {
            const float f = next == -INFINITY ? 1.f : ex2((ref - next) * qs);
            if (h > 0) {
              // the product before: behind it comes S of the next half, or for the last half its own signal
              if (h < mine - 1) ok = warp_wait(&sh.s_full[t][(g + 1) & 1], ((g + 1) >> 1) & 1, abort, limit);
              else ok = warp_wait(&sh.o_prev[t], used2 & 1, abort, limit);
              if (!ok) break;
              fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(t_o + c, o);
                wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(t_o + c, o);
              }
              z *= f;
              z_exact *= f;
            }
            ref = next;
          }
          const float base = ref == -INFINITY ? 0.f : fmaf(ref, qs, kRise);
          const float2 qs2 = make_float2(qs, qs), base2 = make_float2(-base, -base);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          auto weights = [&](auto exact) {
            float2 whole[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < kHalf / 2; ++c) {
              float2 x = fma2(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), qs2, base2);
              x.x = ex2(x.x);
              x.y = ex2(x.y);
              s[c] = pack2(x.x, x.y);
              if constexpr (decltype(exact)::value) whole[c & 1] = add2(whole[c & 1], x);
              sum[c & 1] = add2(sum[c & 1], make_float2(__uint_as_float(s[c] << 16), __uint_as_float(s[c] & 0xffff0000u)));
            }
            if constexpr (decltype(exact)::value) z_exact += (whole[0].x + whole[0].y) + (whole[1].x + whole[1].y);
          };
          if (kPaged && p.alpha) weights(std::true_type{});
          else weights(std::false_type{});
          tmem_st32(t_s + buf * kHalf, s);
          z += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        }
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[t][buf]);
      }
      // Q is free, its last S has been seen: load the next unit's while this one's O is finished
      if (!ok) break;
      const Work next = next_work(k + 1);
      load_q(next);
      if (mine > 0) {
        ok = warp_wait(&sh.o_last[t], used & 1, abort, limit);
        fence_after();
      }
      const uint32_t* flag = sh.flag[k % (2 * kUnits)];
      uint32_t flagged = 0;
      if (!kPaged && ok && mine > 0) {
        ok = warp_wait(&sh.flags_full[k % (2 * kUnits)], k / (2 * kUnits) & 1, abort, limit);
        for (int i = 0; i < 8; i += 4) {
          const uint4 f = *reinterpret_cast<const uint4*>(&flag[i]);
          flagged |= f.x | f.y | f.z | f.w;
        }
      }
      if (!ok) break;
      if (active && rows > 0) {
        const float inv = z > 0.f || z != z ? 1.f / z : 0.f;
        const bool direct = !kPaged && sg.direct;
        const int64_t part = direct ? 0 : tile_part_row(p, sg, w.grp, w.h, w.split, t);
        if (mine == 0 || (!kPaged && flagged)) {
          // no key: O was never written; or non-finite values to add, in place
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld16(t_o + c, o);
            wait_ld();
            if (mine == 0) {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = 0;
            } else {
              add_flagged(p, flag, tile_row_limit(p, sg, w.row0), lim, w.pair ? t : -1, sg.key0, w.h * D + c, o);
            }
            tmem_st16(t_o + c, o);
          }
          wait_st();
        }
        // a thread holds a row and stores it by 32-byte sectors; in a partial, neighbours' sectors touch
        const int at = w.row0 + first + r, tok = at / G;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + static_cast<int64_t>(sg.tok0 + tok) * p.out_stride +
                             (w.h * G + at - tok * G) * D;
        float* po = p.part_o + part * D + r * 8;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(t_o + c, o);
          wait_ld();
          if (!valid) continue;
          if (direct) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = pack2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
            store32(out + c, o, p.out_sectors);
            store32(out + c + 16, o + 8, p.out_sectors);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) store32(po + (c / 8 + e) * sg.part_rows * 8, o + e * 8, 1);
          }
        }
        if (!direct && valid) {
          p.part_m[part + r] = fmaf(ref, qs, kRise);  // what the weights refer to
          p.part_z[part + r] = z;
          if (kPaged && p.alpha) p.part_ze[part + r] = z_exact;
        }
      }
      fence_before();
      g0 += mine;
      used += mine > 0;
      used2 += mine > 1;
      batches += (w.n + kBatch - 1) / kBatch;
      w = next;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_before();
  }
  __syncthreads();
  if (warp == kIssuer) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
  if (tid == 0 && sh.abort) *p.status = 1;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    (void)cudaGetLastError();
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// bf16 [n2][n1][d] with strides of n1 and n2 in bytes, boxes of 64 columns.
bool encode(CUtensorMap* map, const void* base, int d, uint64_t n1, uint64_t n2, uint64_t s1, uint64_t s2, uint32_t b1, uint32_t b2) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), n1, n2}, strides[2] = {s1, s2};
  const cuuint32_t box[3] = {64, b1, b2}, elem[3] = {1, 1, 1};
  const EncodeFn fn = encode_fn();
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kPaged>
cudaError_t launch(const TileParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
  constexpr int bytes = Cfg<D>::o_shared + static_cast<int>(sizeof(Shared));
  static_assert(bytes <= 227 * 1024, "shared memory");
  static SharedMemoryOptIn opt_in;
  const cudaError_t e = opt_in.once(reinterpret_cast<const void*>(tile_mma_kernel<D, kPaged>), bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tile_mma_kernel<D, kPaged>, p, k, v);
}

}  // namespace

cudaError_t launch_tile_mma(const TileParams& p, int D, int64_t keys, cudaStream_t s) {
  CUtensorMap k, v;
  bool ok;
  if (p.paged) {
    const uint64_t row = static_cast<uint64_t>(D) * 2;
    ok = encode(&k, p.pool, D, kPage, static_cast<uint64_t>(p.pages) * p.Hkv * 2, row, row * kPage, kPage, 1);
    v = k;
  } else {
    const uint64_t head = static_cast<uint64_t>(D) * 2;
    ok = encode(&k, p.k, D, p.Hkv, keys, head, p.k_stride * 2, 1, kKeyBlock) &&
         encode(&v, p.v, D, p.Hkv, keys, head, p.v_stride * 2, 1, kKeyBlock);
  }
  if (!ok) return cudaErrorInvalidValue;
  if (p.paged) return D == 64 ? launch<64, true>(p, k, v, s) : launch<128, true>(p, k, v, s);
  return D == 64 ? launch<64, false>(p, k, v, s) : launch<128, false>(p, k, v, s);
}

}  // namespace tkv
