// bf16 tiled attention on the 5th-generation tensor cores (terms and plan:
// tile_attention.h; the mathematics: tile_attention.cu).
//
// One CTA per SM runs one unit: up to 256 rows as two tiles of 128 against a
// stream of 128-key blocks. Ten warps:
//   0-3, 4-7  softmax of tile 0 / 1: one thread per row (TMEM lane), so row
//             maxima and sums need no exchange between threads
//   8         producer: TMA of K and V blocks into a ring of shared-memory slots
//   9         issues tcgen05.mma: S = Q K^T from shared memory, O += P V with P
//             read from TMEM
// TMEM holds, per tile, S (128 fp32 columns) and O (D columns); P (bf16)
// overwrites the S it came from. While one tile is in its softmax the tensor
// cores work for the other. A segment of at most 128 rows that is split anyway
// (a decode step) runs as a PAIR: both halves hold the same rows and take
// alternate key blocks, each with a partial of its own.
//
// Running maximum: O is rescaled only when a row's maximum has risen by more
// than 2^8 over the one its weights refer to (or at the first key): the weights
// stay below 2^8, far inside bf16 and fp32, and O and Z always refer to the
// same maximum, so nothing is lost and most blocks touch O with the MMA alone.
//
// The weights are rounded to bf16 (half a step 2^-8 each, unbiased) because the
// MMA takes P and V in one type; Z sums them before that rounding, in fp32.
//
// Keys that no row of the unit sees (holes, the end of a sequence) have their V
// rows zeroed in shared memory, since 0 * NaN would reach O; keys that only
// some rows see have their non-finite V values taken out there and added at the
// end to the rows that see them.
//
// Every wait is bounded: on running out it raises the CTA's abort flag and the
// caller's status word; each role then leaves its loop, the copies and MMAs in
// flight are awaited (bounded too) and TMEM is given back.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tile_attention.h"

namespace tkv {
namespace {

constexpr int kRows = 128;
constexpr int kThreads = 320;
constexpr int kProducer = 8, kIssuer = 9;
constexpr int kBoxBytes = kKeyBlock * 128;  // 128 rows of 64 bf16 columns, 128-byte swizzle
constexpr int kBatch = 4;                   // key blocks whose page ids are fetched together
constexpr int kMaskBatches = 4;             // batches the mask ring holds

template <int D>
struct Cfg {
  static constexpr int boxes = D / 64;
  static constexpr int tile = boxes * kBoxBytes;  // bytes of a Q, K or V tile
  // Q takes 2 tiles; the ring gets what is left of 227 KB (at D = 64 eight
  // slots keep as many bytes in flight as five do at D = 128)
  static constexpr int slots = D == 128 ? 5 : 8;
  static constexpr int smem = 1024 + (2 + slots) * tile;
  __host__ __device__ static constexpr uint32_t col_o(int t) { return 256 + t * D; }
};

struct Shared {
  uint64_t full[8], empty[8], s_full[2], p_full[2], o_full[2], q_full, drain, ids[kMaskBatches];
  uint32_t tmem;
  int abort;
  uint32_t flag[8];                       // partly seen keys with non-finite V values
  int32_t id[kMaskBatches * 32];          // page ids of recent blocks, -1: none
  alignas(16) uint16_t mask[kMaskBatches * 32];  // their slot masks
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
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b),
      "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b),
      "r"(idesc), "r"(acc)
      : "memory");
}
// Arrives on bar once the MMAs issued so far by this thread are done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
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
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::TKV_W8(r, 0),
      TKV_W8(r, 8), TKV_W8(r, 16), TKV_W8(r, 24), "r"(addr)
      : "memory");
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
__device__ __forceinline__ bool bf16_finite(uint32_t bits) { return (bits & 0x7f80u) != 0x7f80u; }

// Ring position of the i-th K / V block: K blocks run `ahead` blocks ahead of V.
__device__ __forceinline__ int pos_k(int i, int ahead) { return i + max(0, i - ahead + 1); }
__device__ __forceinline__ int pos_v(int i, int ahead, int n) { return i + min(n, i + ahead); }

template <int D, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
    tile_mma_kernel(const __grid_constant__ TileParams p, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D>;
  extern __shared__ char smem_raw[];
  __shared__ Shared sh;
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s_q = smem_u32(smem), s_ring = s_q + 2 * C::tile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &sh.abort;
  const uint64_t limit = p.wait_limit_ns;

  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < C::slots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.p_full[t], 4);
      mbar_init(&sh.o_full[t], 1);
    }
    for (int i = 0; i < kMaskBatches; ++i) mbar_init(&sh.ids[i], 1);
    mbar_init(&sh.q_full, 8);
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    for (int i = 0; i < 8; ++i) sh.flag[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;

  const TileUnit u = tile_unit(p, blockIdx.x);
  const TileSeg& sg = p.seg[u.seg];
  const int pair = sg.pair, ahead = pair ? 2 : 1;
  const int n = u.j1 - u.j0;  // key blocks
  // blocks of each tile: a causal tile 0 may end before tile 1
  int nt[2];
  if (pair) {
    nt[0] = (n + 1) / 2;
    nt[1] = n / 2;
  } else {
    for (int t = 0; t < 2; ++t) {
      const int last = min((t + 1) * kRows, u.rows) - 1;
      nt[t] = last < t * kRows ? 0 : min(n, (tile_row_limit(p, sg, u.row0 + last) + kKeyBlock - 1) / kKeyBlock - u.j0);
      nt[t] = max(nt[t], 0);
    }
  }

  if (warp == kProducer) {
    int pos = 0;
    bool ok = true;
    // page ids and masks, two batches of blocks ahead of their use
    int32_t id_next = -1, id_after = -1;
    uint32_t mask_next = 0;
    const int npages = sg.nkeys / kPage;
    auto fetch_id = [&](int batch) {
      const int pg = (u.j0 + batch * kBatch) * (kKeyBlock / kPage) + lane;
      if (batch * kBatch >= n || pg >= npages) return -1;
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
        const int b = i / kBatch, at = b % kMaskBatches * 32 + lane;
        sh.id[at] = id_next;
        sh.mask[at] = static_cast<uint16_t>(mask_next);
        id_next = id_after;
        mask_next = fetch_mask(id_next);
        id_after = fetch_id(b + 2);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.ids[b % kMaskBatches]);
      }
      const int slot = pos % C::slots, round = pos / C::slots;
      ++pos;
      if (round > 0 && !warp_wait(&sh.empty[slot], (round - 1) & 1, abort, limit)) return false;
      const uint32_t dst = s_ring + slot * C::tile;
      if (lane == 0) mbar_expect(&sh.full[slot], C::tile);
      __syncwarp();
      if (kPaged) {
        const int pg = lane & 7, c = lane >> 3;
        if (c < C::boxes) {
          const int32_t id = sh.id[(i / kBatch % kMaskBatches) * 32 + i % kBatch * 8 + pg];
          const int64_t z = id < 0 ? p.pages * p.Hkv * 2 : (static_cast<int64_t>(id) * p.Hkv + u.h) * 2 + is_v;
          tma_3d(dst + c * kBoxBytes + pg * (kPage * 128), &map_k, c * 64, 0, static_cast<int>(z), &sh.full[slot]);
        }
      } else if (lane < C::boxes) {
        tma_3d(dst + lane * kBoxBytes, is_v ? &map_v : &map_k, lane * 64, u.h, static_cast<int>(sg.key0) + (u.j0 + i) * kKeyBlock,
               &sh.full[slot]);
      }
      return true;
    };
    for (int i = 0; ok && i < min(ahead, n); ++i) ok = load(i, false);
    for (int i = 0; ok && i < n; ++i) {
      ok = load(i, true);
      if (ok && i + ahead < n) ok = load(i + ahead, false);
    }
    if (!ok) --pos;  // the load that gave up was not issued
    // an aborted CTA lets the copies in flight land before it ends
    if (*abort)
      for (int q = max(0, pos - C::slots); q < pos; ++q) warp_wait(&sh.full[q % C::slots], (q / C::slots) & 1, nullptr, limit);
  } else if (warp == kIssuer) {
    if (lane == 0) {
      constexpr uint32_t kIdescS = instr_desc(kKeyBlock, false), kIdescO = instr_desc(D, true);
      auto slot_ready = [&](int pos) { return mbar_wait(&sh.full[pos % C::slots], (pos / C::slots) & 1, abort, limit); };
      auto qk = [&](int t, int pos) {
        const uint32_t a = s_q + (pair ? 0 : t) * C::tile, b = s_ring + pos % C::slots * C::tile;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k / 4) * kBoxBytes + (k % 4) * 32;
          mma_ss(tmem + t * kKeyBlock, smem_desc(a + off, 16, 1024), smem_desc(b + off, 16, 1024), kIdescS, k > 0);
        }
        mma_commit(&sh.s_full[t]);
      };
      auto pv = [&](int t, int pos, bool acc) {
        const uint32_t b = s_ring + pos % C::slots * C::tile;
#pragma unroll
        for (int k = 0; k < kKeyBlock / 16; ++k)
          mma_ts(tmem + C::col_o(t), tmem + t * kKeyBlock + k * 8, smem_desc(b + k * 2048, kBoxBytes, 1024), kIdescO, acc || k > 0);
        mma_commit(&sh.o_full[t]);
      };
      auto run = [&]() {
        if (n == 0) return;
        if (!mbar_wait(&sh.q_full, 0, abort, limit)) return;
        fence_after();
        if (pair) {
          for (int i = 0; i < min(2, n); ++i) {
            const int pk = pos_k(i, 2);
            if (!slot_ready(pk)) return;
            qk(i, pk);
            mma_commit(&sh.empty[pk % C::slots]);
          }
          for (int i = 0; i < n; ++i) {
            const int t = i & 1, pvs = pos_v(i, 2, n);
            if (!slot_ready(pvs)) return;
            if (!mbar_wait(&sh.p_full[t], (i >> 1) & 1, abort, limit)) return;
            fence_after();
            pv(t, pvs, i >= 2);
            mma_commit(&sh.empty[pvs % C::slots]);
            if (i + 2 < n) {
              const int pk = pos_k(i + 2, 2);
              if (!slot_ready(pk)) return;
              qk(t, pk);
              mma_commit(&sh.empty[pk % C::slots]);
            }
          }
          return;
        }
        if (!slot_ready(0)) return;
        for (int t = 0; t < 2; ++t)
          if (nt[t] > 0) qk(t, 0);
        mma_commit(&sh.empty[0]);
        for (int i = 0; i < n; ++i) {
          const int pvs = pos_v(i, 1, n), pk = pos_k(i + 1, 1);
          if (!slot_ready(pvs)) return;
          for (int t = 0; t < 2; ++t) {
            if (i >= nt[t]) continue;
            if (!mbar_wait(&sh.p_full[t], i & 1, abort, limit)) return;
            fence_after();
            pv(t, pvs, i > 0);
            if (i + 1 < nt[t]) {
              if (!slot_ready(pk)) return;
              qk(t, pk);
            }
          }
          mma_commit(&sh.empty[pvs % C::slots]);
          if (i + 1 < n) mma_commit(&sh.empty[pk % C::slots]);
        }
      };
      run();
      if (*abort) {
        mma_commit(&sh.drain);
        mbar_wait(&sh.drain, 0, nullptr, limit);
      }
    }
    __syncwarp();
  } else {
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    const uint32_t t_s = lane_base + t * kKeyBlock, t_o = lane_base + C::col_o(t);
    const int G = p.G;
    const int first = pair ? 0 : t * kRows;  // the tile's first row in the unit
    const int rows = min(kRows, u.rows - first);
    const int row = u.row0 + first + min(r, max(rows - 1, 0));
    const bool valid = r < rows;
    // Q tile into shared memory in the swizzled layout; rows past the end are 0
    if (!pair || t == 0) {
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
      constexpr int kChunks = D / 8;
#pragma unroll 4
      for (int i = r; i < kRows * kChunks; i += kRows) {
        const int rr = i / kChunks, c = i % kChunks;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (rr < rows) {
          const int at = u.row0 + first + rr;
          x = *reinterpret_cast<const uint4*>(q + static_cast<int64_t>(sg.tok0 + at / G) * p.q_stride + (u.h * G + at % G) * D + c * 8);
        }
        *reinterpret_cast<uint4*>(smem + t * C::tile + (c >> 3) * kBoxBytes + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = x;
      }
      fence_proxy();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.q_full);

    const int lim = tile_row_limit(p, sg, row);
    const int lim_first = tile_row_limit(p, sg, u.row0), lim_last = tile_row_limit(p, sg, u.row0 + u.rows - 1);
    const int lim_warp = __shfl_sync(0xffffffffu, lim, 0);  // limits rise with the row
    const float qs = p.qscale;
    float ref = -INFINITY, z = 0.f;  // maximum the weights refer to (unscaled logits), sum of weights
    bool ok = true;
    for (int k = 0; ok && k < nt[t]; ++k) {
      const int i = pair ? 2 * k + t : k;
      const int k0 = (u.j0 + i) * kKeyBlock;
      uint32_t live[4] = {~0u, ~0u, ~0u, ~0u};
      if (kPaged) {
        const int b = i / kBatch;
        if (!(ok = warp_wait(&sh.ids[b % kMaskBatches], (b / kMaskBatches) & 1, abort, limit))) break;
        const uint4 w = *reinterpret_cast<const uint4*>(&sh.mask[b % kMaskBatches * 32 + i % kBatch * 8]);
        live[0] = w.x; live[1] = w.y; live[2] = w.z; live[3] = w.w;
      }
      const bool holes = kPaged && (live[0] & live[1] & live[2] & live[3]) != ~0u;
      const bool cut = !kPaged && k0 + kKeyBlock > lim_warp;
      const bool clean = (holes || (!kPaged && k0 + kKeyBlock > lim_first)) && (pair || t == 0 || i >= nt[0]);

      if (!(ok = warp_wait(&sh.s_full[t], k & 1, abort, limit))) break;
      fence_after();
      uint32_t s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t_s + c * 32, s + c * 32);
      wait_ld();
      if (cut) {
        const int m = lim - k0;
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = c < m ? s[c] : 0xff800000u;
      }
      if (holes) {
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = (live[c / 32] >> (c % 32)) & 1u ? s[c] : 0xff800000u;
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 128; ++c) top[c & 3] = fmaxf(top[c & 3], __uint_as_float(s[c]));
      const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      if (kPaged && sg.spill0 >= 0 && valid) {
        float4* at = reinterpret_cast<float4*>(p.spill + sg.spill0 + static_cast<int64_t>(u.h * G + row % G) * sg.nkeys + k0);
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (k0 + c * 4 < sg.nkeys)
            at[c] = make_float4(__uint_as_float(s[c * 4]) * qs, __uint_as_float(s[c * 4 + 1]) * qs,
                                __uint_as_float(s[c * 4 + 2]) * qs, __uint_as_float(s[c * 4 + 3]) * qs);
      }
      const float next = fmaxf(ref, mx);
      if (__any_sync(0xffffffffu, (next - ref) * qs > 8.f)) {
        const float f = next == -INFINITY ? 1.f : ex2((ref - next) * qs);
        if (k > 0) {
          if (!(ok = warp_wait(&sh.o_full[t], (k - 1) & 1, abort, limit))) break;
          fence_after();
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + c, o);
            wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(t_o + c, o);
          }
          z *= f;
        }
        ref = next;
      }
      const float base = ref == -INFINITY ? 0.f : ref * qs;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float a = ex2(fmaf(__uint_as_float(s[h * 64 + 2 * c]), qs, -base));
          const float b = ex2(fmaf(__uint_as_float(s[h * 64 + 2 * c + 1]), qs, -base));
          sum[c & 3] += a + b;
          s[h * 32 + c] = pack2(a, b);
        }
        tmem_st32(t_s + h * 32, s + h * 32);
      }
      z += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (clean) {
        const int pv = pos_v(i, ahead, n), key = k0 + r;
        if (!(ok = warp_wait(&sh.full[pv % C::slots], (pv / C::slots) & 1, abort, limit))) break;
        const bool none = kPaged ? !((live[r >> 5] >> (r & 31)) & 1u) : key >= lim_last;
        if (none || (!kPaged && key >= lim_first)) {
          char* at = smem + (2 + pv % C::slots) * C::tile + r * 128;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            uint4* w = reinterpret_cast<uint4*>(at + (c >> 3) * kBoxBytes + (((c + r) & 7) << 4));
            if (none) {
              *w = make_uint4(0, 0, 0, 0);
              continue;
            }
            uint4 x = *w;
            uint32_t* e = &x.x;
            bool bad = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (!bf16_finite(e[j])) { e[j] &= 0xffff0000u; bad = true; }
              if (!bf16_finite(e[j] >> 16)) { e[j] &= 0x0000ffffu; bad = true; }
            }
            if (bad) {
              *w = x;
              atomicOr(&sh.flag[(key - lim_first) >> 5], 1u << ((key - lim_first) & 31));
            }
          }
        }
        fence_proxy();
      }
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[t]);
    }
    // flags set by either half (tile 0's, which tile 1 needs, are complete here)
    if (!kPaged) {
      if (t == 0) asm volatile("bar.sync 2, 128;" ::: "memory");
      if (t == 0) asm volatile("bar.arrive 1, 256;" ::: "memory");
      else asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    if (ok && nt[t] > 0) {
      ok = warp_wait(&sh.o_full[t], (nt[t] - 1) & 1, abort, limit);
      fence_after();
    }
    if (ok && (rows > 0)) {
      const float inv = z > 0.f || z != z ? 1.f / z : 0.f;
      const int64_t part = p.direct ? 0 : tile_part_row(p, sg, u.grp, u.h, u.split, t) + r;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + static_cast<int64_t>(sg.tok0 + row / G) * p.out_stride + (u.h * G + row % G) * D;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (nt[t] > 0) {
          tmem_ld32(t_o + c, o);
          wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (!kPaged) {
          for (int w = 0; w < 8; ++w)
            for (uint32_t left = sh.flag[w]; left; left &= left - 1) {
              const int key = lim_first + w * 32 + __ffs(left) - 1;
              if (key >= lim) continue;
              const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + (sg.key0 + key) * p.v_stride + u.h * D + c;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float x = __bfloat162float(v[e]);
                if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
              }
            }
        }
        if (!valid) continue;
        if (p.direct) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 w;
            w.x = pack2(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
            w.y = pack2(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
            w.z = pack2(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
            w.w = pack2(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
            *reinterpret_cast<uint4*>(out + c + e) = w;
          }
        } else {
          float* at = p.part_o + part * D + c;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(at + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (!p.direct && valid) {
        p.part_m[part] = ref * qs;
        p.part_z[part] = z;
      }
    }
    fence_before();
  }
  __syncthreads();
  if (warp == kIssuer) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
  if (tid == 0 && sh.abort && p.status) *p.status = 1;
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
  constexpr int bytes = Cfg<D>::smem;
  const cudaError_t e = cudaFuncSetAttribute(tile_mma_kernel<D, kPaged>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  tile_mma_kernel<D, kPaged><<<static_cast<unsigned>(p.units), kThreads, bytes, s>>>(p, k, v);
  return cudaGetLastError();
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
