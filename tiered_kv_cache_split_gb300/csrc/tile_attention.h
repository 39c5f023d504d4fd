// Shared by the tiled attention kernels (prompt attention and shared-prefix
// decode attention): how a call is cut into segments, units and partials.
//
// A SEGMENT is a run of query tokens over one list of keys: a packed prompt, a
// prefix seen by the whole batch, or a sequence's own pages. The G query heads
// that share a KV head are rows of one matrix, row = token * G + g, so a K / V
// element is read once for all of them and a short segment still fills a tile.
// A UNIT (one CTA) is (segment, row group, KV head, split): the rows of the
// group over a range of 128-key blocks. A unit that covers all keys of its rows
// writes the output (unless it is half a pair's); otherwise it writes a PARTIAL
// (m, Z, unnormalised O) per row, in base 2, and the merge kernel joins the
// partials of each row. O of a
// partial tile lies as [D / 8][rows][8]: a thread per row then stores whole lines
// with its neighbours (and the merge reads whole 32-byte sectors).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "tkv_internal.h"

namespace tkv {

constexpr int kKeyBlock = 128;              // keys of a block, the unit of splitting
constexpr int kMaxSegs = kMaxBatch + 1;
constexpr int kMaxBands = 2 * kMaxSegs;
constexpr int kMaxGroup = 64;               // query heads per KV head

struct TileSeg {
  int64_t key0;      // packed: first key token; paged: first entry of its pages in the page table
  int64_t part0;     // first partial row
  int64_t spill0;    // first spilled logit of head 0 (row stride nkeys per query head), -1: none
  int32_t tok0;      // first query token
  int32_t ntok;      // query tokens
  int32_t nkeys;     // keys (paged: 16 per page)
  int32_t see0;      // causal: token i sees keys [0, see0 + i]
  int32_t splits;    // key ranges per row group (0: the segment has no unit)
  int32_t lead;      // 0: even ranges; else blocks of each range but the last, which has the rest
  int32_t groups;    // row groups
  int32_t part_rows; // rows per partial tile
  int32_t pair;      // 1: one row tile, its two halves of the CTA take alternate key blocks
  int32_t direct;    // 1: its units write the output, else partials
};

struct TileParams {
  const void* q;
  int64_t q_stride;            // elements from one token to the next
  void* out;
  int64_t out_stride;
  int32_t out_sectors;         // 1: rows of out start on multiples of 32 bytes
  const void *k, *v;           // packed keys and values [token][Hkv][D]
  int64_t k_stride, v_stride;
  const void* pool;            // paged: [pages][Hkv][2][16][D]
  const int32_t* table;
  const uint32_t* mask;
  int64_t pages;               // pool pages: ids outside read as empty pages
  float *part_o, *part_m, *part_z;
  float* part_ze;              // Z of unrounded weights, for alpha (fp32: part_z)
  float* spill;
  float* alpha;                // [B][Hkv][alpha slots], or null
  int64_t alpha_stride_h;
  int64_t alpha_first;         // slots ahead of a sequence's own pages
  int32_t* status;             // set to 1 by a wait that gave up: the caller's word, or the device's in host memory
  unsigned long long wait_limit_ns;
  int32_t stall;               // test hook: the CTA of unit 0 withholds its first copy
  float qscale;                // log2(e) / sqrt(D): logits are kept in base 2
  int32_t Hq, Hkv, G;
  int32_t nseg, units;
  int32_t merge_tokens;        // of segments whose units write partials (paged: all)
  int32_t paged, causal;
  int32_t tile_rows, tpg;      // rows of a tile, tiles of a row group
  TileSeg seg[kMaxSegs];
  // Units are numbered by bands, longest first: band i is row groups top, top - 1,
  // .. of a segment (a causal segment's later rows see more keys), each with all
  // KV heads and `splits` key ranges from split0, and has units first_unit .. the
  // next band's.
  struct Band {
    int32_t first_unit, top;
    int32_t seg, split0, splits;
  };
  int32_t nbands;
  Band band[kMaxBands];
};

struct TileUnit {
  int seg, h, split;
  int grp;
  int row0, rows;  // rows of the segment's matrix
  int j0, j1;      // key blocks
};

// keys seen by row r of a segment
__device__ __forceinline__ int tile_row_limit(const TileParams& p, const TileSeg& s, int row) {
  return p.causal ? min(s.nkeys, s.see0 + row / p.G + 1) : s.nkeys;
}

__device__ __forceinline__ TileUnit tile_unit(const TileParams& p, int u) {
  TileUnit t;
  int lo = 0, hi = p.nbands - 1;  // the last band whose first unit is <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.band[mid].first_unit <= u) lo = mid; else hi = mid - 1;
  }
  const TileParams::Band& band = p.band[lo];
  t.seg = band.seg;
  const TileSeg& s = p.seg[t.seg];
  uint32_t r = u - band.first_unit;
  t.split = band.split0 + r % static_cast<uint32_t>(band.splits);
  r /= static_cast<uint32_t>(band.splits);
  t.h = r % static_cast<uint32_t>(p.Hkv);
  t.grp = band.top - static_cast<int>(r / static_cast<uint32_t>(p.Hkv));  // a causal segment's last rows see most keys: they go first
  const int per = s.pair ? p.tile_rows : p.tile_rows * p.tpg;
  t.row0 = t.grp * per;
  t.rows = min(per, s.ntok * p.G - t.row0);
  const int nb = (tile_row_limit(p, s, t.row0 + t.rows - 1) + kKeyBlock - 1) / kKeyBlock;
  if (s.lead) {
    t.j0 = min(nb, t.split * s.lead);
    t.j1 = min(nb, t.j0 + s.lead);
  } else {  // even ranges, the first nb % splits one block longer
    const int each = nb / s.splits, longer = nb % s.splits;
    t.j0 = t.split * each + min(t.split, longer);
    t.j1 = t.j0 + each + (t.split < longer);
  }
  return t;
}

// first partial row of tile `tile` of a unit
__device__ __forceinline__ int64_t tile_part_row(const TileParams& p, const TileSeg& s, int grp, int h, int split, int tile) {
  return s.part0 + (((static_cast<int64_t>(grp) * p.Hkv + h) * s.splits + split) * p.tpg + tile) * s.part_rows;
}

// The dynamic shared memory limit of a kernel, raised once per device.
struct SharedMemoryOptIn {
  std::atomic<bool> done[64] = {};
  cudaError_t once(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
    return e;
  }
};

// tile_attention_mma.cu: the units of a bf16 call; keys: packed key tokens
cudaError_t launch_tile_mma(const TileParams& p, int D, int64_t keys, cudaStream_t s);

}  // namespace tkv
