// Page bookkeeping of the stateless pools: forking, freeing and compacting the
// sequences of a page table, on the device, without a host round trip.
//
// A page id has a count of the table rows that list it (0: the page is free).
// A fork lists the parent's pages once more; only a page that the child will
// append to (a last page with free slots) is copied. A new page is always the
// lowest free id, so results do not depend on timing. Each operator is a small
// plan on one CTA (per call or per sequence) and, where page data moves, a
// second launch over all layers that streams it at 16 bytes per thread; the
// plan bounds the smallest calls (latency), HBM the large ones.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "tkv.h"
#include "tkv_internal.h"

namespace tkv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMoveCtas = 152 * 8;  // one wave of 256-thread CTAs on a GB300
constexpr uint32_t kFullMask = 0xffffu;
constexpr int64_t kMaxPoolPages = int64_t(1) << 27;  // page * 16 + slot is an int32

struct PoolDesc {
  char* base;             // [layers][pages][Hkv][2][16][row]
  int64_t layer_bytes, page_bytes;
  int32_t layers, kv_rows, row_bytes;  // kv_rows = 2 * Hkv blocks of 16 rows per page
};

// Block-wide exclusive scan of one 64-bit value per thread; *total gets the sum.
__device__ unsigned long long block_scan(unsigned long long v, unsigned long long* s_warp, unsigned long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // s_warp may still be read by an earlier scan
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  unsigned long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    const unsigned long long y = s_warp[w];
    before += w < warp ? y : 0;
    all += y;
  }
  *total = all;
  return before + x - v;
}

// ---- fork

struct ForkParams {
  PoolDesc pool;
  int32_t* table;
  int64_t stride;
  int32_t* refs;
  uint32_t* mask;
  int32_t* positions;
  int64_t pages;
  int32_t n, share, max_count;
  int32_t parent[kMaxBatch], child[kMaxBatch], count[kMaxBatch];  // count: the parent's pages
  int32_t* ok;      // scratch: 1 when the plan fits
  int32_t* base;    // scratch [n + 1]: first new page of each fork
  int32_t* fresh;   // scratch: new page ids, ascending
  int32_t* status;
};

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const __grid_constant__ ForkParams p) {
  __shared__ int s_bad, s_base[kMaxBatch + 1];
  __shared__ int s_warp[kPlanWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  for (int i = 0; i < p.n; ++i) {
    if (i > 0 && p.parent[i] == p.parent[i - 1]) continue;
    const int32_t* row = p.table + p.parent[i] * p.stride;
    for (int j = tid; j < p.count[i]; j += kPlanThreads) {
      const int32_t id = row[j];
      if (id < 0 || id >= p.pages || p.refs[id] < 1) s_bad = 1;
    }
  }
  __syncthreads();
  if (s_bad) {
    if (tid == 0) {
      *p.ok = 0;
      *p.status = -1;
    }
    return;
  }
  if (tid < p.n) {
    int need = p.count[tid];
    if (p.share)
      need = need > 0 && (p.mask[p.table[p.parent[tid] * p.stride + need - 1]] & kFullMask) != kFullMask;
    s_base[tid + 1] = need;
  }
  __syncthreads();
  if (tid == 0) {
    s_base[0] = 0;
    for (int i = 0; i < p.n; ++i) s_base[i + 1] += s_base[i];
  }
  __syncthreads();
  const int need = s_base[p.n];
  // the lowest free ids: each warp looks at 16 runs of 32 ids per round
  constexpr int kRuns = 16, kRound = kPlanWarps * kRuns * 32;
  int found = 0;
  for (int64_t at = 0; found < need && at < p.pages; at += kRound) {
    uint32_t free_bits[kRuns];
    int mine = 0;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const int64_t id = at + (warp * kRuns + r) * 32 + lane;
      const bool is_free = id < p.pages && p.refs[id] == 0;
      free_bits[r] = __ballot_sync(0xffffffffu, is_free);
      mine += __popc(free_bits[r]);
    }
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    int rank = found, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
      rank += w < warp ? s_warp[w] : 0;
      all += s_warp[w];
    }
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const int k = rank + __popc(free_bits[r] & ((1u << lane) - 1));
      if (((free_bits[r] >> lane) & 1u) && k < need)
        p.fresh[k] = static_cast<int32_t>(at + (warp * kRuns + r) * 32 + lane);
      rank += __popc(free_bits[r]);
    }
    found += all;
    __syncthreads();
  }
  if (tid <= p.n) p.base[tid] = s_base[tid];
  if (tid == 0) {
    *p.ok = found >= need;
    *p.status = found >= need ? 0 : need - found;
  }
}

// Copies the 16-byte chunks of one page of one layer; the parent's page is read
// by the CTAs of all its children at about the same time, so HBM sees it once.
// Three copies of 2000 tokens, 28 layers of 4 heads at d 128: 115 MB to read and 344
// to write in 72 us, 6.4 TB/s; a copy with torch reaches 6.8. Of the 344 MB, 287
// are in HBM when the launch ends and the rest still in the L2.
__device__ __forceinline__ void copy_page(const PoolDesc& d, int layer, int64_t src, int64_t dst) {
  const int4* from = reinterpret_cast<const int4*>(d.base + layer * d.layer_bytes + src * d.page_bytes);
  int4* to = reinterpret_cast<int4*>(d.base + layer * d.layer_bytes + dst * d.page_bytes);
  const int n = static_cast<int>(d.page_bytes / 16);
  for (int i = threadIdx.x; i < n; i += kMoveThreads * 4) {
    int4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * kMoveThreads < n) x[u] = from[i + u * kMoveThreads];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * kMoveThreads < n) to[i + u * kMoveThreads] = x[u];
  }
}

__global__ void __launch_bounds__(kMoveThreads) fork_apply_kernel(const __grid_constant__ ForkParams p) {
  cudaGridDependencySynchronize();
  if (!*p.ok) return;
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x;
  const int64_t all = static_cast<int64_t>(gridDim.x) * kMoveThreads;
  // the children's rows, counts, masks and positions
  for (int64_t w = tid; w < static_cast<int64_t>(p.n) * p.max_count; w += all) {
    const int i = static_cast<int>(w / p.max_count), j = static_cast<int>(w % p.max_count);
    if (j >= p.count[i]) continue;
    const int32_t from = p.table[p.parent[i] * p.stride + j];
    int32_t id = from;
    const int base = p.base[i], need = p.base[i + 1] - base;
    if (!p.share) id = p.fresh[base + j];
    else if (need && j == p.count[i] - 1) id = p.fresh[base];
    p.table[p.child[i] * p.stride + j] = id;
    if (id == from) {
      atomicAdd(p.refs + id, 1);
    } else {
      p.refs[id] = 1;
      p.mask[id] = p.mask[from];
      if (p.positions)
        for (int s = 0; s < kPage; ++s) p.positions[static_cast<int64_t>(id) * kPage + s] = p.positions[static_cast<int64_t>(from) * kPage + s];
    }
  }
  // the pages' data: one (layer, page) per CTA at a time, children of a page side by side
  const int per = p.share ? 1 : p.max_count;
  const int64_t records = static_cast<int64_t>(p.pool.layers) * per * p.n;
  for (int64_t w = blockIdx.x; w < records; w += gridDim.x) {
    const int i = static_cast<int>(w % p.n);
    const int j = p.share ? p.count[i] - 1 : static_cast<int>(w / p.n % per);
    const int layer = static_cast<int>(w / (static_cast<int64_t>(p.n) * per));
    const int base = p.base[i];
    if (j < 0 || j >= p.count[i] || p.base[i + 1] == base) continue;
    copy_page(p.pool, layer, p.table[p.parent[i] * p.stride + j], p.fresh[p.share ? base : base + j]);
  }
}

// ---- free

struct FreeParams {
  int32_t* table;
  int64_t stride;
  int32_t* refs;
  uint32_t* mask;
  int64_t pages;
  int32_t n, max_count;
  int32_t seq[kMaxBatch], count[kMaxBatch];
  int32_t* status;
};

__global__ void __launch_bounds__(kMoveThreads) free_kernel(const __grid_constant__ FreeParams p) {
  const int64_t all = static_cast<int64_t>(gridDim.x) * kMoveThreads;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x;
       w < static_cast<int64_t>(p.n) * p.max_count; w += all) {
    const int i = static_cast<int>(w / p.max_count), j = static_cast<int>(w % p.max_count);
    if (j >= p.count[i]) continue;
    int32_t* at = p.table + p.seq[i] * p.stride + j;
    const int32_t id = *at;
    *at = -1;
    if (id < 0 || id >= p.pages) {
      *p.status = -1;
      continue;
    }
    const int old = atomicSub(p.refs + id, 1);
    if (old < 1) {  // not held: put the count back
      atomicAdd(p.refs + id, 1);
      *p.status = -1;
    } else if (old == 1) {
      p.mask[id] = 0;
    }
  }
}

// ---- compact

struct CompactParams {
  PoolDesc pool;
  int32_t* table;
  int64_t stride;
  int32_t* refs;       // null: every listed page belongs to its row alone
  uint32_t* mask;
  int32_t* positions;
  int64_t pages;
  int32_t n;
  int32_t count[kMaxBatch];
  int64_t move0[kMaxBatch];  // first entry of each sequence in from / to
  int32_t* moves;      // scratch [n]: tokens each sequence moves
  int32_t *from, *to;  // scratch: page * 16 + slot
  int32_t* new_counts;
};

// One CTA per sequence, kPer consecutive pages per thread (16384 pages are the
// most; a row of 288 took 19 us with 16 per thread, 9 with one). Private pages in
// list order keep the first ceil(tokens / 16) of them; the valid slots of the
// rest, in order, fill the holes of those kept, in order. Shared pages stay as
// they are.
template <int kPer>
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const __grid_constant__ CompactParams p) {
  __shared__ unsigned long long s_warp[kPlanWarps];
  __shared__ int s_bad;
  const int b = blockIdx.x, tid = threadIdx.x, n = p.count[b];
  int32_t* row = p.table + b * p.stride;
  const int j0 = tid * kPer;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  int32_t id[kPer];
  uint32_t bits[kPer];
  uint32_t mine = 0;  // bit i: page j0 + i is private
  unsigned long long sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    id[i] = -1;
    bits[i] = 0;
    if (j0 + i >= n) continue;
    id[i] = row[j0 + i];
    if (id[i] < 0 || id[i] >= p.pages) {
      s_bad = 1;
      continue;
    }
    const int32_t held = p.refs ? p.refs[id[i]] : 1;
    if (held < 1) s_bad = 1;
    if (held != 1) continue;
    bits[i] = p.mask[id[i]] & kFullMask;
    mine |= 1u << i;
    sum += (1ull << 32) | __popc(bits[i]);
  }
  __syncthreads();
  if (s_bad) {  // nothing of this sequence changes
    if (tid == 0) {
      p.moves[b] = 0;
      p.new_counts[b] = -1;
    }
    return;
  }
  unsigned long long total;
  int rank = static_cast<int>(block_scan(sum, s_warp, &total) >> 32);
  const int tokens = static_cast<int>(total & 0xffffffffu), keep = (tokens + kPage - 1) / kPage;
  uint32_t front = 0;  // private pages that stay
  unsigned long long hm = 0;
  int stay = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (id[i] < 0) continue;
    if (!((mine >> i) & 1u)) {
      ++stay;
      continue;
    }
    if (rank++ < keep) {
      front |= 1u << i;
      ++stay;
      hm += static_cast<unsigned long long>(kPage - __popc(bits[i])) << 40;
    } else {
      hm += static_cast<unsigned long long>(__popc(bits[i])) << 20;
    }
  }
  // holes of the pages kept, tokens that move, pages that stay: 24, 20 and 20 bits
  unsigned long long all;
  const unsigned long long before = block_scan(hm | static_cast<unsigned long long>(stay), s_warp, &all);
  int at = static_cast<int>(before & 0xfffffu), mover = static_cast<int>(before >> 20 & 0xfffffu), hole = static_cast<int>(before >> 40);
  const int kept = static_cast<int>(all & 0xfffffu), movers = static_cast<int>(all >> 20 & 0xfffffu);
  int32_t* from = p.from + p.move0[b];
  int32_t* to = p.to + p.move0[b];
  // every read of the row came before the scans' barriers
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (id[i] < 0) continue;
    const bool is_front = (front >> i) & 1u, is_tail = ((mine >> i) & 1u) && !is_front;
    if (is_front) {
      uint32_t holes = ~bits[i] & kFullMask;
      while (holes && hole < movers) {
        const int s = __ffs(holes) - 1;
        holes &= holes - 1;
        bits[i] |= 1u << s;
        to[hole++] = id[i] * kPage + s;
      }
      hole += __popc(holes);
      p.mask[id[i]] = bits[i];
    } else if (is_tail) {
      for (uint32_t left = bits[i]; left; left &= left - 1) from[mover++] = id[i] * kPage + __ffs(left) - 1;
      p.mask[id[i]] = 0;
      if (p.refs) p.refs[id[i]] = 0;
      if (p.positions)  // its tokens' slots are emptied by the move
        for (uint32_t left = ~bits[i] & kFullMask; left; left &= left - 1)
          p.positions[static_cast<int64_t>(id[i]) * kPage + __ffs(left) - 1] = -1;
    }
    if (!is_tail) row[at++] = id[i];
  }
  __syncthreads();
  for (int j = kept + tid; j < n; j += kPlanThreads) row[j] = -1;
  if (tid == 0) {
    p.moves[b] = movers;
    p.new_counts[b] = kept;
  }
}

// One warp per moved token of the CTA's layer (blockIdx.y): its 2 * Hkv rows, 16
// bytes per lane, four in flight. Index arithmetic is 32-bit and by shifts: with
// divisions the issue slots, not HBM, were the bound. 264 MB to read and write: 41
// us, 6.4 TB/s (a copy with torch: 6.8); 217 MB of it pass HBM within the launch.
__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(const __grid_constant__ CompactParams p) {
  __shared__ int s_first[kMaxBatch + 1];
  cudaGridDependencySynchronize();
  if (threadIdx.x == 0) {
    int at = 0;
    for (int b = 0; b < p.n; ++b) {
      s_first[b] = at;
      at += p.moves[b];
    }
    s_first[p.n] = at;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, tokens = s_first[p.n];
  const int log_chunks = 31 - __clz(p.pool.row_bytes / 16);  // 16-byte chunks of a row: 8, 16 or 32
  const int work = p.pool.kv_rows << log_chunks;             // of a token
  const int block = kPage * p.pool.row_bytes;                // from a row to the next head's, or K's to V's
  char* base = p.pool.base + blockIdx.y * p.pool.layer_bytes;
  for (int k = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); k < tokens; k += gridDim.x * (kMoveThreads / 32)) {
    int lo = 0, hi = p.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_first[mid] <= k) lo = mid; else hi = mid - 1;
    }
    const int64_t at = p.move0[lo] + k - s_first[lo];
    const int32_t from = p.from[at], to = p.to[at];
    if (blockIdx.y == 0 && p.positions && lane == 0) {  // a token's slot is read here alone, so it can be emptied here
      p.positions[to] = p.positions[from];
      p.positions[from] = -1;
    }
    const char* src = base + (from / kPage) * p.pool.page_bytes + (from % kPage) * p.pool.row_bytes;
    char* dst = base + (to / kPage) * p.pool.page_bytes + (to % kPage) * p.pool.row_bytes;
    for (int i = lane; i < work; i += 32 * 4) {
      int4 x[4];
      int off[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = i + 32 * u;
        off[u] = (c >> log_chunks) * block + (c & ((1 << log_chunks) - 1)) * 16;
        if (c < work) x[u] = *reinterpret_cast<const int4*>(src + off[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + 32 * u < work) *reinterpret_cast<int4*>(dst + off[u]) = x[u];
    }
  }
}

// ---- host side

// Launches `kernel` so that its CTAs may start while the plan ahead of it on
// the stream ends (each waits for the plan before it reads).
template <typename P>
cudaError_t launch_after(void (*kernel)(P), const P& p, dim3 ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = ctas;
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

bool misaligned(const void* ptr, size_t to) { return reinterpret_cast<uintptr_t>(ptr) % to != 0; }
size_t align256(size_t x) { return (x + 255) / 256 * 256; }

int check_pool(PoolDesc* d, void* pool, int32_t n_layers, int64_t pool_pages, int32_t n_kv_heads, int32_t head_dim, int32_t kv_dtype) {
  if (n_layers < 1 || n_layers > 65535 || n_kv_heads < 1 || n_kv_heads > 65535 || pool_pages < 1 || pool_pages > kMaxPoolPages)
    return report(TKV_ERR_INVALID_ARG, "bad pool shape");
  if (head_dim != 64 && head_dim != 128) return report(TKV_ERR_INVALID_ARG, "head_dim must be 64 or 128");
  if (kv_dtype != TKV_DTYPE_F32 && kv_dtype != TKV_DTYPE_BF16) return report(TKV_ERR_INVALID_ARG, "kv_dtype");
  if (!pool) return report(TKV_ERR_INVALID_ARG, "null pointer");
  if (misaligned(pool, 16)) return report(TKV_ERR_INVALID_ARG, "pool not 16-byte aligned");
  d->base = static_cast<char*>(pool);
  d->layers = n_layers;
  d->kv_rows = 2 * n_kv_heads;
  d->row_bytes = head_dim * (kv_dtype == TKV_DTYPE_BF16 ? 2 : 4);
  d->page_bytes = static_cast<int64_t>(d->kv_rows) * kPage * d->row_bytes;
  d->layer_bytes = pool_pages * d->page_bytes;
  return TKV_OK;
}

int check_rows(int32_t rows, int32_t max_pages, const int32_t* page_counts) {
  if (rows < 1 || max_pages < 1 || max_pages > kMaxSeqPages)
    return report(TKV_ERR_INVALID_ARG, "max_pages must be 1 to %d, rows at least 1", kMaxSeqPages);
  if (!page_counts) return report(TKV_ERR_INVALID_ARG, "null pointer");
  for (int i = 0; i < rows; ++i)
    if (page_counts[i] < 0 || page_counts[i] > max_pages)
      return report(TKV_ERR_INVALID_ARG, "page_counts[%d] out of 0..max_pages", i);
  return TKV_OK;
}

struct ForkScratch {
  size_t o_base, o_fresh, bytes;
};
ForkScratch fork_scratch(int32_t n, int64_t most) {
  ForkScratch s;
  s.o_base = 256;
  s.o_fresh = s.o_base + align256(static_cast<size_t>(n + 1) * 4);
  s.bytes = s.o_fresh + align256(static_cast<size_t>(most) * 4);
  return s;
}

int fork_check(int32_t rows, int32_t max_pages, const int32_t* page_counts, int32_t n, const int32_t* parents,
               const int32_t* children, int32_t share, int64_t* most) {
  if (int st = check_rows(rows, max_pages, page_counts)) return st;
  if (n < 1 || n > kMaxBatch) return report(TKV_ERR_INVALID_ARG, "1 to %d forks per call", kMaxBatch);
  if (!parents || !children) return report(TKV_ERR_INVALID_ARG, "null pointer");
  *most = 0;
  bool parent_empty = false;  // a child's row is empty, so only an empty parent can be a child too
  for (int i = 0; i < n; ++i) {
    if (parents[i] < 0 || parents[i] >= rows || children[i] < 0 || children[i] >= rows)
      return report(TKV_ERR_INVALID_ARG, "fork %d: row out of range", i);
    if (page_counts[children[i]] != 0) return report(TKV_ERR_INVALID_ARG, "fork %d: the child's row holds pages", i);
    parent_empty |= page_counts[parents[i]] == 0;
    *most += share ? 1 : page_counts[parents[i]];
  }
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < i; ++j)
      if (children[j] == children[i]) return report(TKV_ERR_INVALID_ARG, "fork %d: a child listed twice", i);
  for (int i = 0; parent_empty && i < n; ++i)
    for (int j = 0; j < n; ++j)
      if (parents[j] == children[i]) return report(TKV_ERR_INVALID_ARG, "fork %d: a child that is a parent too", i);
  return TKV_OK;
}

struct CompactScratch {
  size_t o_from, o_to, bytes;
};
// A sequence of n pages moves at most 8 n tokens: they come out of the pages
// given up and go into those kept, and one of the two is at most half of them.
CompactScratch compact_scratch(int64_t pages) {
  CompactScratch s;
  s.o_from = align256(kMaxBatch * 4);
  s.o_to = s.o_from + align256(static_cast<size_t>(pages) * 8 * 4);
  s.bytes = s.o_to + align256(static_cast<size_t>(pages) * 8 * 4);
  return s;
}

int bind(void* scratch, size_t bytes, size_t need) {
  if (!scratch) return report(TKV_ERR_INVALID_ARG, "null scratch: need %zu bytes", need);
  if (bytes < need) return report(TKV_ERR_CAPACITY, "scratch too small: need %zu bytes", need);
  if (misaligned(scratch, 256)) return report(TKV_ERR_INVALID_ARG, "scratch not 256-byte aligned");
  return TKV_OK;
}

int ctas_for(int64_t items) { return static_cast<int>(std::min<int64_t>(std::max<int64_t>(items, 1), kMoveCtas)); }

int launched(const char* what, cudaError_t e) {
  return e == cudaSuccess ? TKV_OK : report(TKV_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
}

}  // namespace
}  // namespace tkv

using namespace tkv;

extern "C" {

tkv_status tkv_fork_sequences_scratch_size(int32_t rows, int32_t max_pages, const int32_t* page_counts, int32_t n_forks,
                                           const int32_t* parents, const int32_t* children, int32_t share,
                                           size_t* scratch_bytes) {
  if (!scratch_bytes) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  int64_t most;
  if (int st = fork_check(rows, max_pages, page_counts, n_forks, parents, children, share, &most)) return tkv_status(st);
  *scratch_bytes = fork_scratch(n_forks, most).bytes;
  return TKV_OK;
}

tkv_status tkv_fork_sequences(void* pool, int32_t n_layers, int64_t pool_pages, int32_t n_kv_heads, int32_t head_dim,
                              int32_t kv_dtype, int32_t* page_table, int32_t rows, int32_t max_pages,
                              const int32_t* page_counts, int32_t* page_refs, uint32_t* slot_mask, int32_t* positions,
                              int32_t n_forks, const int32_t* parents, const int32_t* children, int32_t share,
                              void* scratch, size_t scratch_bytes, int32_t* status, tkv_stream stream) {
  ForkParams p{};
  int64_t most;
  if (int st = check_pool(&p.pool, pool, n_layers, pool_pages, n_kv_heads, head_dim, kv_dtype)) return tkv_status(st);
  if (int st = fork_check(rows, max_pages, page_counts, n_forks, parents, children, share, &most)) return tkv_status(st);
  if (!page_table || !page_refs || !slot_mask || !status) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  const ForkScratch sc = fork_scratch(n_forks, most);
  if (int st = bind(scratch, scratch_bytes, sc.bytes)) return tkv_status(st);
  p.table = page_table; p.stride = max_pages;
  p.refs = page_refs; p.mask = slot_mask; p.positions = positions;
  p.pages = pool_pages;
  p.n = n_forks; p.share = share != 0;
  for (int i = 0; i < n_forks; ++i) {
    p.parent[i] = parents[i];
    p.child[i] = children[i];
    p.count[i] = page_counts[parents[i]];
    p.max_count = std::max(p.max_count, p.count[i]);
  }
  p.ok = static_cast<int32_t*>(scratch);
  p.base = reinterpret_cast<int32_t*>(static_cast<char*>(scratch) + sc.o_base);
  p.fresh = reinterpret_cast<int32_t*>(static_cast<char*>(scratch) + sc.o_fresh);
  p.status = status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  fork_plan_kernel<<<1, kPlanThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return tkv_status(launched("fork plan", e));
  const int64_t records = static_cast<int64_t>(n_layers) * (p.share ? 1 : p.max_count) * n_forks;
  const int64_t entries = static_cast<int64_t>(n_forks) * p.max_count / kMoveThreads;
  return tkv_status(launched("fork", launch_after(fork_apply_kernel, p, ctas_for(std::max(records, entries)), st)));
}

tkv_status tkv_free_sequences(int32_t* page_table, int32_t rows, int32_t max_pages, const int32_t* page_counts,
                              int64_t pool_pages, int32_t* page_refs, uint32_t* slot_mask, int32_t n_seqs,
                              const int32_t* seqs, int32_t* status, tkv_stream stream) {
  if (int st = check_rows(rows, max_pages, page_counts)) return tkv_status(st);
  if (n_seqs < 1 || n_seqs > kMaxBatch) return tkv_status(report(TKV_ERR_INVALID_ARG, "1 to %d sequences per call", kMaxBatch));
  if (pool_pages < 1 || pool_pages > kMaxPoolPages) return tkv_status(report(TKV_ERR_INVALID_ARG, "bad pool shape"));
  if (!page_table || !page_refs || !slot_mask || !seqs || !status) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  FreeParams p{};
  p.table = page_table; p.stride = max_pages;
  p.refs = page_refs; p.mask = slot_mask;
  p.pages = pool_pages;
  p.n = n_seqs;
  p.status = status;
  for (int i = 0; i < n_seqs; ++i) {
    if (seqs[i] < 0 || seqs[i] >= rows) return tkv_status(report(TKV_ERR_INVALID_ARG, "sequence %d: row out of range", i));
    for (int j = 0; j < i; ++j)
      if (seqs[j] == seqs[i]) return tkv_status(report(TKV_ERR_INVALID_ARG, "sequence %d: a row listed twice", i));
    p.seq[i] = seqs[i];
    p.count[i] = page_counts[seqs[i]];
    p.max_count = std::max(p.max_count, p.count[i]);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int32_t), st);
  if (e != cudaSuccess) return tkv_status(report(TKV_ERR_CUDA, "cudaMemsetAsync failed: %s", cudaGetErrorString(e)));
  if (p.max_count == 0) return TKV_OK;
  free_kernel<<<ctas_for((static_cast<int64_t>(n_seqs) * p.max_count + kMoveThreads - 1) / kMoveThreads), kMoveThreads, 0, st>>>(p);
  return tkv_status(launched("free", cudaGetLastError()));
}

tkv_status tkv_compact_sequences_scratch_size(int32_t rows, int32_t max_pages, const int32_t* page_counts, size_t* scratch_bytes) {
  if (!scratch_bytes) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  if (int st = check_rows(rows, max_pages, page_counts)) return tkv_status(st);
  if (rows > kMaxBatch) return tkv_status(report(TKV_ERR_INVALID_ARG, "1 to %d sequences per call", kMaxBatch));
  int64_t pages = 0;
  for (int i = 0; i < rows; ++i) pages += page_counts[i];
  *scratch_bytes = compact_scratch(pages).bytes;
  return TKV_OK;
}

tkv_status tkv_compact_sequences(void* pool, int32_t n_layers, int64_t pool_pages, int32_t n_kv_heads, int32_t head_dim,
                                 int32_t kv_dtype, int32_t* page_table, int32_t rows, int32_t max_pages,
                                 const int32_t* page_counts, int32_t* page_refs, uint32_t* slot_mask, int32_t* positions,
                                 int32_t* new_counts, void* scratch, size_t scratch_bytes, tkv_stream stream) {
  CompactParams p{};
  size_t need;
  if (int st = check_pool(&p.pool, pool, n_layers, pool_pages, n_kv_heads, head_dim, kv_dtype)) return tkv_status(st);
  if (tkv_status st = tkv_compact_sequences_scratch_size(rows, max_pages, page_counts, &need)) return st;
  if (!page_table || !slot_mask || !new_counts) return tkv_status(report(TKV_ERR_INVALID_ARG, "null pointer"));
  if (int st = bind(scratch, scratch_bytes, need)) return tkv_status(st);
  p.table = page_table; p.stride = max_pages;
  p.refs = page_refs; p.mask = slot_mask; p.positions = positions;
  p.pages = pool_pages;
  p.n = rows;
  int64_t pages = 0;
  for (int i = 0; i < rows; ++i) {
    p.count[i] = page_counts[i];
    p.move0[i] = pages * 8;
    pages += page_counts[i];
  }
  const CompactScratch sc = compact_scratch(pages);
  p.moves = static_cast<int32_t*>(scratch);
  p.from = reinterpret_cast<int32_t*>(static_cast<char*>(scratch) + sc.o_from);
  p.to = reinterpret_cast<int32_t*>(static_cast<char*>(scratch) + sc.o_to);
  p.new_counts = new_counts;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int32_t most = *std::max_element(page_counts, page_counts + rows);
  if (most <= kPlanThreads) compact_plan_kernel<1><<<rows, kPlanThreads, 0, st>>>(p);
  else if (most <= 4 * kPlanThreads) compact_plan_kernel<4><<<rows, kPlanThreads, 0, st>>>(p);
  else compact_plan_kernel<kMaxSeqPages / kPlanThreads><<<rows, kPlanThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return tkv_status(launched("compact plan", e));
  return tkv_status(launched("compact", launch_after(compact_move_kernel, p, dim3(std::max(1, ctas_for(pages * n_layers) / n_layers), n_layers), st)));
}

}  // extern "C"
