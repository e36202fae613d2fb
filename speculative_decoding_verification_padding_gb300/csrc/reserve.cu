// reserve.cu — sv_reserve_kv: the blocks, cache slots and positions of a
// step's rows, built on the GPU from the requests' lengths; sv_slot_windows:
// the row windows that keep what was not served out of the step.
//
// The counterpart of sv_commit_kv's release: entries [ctx / 16,
// ceil((ctx + rows) / 16)) of a request's table that are -1 are new.  With
// n_i new blocks for request i and S_i = n_0 + .. + n_i, request i is served
// iff n_i = 0 or S_i <= free count, so the served ones are a prefix of those
// that need blocks, and new block k overall (in (request, table index)
// order) is free_list[free - 1 - k].
//
// Bound: latency.  A step moves a few KB; what costs is the chain offsets,
// lengths -> table entries -> scan -> free list -> stores, and the search for
// every row's request.  One CTA walks the chain with every list spread flat
// over its threads (entries and rows, not requests, so that one long request
// costs no more than many short ones), the per-request state in shared memory.
// With more rows than threads, a cluster of up to eight CTAs walks it side by
// side, each with the whole per-request state and a share of the rows: only
// the first writes tables and counts, and what a row's check finds wrong is
// told to all.  More rows than shared memory holds go to a second launch.
// Measured: see the figures at kClusterRows.

#include <limits.h>

#include "sv_internal.cuh"

namespace sv {
namespace rsv {

struct Args {
  const int32_t* cu;
  const int32_t* parent;      // null: chains
  const int32_t* ctx;
  const int32_t* pos_offset;  // null: 0
  int32_t* tables;
  const int32_t* free_list;
  int32_t* free_count;
  int32_t* slots;
  int32_t* positions;
  int32_t* taken;
  int32_t* dev_status;
  int R, N, max_rows, max_blocks, num_blocks, capacity;
  int inline_rows;  // this launch writes slots and positions too
  int cluster;      // CTAs that share the rows
};

constexpr int kMaxRequests = 8192;  // five ints of shared memory each
// A CTA's share of the rows before another CTA joins its cluster.  Measured
// with a copy of the tables before every call taken off: one chain 4.0 us, 256
// chains of 5 rows 6.9, 512 of 2 to 9 (2816 rows) 8.0 (9.0 with twice the
// share), 256 of 17 7.6 (17.6 in one CTA and a second launch), 2000 of 5 13.7
// (27.6).
constexpr int kClusterRows = 1024;
constexpr int kMaxCluster = 8;
constexpr size_t kMaxSmem = 200 * 1024;  // more: the rows go to a second launch
constexpr size_t kFreeSmem = 47 * 1024;  // less may be had unasked: 48 KB with the kernel's own scan words
// Chains without parents have nothing to check: from here on a second launch
// over all SMs is faster (75000 rows 12.7 us against 17.9; 23000 rows 8.4 both).
constexpr int kChainRows = 32768;
constexpr int kRowUnroll = 2;    // rows of a thread side by side
constexpr int kRowTile = 1024;  // rows per CTA of the second launch
constexpr int kRowThreads = 256;

// Shared memory: offsets [R + 1], entry prefix [R + 1], new blocks then start
// rank [R], first new entry [R], contexts [R]; for rows handled inline the
// owners of this CTA's [share] and the parents of all [N].
inline size_t plan_smem(int R, long share, long N) {
  return sizeof(int) * (5 * (size_t)R + 2) + 2 * (size_t)((share + 1) & ~1L) + (size_t)N;
}

// The largest i in [0, n) with v[i] <= x (0 if there is none).
__device__ __forceinline__ int last_not_above(const int* v, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Exclusive prefix of v over the block's threads; *total is their sum.  s_warp:
// 32 words that no thread reads or writes from another scan without a barrier
// between.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = 0, sum = 0;
  const int nw = (int)(blockDim.x >> 5);
  {
    int w = lane < nw ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
    sum = __shfl_sync(0xffffffffu, w, 31);
  }
  *total = sum;
  return (warp ? before : 0) + x - v;
}

// The smaller of v and an int in the shared memory of any CTA of the cluster.
__device__ __forceinline__ void dsmem_min(uint32_t at, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;\n" ::"r"(at), "r"(v) : "memory");
}

// Parents as one byte: local indexes are below 128; anything else is -2.
__device__ __forceinline__ int8_t parent_byte(int p) {
  return p >= -1 && p < kMaxRows ? (int8_t)p : (int8_t)-2;
}

// Edges from node j up to the root.  Parents lie before their children, which
// the walk itself insists on: it ends whatever the parents are.
__device__ __forceinline__ int depth_of(const int8_t* par, int j) {
  int depth = 0;
  for (int p = j; p > 0; ++depth) {
    const int up = par[p];
    if (up >= p) break;
    p = up;
  }
  return depth;
}

__global__ void __launch_bounds__(1024) plan_kernel(Args a) {
  griddep_entry();
  extern __shared__ __align__(16) int s_mem[];
  const int R = a.R;
  int* s_cu = s_mem;             // [R + 1]
  int* s_e0 = s_cu + R + 1;      // [R + 1] prefix of table entries looked at
  int* s_new = s_e0 + R + 1;     // [R] new blocks, then rank of the first (-1: refused)
  int* s_first = s_new + R;      // [R] first new entry (INT_MAX: none, -1: malformed)
  int* s_ctx = s_first + R;      // [R]
  const int C = a.cluster, rank = C > 1 ? (int)cluster_rank() : 0;
  const int share = a.inline_rows ? ((a.N + C - 1) / C + 1) & ~1 : 0;
  const int row0 = rank * share, row1 = min(a.N, row0 + share);  // this CTA's rows
  uint16_t* s_own = reinterpret_cast<uint16_t*>(s_ctx + R);  // [share] the row's request
  int8_t* s_par = reinterpret_cast<int8_t*>(s_own + share);  // [N] with inline_rows
  __shared__ int s_warp[4][32], s_popped, s_fc;  // a scan's two rounds alternate
  const int tid = threadIdx.x, nt = blockDim.x;
  if (tid == 0) {
    s_popped = 0;
    s_fc = max(0, min(*a.free_count, a.capacity));
  }
  // the parents need nothing else: their loads go out first
  if (a.inline_rows && a.parent)
    for (int r = tid; r < a.N; r += nt) s_par[r] = parent_byte(a.parent[r]);

  // ---- requests: offsets, lengths, how many table entries they span ----
  int carry = 0, turn = 0;
  for (int base = 0; base < R; base += nt, turn ^= 1) {
    const int i = base + tid;
    int e = 0;
    if (i < R) {
      const long c0 = a.cu[i], c1 = a.cu[i + 1], ctx = a.ctx[i];
      const long rows = c1 - c0;
      int finding = 0;
      if (rows < 1 || rows > a.max_rows || c0 < 0 || c1 > a.N) finding = SV_DEV_BAD_WINDOW;
      else if (ctx < 0 || ctx + rows > (long)a.max_blocks * kBlockSize) finding = SV_DEV_BAD_LENGTH;
      if (finding) {
        if (rank == 0) flag(a.dev_status, finding);
      } else e = (int)((ctx + rows + kBlockSize - 1) / kBlockSize - ctx / kBlockSize);
      s_cu[i] = (int)c0;
      s_ctx[i] = (int)ctx;
      if (i == R - 1) s_cu[R] = (int)c1;
      s_new[i] = 0;
      s_first[i] = finding ? -1 : INT_MAX;
    }
    int total;
    const int excl = block_scan(e, s_warp[turn], &total);
    if (i < R) s_e0[i] = carry + excl;
    carry += total;
  }
  if (tid == 0) s_e0[R] = carry;
  const int E = carry;
  // (every CTA's state is set up before another one may write to it)
  if (C > 1) cluster_sync();
  else __syncthreads();

  // ---- entries: which are new; rows: are the parents sound ----
  for (int x = tid; x < E; x += nt) {
    const int i = last_not_above(s_e0, R, x);
    const int ctx = s_ctx[i];
    const int t0 = ctx / kBlockSize, t = t0 + (x - s_e0[i]);
    const int id = a.tables[(size_t)i * a.max_blocks + t];
    // a block that holds committed tokens has to be there already
    if (id < -1 || id >= a.num_blocks || (id == -1 && t == t0 && ctx % kBlockSize)) {
      if (rank == 0) flag(a.dev_status, SV_DEV_BAD_BLOCK_ID);
      atomicMin(&s_first[i], -1);
    } else if (id == -1) {
      atomicAdd(&s_new[i], 1);
      atomicMin(&s_first[i], t);
    }
  }
  // (kRowUnroll rows of a thread side by side: a search is a chain of
  // dependent reads)
  if ((a.parent || a.inline_rows) && R > 0) {
    const int from = a.inline_rows ? row0 : 0, to = a.inline_rows ? row1 : a.N;
    for (int r0 = from + tid; r0 < to; r0 += kRowUnroll * nt) {
      int own[kRowUnroll], p[kRowUnroll];
#pragma unroll
      for (int u = 0; u < kRowUnroll; ++u) {
        const int r = r0 + u * nt;
        p[u] = -2;
        if (r < to && a.parent) p[u] = a.inline_rows ? s_par[r] : (int)parent_byte(a.parent[r]);
        own[u] = 0;
      }
      // the largest i with s_cu[i] <= r, bit by bit from the top
      for (int step = 32 - __clz(R); step > 0; --step) {
#pragma unroll
        for (int u = 0; u < kRowUnroll; ++u) {
          const int at = own[u] + (1 << (step - 1));
          if (at < R && s_cu[at] <= r0 + u * nt) own[u] = at;
        }
      }
#pragma unroll
      for (int u = 0; u < kRowUnroll; ++u) {
        const int r = r0 + u * nt;
        if (r >= to) continue;
        const int i = own[u], j = r - s_cu[i];
        if (a.inline_rows) s_own[r - row0] = (uint16_t)i;
        if (!a.parent || j < 0 || r >= s_cu[i + 1]) continue;
        if (s_e0[i + 1] == s_e0[i]) continue;  // found malformed above
        if (j == 0 ? p[u] != -1 : (p[u] < 0 || p[u] >= j)) {
          flag(a.dev_status, SV_DEV_BAD_PARENT);
          for (int c = 0; c < C; ++c) {  // in every CTA of the cluster
            if (c == rank) atomicMin(&s_first[i], -1);
            else dsmem_min(dsmem_addr(smem_u32(&s_first[i]), (uint32_t)c), -1);
          }
        }
      }
    }
  }
  // (also: every CTA has looked at the table entries before the first writes new ones)
  if (C > 1) cluster_sync();
  else __syncthreads();

  // ---- requests: who is served ----
  const int fc = s_fc;
  carry = 0;
  turn = 0;
  for (int base = 0; base < R; base += nt, turn ^= 1) {
    const int i = base + tid;
    int n = 0, first = -1;
    if (i < R) {
      n = s_new[i];
      first = s_first[i];
      // new entries end the range: none of them may lie before one in use
      if (first >= 0 && n > 0 && first + n != s_ctx[i] / kBlockSize + s_e0[i + 1] - s_e0[i]) {
        if (rank == 0) flag(a.dev_status, SV_DEV_BAD_BLOCK_ID);
        s_first[i] = first = -1;
      }
      if (first < 0) n = 0;
    }
    int total;
    const int start = carry + block_scan(n, s_warp[2 + turn], &total);
    if (i < R) {
      const bool fits = n == 0 || start + n <= fc;
      const bool served = first >= 0 && fits;
      s_new[i] = served ? start : -1;
      if (rank == 0) {
        if (!fits) flag(a.dev_status, SV_DEV_POOL_EMPTY);
        a.taken[i] = served ? n : -1;
      }
      if (served && n > 0) atomicMax(&s_popped, start + n);
    }
    carry += total;
  }
  __syncthreads();

  // ---- entries: the new ones take their block ----
  for (int x = tid; rank == 0 && x < E; x += nt) {
    const int i = last_not_above(s_e0, R, x);
    const int t = s_ctx[i] / kBlockSize + (x - s_e0[i]);
    const int start = s_new[i], first = s_first[i];
    if (start < 0 || t < first) continue;
    const int id = a.free_list[fc - 1 - (start + t - first)];
    if (id >= 0 && id < a.num_blocks) a.tables[(size_t)i * a.max_blocks + t] = id;
    else flag(a.dev_status, SV_DEV_BAD_BLOCK_ID);  // the entry stays -1
  }
  if (rank == 0 && tid == 0 && s_popped > 0) *a.free_count = fc - s_popped;

  // ---- rows: slot and position (ids straight from the free list) ----
  if (!a.inline_rows) return;
  for (int r0 = row0 + tid; r0 < row1; r0 += kRowUnroll * nt) {
    int id[kRowUnroll], off[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {  // every row's loads
      const int r = r0 + u * nt;
      id[u] = -1;
      off[u] = 0;
      if (r >= row1 || R == 0) continue;
      const int i = s_own[r - row0], j = r - s_cu[i];
      if (j < 0 || r >= s_cu[i + 1] || s_new[i] < 0) continue;
      const int t = (s_ctx[i] + j) / kBlockSize, first = s_first[i];
      id[u] = t < first ? a.tables[(size_t)i * a.max_blocks + t]
                        : a.free_list[fc - 1 - (s_new[i] + t - first)];
      if (a.pos_offset && a.positions) off[u] = a.pos_offset[i];
    }
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const int r = r0 + u * nt;
      if (r >= row1) continue;
      int slot = -1, pos = -1;
      if (id[u] >= 0 && id[u] < a.num_blocks) {
        const int i = s_own[r - row0], j = r - s_cu[i], ctx = s_ctx[i];
        slot = id[u] * kBlockSize + (ctx + j) % kBlockSize;
        if (a.positions) pos = ctx + off[u] + (a.parent ? depth_of(s_par + s_cu[i], j) : j);
      }
      a.slots[r] = slot;
      if (a.positions) a.positions[r] = pos;
    }
  }
}

// Slots and positions of kRowTile packed rows per CTA, once the tables are
// written.  Parents reach back kMaxRows - 1 rows at most.
__global__ void __launch_bounds__(kRowThreads) rows_kernel(Args a) {
  griddep_entry();
  __shared__ int8_t s_par[kRowTile + kMaxRows];
  const int base = blockIdx.x * kRowTile;
  const int end = min(a.N, base + kRowTile);
  const int lo = max(0, base - (kMaxRows - 1));
  if (a.parent) {
    for (int r = lo + threadIdx.x; r < end; r += kRowThreads)
      s_par[r - lo] = parent_byte(a.parent[r]);
    __syncthreads();
  }
  for (int r = base + threadIdx.x; r < end; r += kRowThreads) {
    int slot = -1, pos = -1;
    if (a.R > 0) {
      const int i = find_segment(a.cu, a.R, r);
      const int c0 = a.cu[i], j = r - c0;
      if (j >= 0 && r < a.cu[i + 1] && a.taken[i] >= 0) {
        const int ctx = a.ctx[i];
        const int id = a.tables[(size_t)i * a.max_blocks + (ctx + j) / kBlockSize];
        if (id >= 0) {
          int depth = j;
          if (a.parent) {
            const int8_t* par = s_par + (c0 - lo);
            depth = depth_of(par, j);
          }
          slot = id * kBlockSize + (ctx + j) % kBlockSize;
          pos = ctx + (a.pos_offset ? a.pos_offset[i] : 0) + depth;
        }
      }
    }
    a.slots[r] = slot;
    if (a.positions) a.positions[r] = pos;
  }
}

// sv_slot_windows: a warp for each request looks at its rows' slots (four a
// lane at most).  Launch and two dependent loads: 1.2 us for one request of six
// rows, 1.3 for 256 of five, 1.8 for 8192 of five, in a graph of such calls.
constexpr int kWindowWarps = 8;
__global__ void __launch_bounds__(32 * kWindowWarps) slot_windows_kernel(sv_batch bt,
                                                                         const int32_t* slots,
                                                                         long n_slots,
                                                                         int32_t* row_end) {
  griddep_entry();
  const int i = blockIdx.x * kWindowWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= bt.n_req) return;
  bt.row_begin = bt.row_end = nullptr;
  const Window w = window_of(bt, i);
  bool there = w.ok;
  if (w.ok)
    for (int j = lane; j < w.lim; j += 32) {
      const int s = slots[w.cu + j];
      there = there && s >= 0 && s < n_slots;
    }
  there = __all_sync(0xffffffffu, there);
  if (lane == 0) row_end[i] = there ? w.lim : 0;
}

}  // namespace rsv
}  // namespace sv

using namespace sv;

extern "C" sv_status sv_reserve_kv(const sv_paged_kv* kv, const sv_batch* bt,
                                   const sv_block_pool* pool, const int32_t* pos_offset,
                                   int32_t* slots, int32_t* positions, int32_t* taken,
                                   int32_t* dev_status, void* stream) {
  SV_TRACE("sv_reserve_kv");
  if (!kv || !bt || !pool) return SV_ERR_INVALID_ARGUMENT;
  if (bt->n_req < 0 || bt->total_rows < 0 || bt->max_rows_per_req < 1)
    return SV_ERR_INVALID_ARGUMENT;
  if (kv->num_blocks < 0 || kv->max_blocks_per_req < 0 || pool->capacity < 0)
    return SV_ERR_INVALID_ARGUMENT;
  if (kv->block_size != kBlockSize || kv->num_blocks > INT_MAX / kBlockSize ||
      kv->max_blocks_per_req > INT_MAX / kBlockSize || bt->n_req > rsv::kMaxRequests ||
      bt->total_rows > 1 << 30)
    return SV_ERR_UNSUPPORTED_SHAPE;
  if (bt->parent && bt->max_rows_per_req > kMaxRows) return SV_ERR_UNSUPPORTED_SHAPE;
  // the entries of all requests are numbered in 32 bits
  const long span = min((long)kv->max_blocks_per_req, bt->max_rows_per_req / kBlockSize + 2L);
  if (bt->n_req * span > INT_MAX) return SV_ERR_UNSUPPORTED_SHAPE;
  if (bt->n_req == 0 && bt->total_rows == 0) return SV_OK;
  if (!pool->free_list || !pool->free_count || (bt->total_rows > 0 && !slots))
    return SV_ERR_INVALID_ARGUMENT;
  if (bt->n_req > 0 && (!bt->cu_rows || !kv->block_tables || !kv->cache_lens || !taken))
    return SV_ERR_INVALID_ARGUMENT;
  rsv::Args a;
  a.cu = bt->cu_rows;
  a.parent = bt->parent;
  a.ctx = kv->cache_lens;
  a.pos_offset = pos_offset;
  a.tables = kv->block_tables;
  a.free_list = pool->free_list;
  a.free_count = pool->free_count;
  a.slots = slots;
  a.positions = positions;
  a.taken = taken;
  a.dev_status = dev_status;
  a.R = bt->n_req;
  a.N = bt->total_rows;
  a.max_rows = bt->max_rows_per_req;
  a.max_blocks = kv->max_blocks_per_req;
  a.num_blocks = kv->num_blocks;
  a.capacity = pool->capacity;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.cluster = 1;
  while (a.cluster < rsv::kMaxCluster && a.N > (long)a.cluster * rsv::kClusterRows) a.cluster *= 2;
  size_t smem = rsv::plan_smem(a.R, (a.N + a.cluster - 1) / a.cluster, a.N);
  a.inline_rows = smem <= rsv::kMaxSmem && (a.parent || a.N <= rsv::kChainRows) ? 1 : 0;
  if (!a.inline_rows) {
    a.cluster = 1;
    smem = rsv::plan_smem(a.R, 0, 0);
  }
  if (smem > rsv::kFreeSmem) {
    static PerDevice smem_set;
    if (smem_limit_once(smem_set, rsv::plan_kernel, rsv::kMaxSmem) != cudaSuccess)
      return SV_ERR_CUDA;
  }
  // one thread per row or request, up to a full CTA: few warps meet a
  // barrier sooner
  const int want = max(a.R, min(a.N, 1024));
  const unsigned threads = (unsigned)max(128, min(1024, (want + 31) / 32 * 32));
  const cudaError_t e =
      a.cluster > 1 ? sv::launch_cluster(rsv::plan_kernel, (unsigned)a.cluster, threads, smem, s, a.cluster, a)
                    : sv::launch(rsv::plan_kernel, 1, threads, smem, s, a);
  if (e != cudaSuccess) return SV_ERR_CUDA;
  if (!a.inline_rows) {
    const unsigned grid = (unsigned)(((long)a.N + rsv::kRowTile - 1) / rsv::kRowTile);
    if (sv::launch(rsv::rows_kernel, grid, rsv::kRowThreads, 0, s, a) != cudaSuccess)
      return SV_ERR_CUDA;
  }
  return SV_OK;
}

extern "C" sv_status sv_slot_windows(const sv_paged_kv* kv, const sv_batch* bt, const int32_t* slots,
                                     int32_t* row_end, void* stream) {
  SV_TRACE("sv_slot_windows");
  if (!kv || !bt) return SV_ERR_INVALID_ARGUMENT;
  if (bt->n_req < 0 || bt->total_rows < 0 || bt->max_rows_per_req < 1 || kv->num_blocks < 0)
    return SV_ERR_INVALID_ARGUMENT;
  if (kv->block_size != kBlockSize || bt->max_rows_per_req > kMaxRows)
    return SV_ERR_UNSUPPORTED_SHAPE;
  if (bt->n_req == 0) return SV_OK;
  if (!bt->cu_rows || !row_end || (bt->total_rows > 0 && !slots)) return SV_ERR_INVALID_ARGUMENT;
  const unsigned grid = ((unsigned)bt->n_req + rsv::kWindowWarps - 1) / rsv::kWindowWarps;
  if (sv::launch(rsv::slot_windows_kernel, grid, 32 * rsv::kWindowWarps, 0,
                 static_cast<cudaStream_t>(stream), *bt, slots, (long)kv->num_blocks * kBlockSize,
                 row_end) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}
