// pages.cu — which pages of a long cache a draft row attends.
//
//   sv_bound_pages   least and greatest key element of each complete page;
//   sv_score_pages   an upper bound of the products of a row's queries with a
//                    page's keys;
//   sv_select_pages  the pages of greatest score.
//
// Source: [SSD] section details (PagedAttention: the page is the unit of the
// cache); the selection itself is on none of the pages and fixed in the header.

#include <algorithm>

#include "sv_internal.cuh"

namespace sv {
namespace pg {

constexpr int kMaxRequests = 8192;  // offsets of a call's pages in shared memory

// Exclusive prefix sums of count(i), i < n, into off[0 .. n] (shared memory),
// by all threads of the block (a multiple of 32, at most 1024).
template <class F>
__device__ __forceinline__ void block_offsets(int* off, int n, F&& count) {
  __shared__ int s_warp[32];
  __shared__ int s_carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  if (tid == 0) s_carry = 0;
  for (int base = 0; base < n; base += blockDim.x) {
    const int i = base + tid;
    const int v = i < n ? count(i) : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int before = s_carry;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
    if (i < n) off[i] = before + x - v;
    __syncthreads();
    if (tid == blockDim.x - 1) s_carry = before + x;
    (void)nw;
    __syncthreads();
  }
  if (tid == 0) off[n] = s_carry;
  __syncthreads();
}

// ---------------------------------------------------------------- bounds --

struct BoundArgs {
  const __nv_bfloat16* k;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* from;
  __nv_bfloat16* bounds;
  int32_t* dev_status;
  int R, num_blocks, Hkv, max_blocks;
};

constexpr int kBoundThreads = 256;

// One warp takes one (page, KV head): 16 rows of D keys, 16 bytes a lane and
// load, every load of the page in flight at once; lane l keeps column chunk
// l % (D / 8) of the rows l / (D / 8), l / (D / 8) + step, ... and the lanes of
// a column meet by shuffles.  min and max of bf16 are exact.
template <int D>
__global__ void __launch_bounds__(kBoundThreads) bound_kernel(BoundArgs a) {
  griddep_entry();
  extern __shared__ int s_off[];
  block_offsets(s_off, a.R, [&](int i) {
    const int len = a.lens[i], from = a.from ? a.from[i] : 0;
    if (len < 0 || from < 0 || len > (long)a.max_blocks * kBlockSize) {
      if (blockIdx.x == 0) flag(a.dev_status, SV_DEV_BAD_LENGTH);
      return 0;
    }
    return max(0, len / kBlockSize - from / kBlockSize);
  });
  const int total = s_off[a.R];
  constexpr int kCols = D / 8;           // 16-byte chunks of a row
  constexpr int kRowsAtOnce = 32 / kCols;
  constexpr int kLoads = kBlockSize / kRowsAtOnce;
  const int lane = threadIdx.x & 31;
  const long nwarp = (long)gridDim.x * (kBoundThreads / 32);
  for (long x = (long)blockIdx.x * (kBoundThreads / 32) + (threadIdx.x >> 5);
       x < (long)total * a.Hkv; x += nwarp) {
    const int page = (int)(x / a.Hkv), g = (int)(x % a.Hkv);
    int lo = 0, hi = a.R - 1;  // the request whose range holds the page
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_off[mid] <= page) lo = mid; else hi = mid - 1;
    }
    const int t = page - s_off[lo] + (a.from ? a.from[lo] / kBlockSize : 0);
    const int b = __ldg(a.tables + (size_t)lo * a.max_blocks + t);
    if (b < 0 || b >= a.num_blocks) {
      if (lane == 0) flag(a.dev_status, SV_DEV_BAD_BLOCK_ID);
      continue;
    }
    const size_t row = ((size_t)b * a.Hkv + g) * kBlockSize;
    const uint4* src = reinterpret_cast<const uint4*>(a.k + row * D) + lane;
    uint4 v[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) v[k] = __ldg(src + k * 32);
    __nv_bfloat162 mn[4], mx[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) mn[e] = mx[e] = reinterpret_cast<__nv_bfloat162*>(&v[0])[e];
#pragma unroll
    for (int k = 1; k < kLoads; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 y = reinterpret_cast<__nv_bfloat162*>(&v[k])[e];
        mn[e] = __hmin2(mn[e], y);
        mx[e] = __hmax2(mx[e], y);
      }
#pragma unroll
    for (int o = kCols; o < 32; o <<= 1)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        mn[e] = __hmin2(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], o));
        mx[e] = __hmax2(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
      }
    // the first kCols lanes write the least, the next the greatest elements
    if (lane < 2 * kCols) {
      const bool up = lane >= kCols;
      uint4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) reinterpret_cast<__nv_bfloat162*>(&w)[e] = up ? mx[e] : mn[e];
      reinterpret_cast<uint4*>(a.bounds + ((size_t)b * a.Hkv + g) * 2 * D)[lane] = w;
    }
  }
}

// ----------------------------------------------------------------- score --

struct ScoreArgs {
  sv_batch bt;
  const __nv_bfloat16* q;
  const __nv_bfloat16* bounds;
  const int32_t* tables;
  const int32_t* lens;
  float* scores;
  int32_t* dev_status;
  int num_blocks, Hkv, max_blocks, Hq, group, max_pages;
  int per;   // pages a CTA takes
  int g2;    // the group rounded up to a power of two
};

constexpr int kScoreThreads = 128;
constexpr int kScoreTiles = 8;  // 16-row tiles of a CTA
constexpr int kMaxPer = 256;

// For a row's query head h and page t: sum_d max(q lo, q hi) = min(q, 0) . lo +
// max(q, 0) . hi, a product of [q-, q+] with the 2 D contiguous elements [lo,
// hi] of the page: exact bf16 factors, fp32 sums, on mma.sync m16n8k16 (16
// virtual rows x 8 pages x 16 elements).  A 16-row tile holds 16 / g2 rows, its
// g2 >= group slots the group's heads (some twice: the maximum over the slots
// does not see that).  The k order of a product is free, so a lane takes 16
// consecutive bytes of a page's bounds as the operands of two steps: the bounds
// go from global memory to registers without a stop, 16 pages a warp at once.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(ScoreArgs a) {
  griddep_entry();
  constexpr int kSteps = 2 * D / 16;
  constexpr int kPairs = kSteps / 2;  // 16-byte chunks a lane holds of a page
  extern __shared__ __align__(16) uint4 s_q[];  // [tile][step][lane]
  __shared__ int s_tbl[kMaxPer];
  const int i = blockIdx.z / a.Hkv, g = blockIdx.z % a.Hkv;
  const Window w = window_of(a.bt, i);
  const int ctx = a.lens[i];
  const bool first = blockIdx.x == 0 && blockIdx.y == 0 && g == 0 && threadIdx.x == 0;
  if (!w.ok) {
    if (first) flag(a.dev_status, SV_DEV_BAD_WINDOW);
    return;
  }
  const int n = ctx / kBlockSize;
  if (ctx < 0 || ctx > (long)a.max_blocks * kBlockSize || n > a.max_pages) {
    if (first) flag(a.dev_status, SV_DEV_BAD_LENGTH);
    return;
  }
  const int per_tile = 16 / a.g2;  // rows of a tile
  const int r0 = w.b + blockIdx.y * kScoreTiles * per_tile;
  const int nr = min(w.e - r0, kScoreTiles * per_tile);
  const int p0 = blockIdx.x * a.per, p1 = min(n, p0 + a.per);
  if (nr <= 0 || p0 >= p1) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const int tiles = (nr + per_tile - 1) / per_tile;
  for (int p = p0 + tid; p < p1; p += kScoreThreads) {
    int b = __ldg(a.tables + (size_t)i * a.max_blocks + p);
    if (b < 0 || b >= a.num_blocks) {
      if (blockIdx.y == 0 && g == 0) flag(a.dev_status, SV_DEV_BAD_BLOCK_ID);
      b = -1;
    }
    s_tbl[p - p0] = b;
  }
  // [q-, q+] of the tiles' rows in the order the products take them
  for (int x = tid; x < tiles * kPairs * 32; x += kScoreThreads) {
    const int l = x & 31, c = (x >> 5) % kPairs, mt = (x >> 5) / kPairs;
    const int chunk = c * 4 + (l & 3);
    uint4 v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int slot = (l >> 2) + 8 * k;
      const int r = min(mt * per_tile + slot / a.g2, nr - 1), h = (slot % a.g2) % a.group;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + ((size_t)(w.cu + r0 + r) * a.Hq + g * a.group + h) * D);
      v[k] = __ldg(src + chunk % (D / 8));
      const __nv_bfloat162 z = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        __nv_bfloat162& y = reinterpret_cast<__nv_bfloat162*>(&v[k])[e];
        y = chunk < D / 8 ? __hmin2(y, z) : __hmax2(y, z);
      }
    }
    s_q[(mt * kSteps + 2 * c) * 32 + l] = make_uint4(v[0].x, v[1].x, v[0].y, v[1].y);
    s_q[(mt * kSteps + 2 * c + 1) * 32 + l] = make_uint4(v[0].z, v[1].z, v[0].w, v[1].w);
  }
  __syncthreads();
  for (int p = p0 + warp * 16; p < p1; p += (kScoreThreads / 32) * 16) {
    uint4 bd[2][kPairs];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int page = p + nt * 8 + gq;
      const int b = page < p1 ? s_tbl[page - p0] : -1;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.bounds + ((size_t)max(b, 0) * a.Hkv + g) * 2 * D) + tq;
#pragma unroll
      for (int c = 0; c < kPairs; ++c) bd[nt][c] = b >= 0 ? __ldg(src + c * 4) : make_uint4(0, 0, 0, 0);
    }
    for (int mt = 0; mt < tiles; ++mt) {
      float acc[2][4] = {};
#pragma unroll
      for (int c = 0; c < kPairs; ++c) {
        const uint4 x = s_q[(mt * kSteps + 2 * c) * 32 + lane];
        const uint4 y = s_q[(mt * kSteps + 2 * c + 1) * 32 + lane];
        const uint32_t ax[4] = {x.x, x.y, x.z, x.w}, ay[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          mma16816(acc[nt], ax, bd[nt][c].x, bd[nt][c].y);
          mma16816(acc[nt], ay, bd[nt][c].z, bd[nt][c].w);
        }
      }
      // the maximum over each row's g2 slots: lanes gq and gq + 8
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        if (a.g2 == 16)
#pragma unroll
          for (int e = 0; e < 2; ++e) acc[nt][e] = acc[nt][e + 2] = fmaxf(acc[nt][e], acc[nt][e + 2]);
        for (int o = 1; o < a.g2 && o < 8; o <<= 1)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[nt][e] = fmaxf(acc[nt][e], __shfl_xor_sync(0xffffffffu, acc[nt][e], 4 * o));
        if (gq % min(a.g2, 8) != 0) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int slot = gq + (e >> 1) * 8;
          const int r = mt * per_tile + slot / a.g2, page = p + nt * 8 + 2 * tq + (e & 1);
          if (slot % a.g2 == 0 && r < nr && page < p1)
            a.scores[((size_t)(w.cu + r0 + r) * a.Hkv + g) * a.max_pages + page] = acc[nt][e];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- select --

struct SelectArgs {
  sv_batch bt;
  const float* scores;
  const int32_t* lens;
  int32_t* pages;
  int32_t* dev_status;
  int Hkv, max_blocks, max_pages, n_first, n_last, n_keep;
};

constexpr int kSelectThreads = 256;

// Whole numbers in the order of the scores: NaN below everything, -0 = +0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA a (row, KV head).  The n_keep-th greatest key is found digit by digit
// (8 bits, from the highest) in counts of the keys that agree with the digits
// found before; then the pages above it and the first of those equal to it are
// written in order.
__global__ void __launch_bounds__(kSelectThreads) select_kernel(SelectArgs a) {
  griddep_entry();
  extern __shared__ uint32_t s_key[];
  __shared__ int s_hist[256];
  __shared__ int s_warp[2][kSelectThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int r = blockIdx.x, g = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (r >= a.bt.cu_rows[a.bt.n_req]) return;
  const int i = find_segment(a.bt.cu_rows, a.bt.n_req, r);
  const Window w = window_of(a.bt, i);
  const int ctx = a.lens[i], n = ctx / kBlockSize;
  if (!w.ok) {
    if (tid == 0 && g == 0) flag(a.dev_status, SV_DEV_BAD_WINDOW);
    return;
  }
  if (ctx < 0 || ctx > (long)a.max_blocks * kBlockSize || n > a.max_pages) {
    if (tid == 0 && g == 0) flag(a.dev_status, SV_DEV_BAD_LENGTH);
    return;
  }
  if (r < w.cu + w.b || r >= w.cu + w.e) return;
  int32_t* out = a.pages + ((size_t)r * a.Hkv + g) * a.n_keep;
  if (n <= a.n_keep) {
    for (int t = tid; t < a.n_keep; t += kSelectThreads) out[t] = t < n ? t : -1;
    return;
  }
  const float* s = a.scores + ((size_t)r * a.Hkv + g) * a.max_pages;
  for (int t = tid; t < n; t += kSelectThreads)
    s_key[t] = (t < a.n_first || t >= n - a.n_last) ? 0xffffffffu : score_key(__ldg(s + t));
  if (tid == 0) {
    s_prefix = 0u;
    s_need = a.n_keep;
  }
  for (int shift = 24; shift >= 0; shift -= 8) {
    s_hist[tid] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    const uint32_t prefix = s_prefix;
    for (int t = tid; t < n; t += kSelectThreads) {
      const uint32_t k = s_key[t];
      if ((k & above) == prefix) atomicAdd(&s_hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // keys in the digits above lane's eight, from the highest digit down
      int c[8], sum = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += c[k] = s_hist[255 - (lane * 8 + k)];
      int x = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const int need = s_need;
      __syncwarp();
      int before = x - sum;
      if (before < need && x >= need) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (before < need && before + c[k] >= need) {
            s_prefix = prefix | ((uint32_t)(255 - (lane * 8 + k)) << shift);
            s_need = need - before;
          }
          before += c[k];
        }
      }
    }
    __syncthreads();
  }
  const uint32_t kth = s_prefix;
  const int need = s_need;  // of the pages whose key is kth, the first so many
  int above = 0, equal = 0;  // written so far
  for (int base = 0; base < n; base += kSelectThreads) {
    const int t = base + tid;
    const uint32_t k = t < n ? s_key[t] : 0u;
    const bool up = t < n && k > kth, eq = t < n && k == kth;
    const unsigned bu = __ballot_sync(0xffffffffu, up), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      s_warp[0][warp] = __popc(bu);
      s_warp[1][warp] = __popc(be);
    }
    __syncthreads();
    int u = above, e = equal;
    for (int x = 0; x < kSelectThreads / 32; ++x) {
      if (x < warp) { u += s_warp[0][x]; e += s_warp[1][x]; }
      above += s_warp[0][x];
      equal += s_warp[1][x];
    }
    const unsigned below = (1u << lane) - 1u;
    u += __popc(bu & below);
    e += __popc(be & below);
    if (up || (eq && e < need)) out[u + min(e, need)] = t;
    __syncthreads();
  }
}

static sv_status check(const sv_paged_kv* kv, const sv_batch* bt) {
  if (!kv) return SV_ERR_INVALID_ARGUMENT;
  if (kv->block_size != kBlockSize) return SV_ERR_UNSUPPORTED_SHAPE;
  if (kv->n_kv_heads < 1 || kv->num_blocks < 0 || kv->max_blocks_per_req < 0)
    return SV_ERR_INVALID_ARGUMENT;
  if (!bt) return SV_OK;
  if (bt->n_req < 0 || bt->total_rows < 0 || bt->max_rows_per_req < 1) return SV_ERR_INVALID_ARGUMENT;
  if (bt->max_rows_per_req > kMaxRows) return SV_ERR_UNSUPPORTED_SHAPE;
  if (bt->n_req > 0 && !bt->cu_rows) return SV_ERR_INVALID_ARGUMENT;
  return SV_OK;
}

}  // namespace pg
}  // namespace sv

using namespace sv;

extern "C" sv_status sv_bound_pages(const sv_paged_kv* kv, int32_t n_req, const int32_t* from_len,
                                    void* bounds, int32_t* dev_status, void* stream) {
  SV_TRACE("sv_bound_pages");
  const sv_status st = pg::check(kv, nullptr);
  if (st != SV_OK) return st;
  if (kv->head_dim != 64 && kv->head_dim != 128) return SV_ERR_UNSUPPORTED_SHAPE;
  if (n_req < 0) return SV_ERR_INVALID_ARGUMENT;
  if (n_req > pg::kMaxRequests) return SV_ERR_UNSUPPORTED_SHAPE;
  if (n_req == 0) return SV_OK;
  if (!kv->k_cache || !kv->block_tables || !kv->cache_lens || !bounds) return SV_ERR_INVALID_ARGUMENT;
  if (((uintptr_t)kv->k_cache | (uintptr_t)bounds) & 15) return SV_ERR_INVALID_ARGUMENT;
  // the pages of a call are counted in 32 bits
  if ((long)n_req * kv->max_blocks_per_req >= (1L << 31)) return SV_ERR_UNSUPPORTED_SHAPE;
  pg::BoundArgs a;
  a.k = static_cast<const __nv_bfloat16*>(kv->k_cache);
  a.tables = kv->block_tables;
  a.lens = kv->cache_lens;
  a.from = from_len;
  a.bounds = static_cast<__nv_bfloat16*>(bounds);
  a.dev_status = dev_status;
  a.R = n_req;
  a.num_blocks = kv->num_blocks;
  a.Hkv = kv->n_kv_heads;
  a.max_blocks = kv->max_blocks_per_req;
  const int nsm = num_sms();
  if (nsm < 1) return SV_ERR_CUDA;
  const long most = ((long)n_req * kv->max_blocks_per_req * kv->n_kv_heads + 7) / 8;
  const int grid = (int)std::max(1L, std::min(4L * nsm, most));
  const size_t smem = sizeof(int) * (size_t)(n_req + 1);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      kv->head_dim == 128 ? sv::launch(pg::bound_kernel<128>, grid, pg::kBoundThreads, smem, s, a)
                          : sv::launch(pg::bound_kernel<64>, grid, pg::kBoundThreads, smem, s, a);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

extern "C" sv_status sv_score_pages(const sv_paged_kv* kv, const sv_batch* bt, const void* q,
                                    int32_t n_q_heads, const void* bounds, float* scores,
                                    int32_t max_pages, int32_t* dev_status, void* stream) {
  SV_TRACE("sv_score_pages");
  if (!bt) return SV_ERR_INVALID_ARGUMENT;
  const sv_status st = pg::check(kv, bt);
  if (st != SV_OK) return st;
  if (kv->head_dim != 64 && kv->head_dim != 128) return SV_ERR_UNSUPPORTED_SHAPE;
  if (n_q_heads < 1 || n_q_heads % kv->n_kv_heads != 0 || max_pages < 0) return SV_ERR_INVALID_ARGUMENT;
  if (n_q_heads / kv->n_kv_heads > 16) return SV_ERR_UNSUPPORTED_SHAPE;
  if (bt->n_req == 0 || bt->total_rows == 0 || max_pages == 0) return SV_OK;
  if (!q || !bounds || !scores || !kv->block_tables || !kv->cache_lens) return SV_ERR_INVALID_ARGUMENT;
  if (((uintptr_t)q | (uintptr_t)bounds) & 15) return SV_ERR_INVALID_ARGUMENT;
  if ((uintptr_t)scores & 3) return SV_ERR_INVALID_ARGUMENT;
  if ((long)bt->n_req * kv->n_kv_heads > 65535) return SV_ERR_UNSUPPORTED_SHAPE;
  pg::ScoreArgs a;
  a.bt = *bt;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.bounds = static_cast<const __nv_bfloat16*>(bounds);
  a.tables = kv->block_tables;
  a.lens = kv->cache_lens;
  a.scores = scores;
  a.dev_status = dev_status;
  a.num_blocks = kv->num_blocks;
  a.Hkv = kv->n_kv_heads;
  a.max_blocks = kv->max_blocks_per_req;
  a.Hq = n_q_heads;
  a.group = n_q_heads / kv->n_kv_heads;
  a.max_pages = max_pages;
  a.g2 = 1;
  while (a.g2 < a.group) a.g2 *= 2;
  const int nsm = num_sms();
  if (nsm < 1) return SV_ERR_CUDA;
  const long units = (long)bt->n_req * kv->n_kv_heads * max_pages;
  a.per = units <= 64L * 8 * nsm ? 64 : pg::kMaxPer;
  const int per_block = pg::kScoreTiles * (16 / a.g2);
  const int most_rows = std::min(bt->max_rows_per_req, bt->total_rows);
  const dim3 grid((max_pages + a.per - 1) / a.per, (most_rows + per_block - 1) / per_block,
                  bt->n_req * kv->n_kv_heads);
  const int tiles = std::min(pg::kScoreTiles, (most_rows + 16 / a.g2 - 1) / (16 / a.g2));
  const size_t smem = (size_t)tiles * (2 * kv->head_dim / 16) * 32 * 16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  static PerDevice set128, set64;
  if (smem_limit_once(set128, pg::score_kernel<128>, 65536) != cudaSuccess ||
      smem_limit_once(set64, pg::score_kernel<64>, 65536) != cudaSuccess)
    return SV_ERR_CUDA;
  const cudaError_t e =
      kv->head_dim == 128 ? sv::launch(pg::score_kernel<128>, grid, pg::kScoreThreads, smem, s, a)
                          : sv::launch(pg::score_kernel<64>, grid, pg::kScoreThreads, smem, s, a);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

extern "C" sv_status sv_select_pages(const sv_paged_kv* kv, const sv_batch* bt, const float* scores,
                                     int32_t max_pages, int32_t n_first, int32_t n_last,
                                     int32_t n_keep, int32_t* pages, int32_t* dev_status,
                                     void* stream) {
  SV_TRACE("sv_select_pages");
  if (!bt) return SV_ERR_INVALID_ARGUMENT;
  const sv_status st = pg::check(kv, bt);
  if (st != SV_OK) return st;
  if (max_pages < 0 || n_first < 0 || n_last < 0 || n_keep < 1 || (long)n_first + n_last > n_keep)
    return SV_ERR_INVALID_ARGUMENT;
  if (n_keep > 1024 || max_pages > 49152 || kv->n_kv_heads > 65535) return SV_ERR_UNSUPPORTED_SHAPE;
  if (bt->n_req == 0 || bt->total_rows == 0) return SV_OK;
  if ((max_pages > 0 && !scores) || !pages || !kv->cache_lens) return SV_ERR_INVALID_ARGUMENT;
  pg::SelectArgs a;
  a.bt = *bt;
  a.scores = scores;
  a.lens = kv->cache_lens;
  a.pages = pages;
  a.dev_status = dev_status;
  a.Hkv = kv->n_kv_heads;
  a.max_blocks = kv->max_blocks_per_req;
  a.max_pages = max_pages;
  a.n_first = n_first;
  a.n_last = n_last;
  a.n_keep = n_keep;
  static PerDevice set;
  if (smem_limit_once(set, pg::select_kernel, 49152 * 4) != cudaSuccess) return SV_ERR_CUDA;
  const cudaError_t e =
      sv::launch(pg::select_kernel, dim3(bt->total_rows, kv->n_kv_heads), pg::kSelectThreads,
                 (size_t)max_pages * 4, static_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
