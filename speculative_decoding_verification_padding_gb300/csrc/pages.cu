// pages.cu — which pages of a long cache a draft row attends.
//
//   sv_bound_pages   least and greatest key element of each complete page;
//   sv_score_pages   an upper bound of the products of a row's queries with a
//                    page's keys;
//   sv_select_pages  the pages of greatest score.
//
// Source: [SSD] section details (PagedAttention: the page is the unit of the
// cache).  The selection itself is on none of the pages and fixed in the header; that a
// page's products are bounded by its keys' least and greatest elements is the published
// method of Tang et al., "Quest: Query-Aware Sparsity for Efficient Long-Context LLM
// Inference" (ICML 2024).

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
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
// a column meet by shuffles.  min and max of bf16 are exact.  Bound by HBM: 24 prompts
// of 500 .. 40000 tokens, 8 heads of 128, take 80 us, 6.2 TB/s.
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
constexpr int kScoreTiles = 8;  // tiles of 16 virtual rows of a CTA
constexpr int kMaxPer = 512;

// The greater of two, NaN where one is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}

// MT tiles of 16 virtual rows (from row r0 on) by a warp's 8 E pages from `page`
// on: E MT chains of products side by side.  A thread has of each tile the slots
// gq and gq + 8 by the pages 2 tq, 2 tq + 1 of each eight, taken in pairs of eights:
// v[eight * 4 + half * 2 + odd].  The maximum over a row's G2 slots is one over lanes: at each step a
// lane keeps half of its values and hands the other half over, so that in the
// end every value is in one lane only.  `worst` becomes NaN where a sum is.
template <int D, int G2, int MT, int E>
__device__ __forceinline__ void score_tiles(const uint4 (&bd)[E][2 * D / 32], const uint4* sq,
                                            int r0, int nr, int page, int p1, int lane,
                                            unsigned known, float* out, size_t row_step, float& worst) {
  constexpr int kPairs = 2 * D / 32;
  const int gq = lane >> 2, tq = lane & 3;
  float acc[MT][E][4] = {};
#pragma unroll
  for (int c = 0; c < kPairs; ++c) {
#pragma unroll
    for (int k = 0; k < MT; ++k) {
      const uint4 x = sq[((k * kPairs + c) * 2) * 32], y = sq[((k * kPairs + c) * 2 + 1) * 32];
      const uint32_t ax[4] = {x.x, x.y, x.z, x.w}, ay[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int nt = 0; nt < E; ++nt) mma16816(acc[k][nt], ax, bd[nt][c].x, bd[nt][c].y);
#pragma unroll
      for (int nt = 0; nt < E; ++nt) mma16816(acc[k][nt], ay, bd[nt][c].z, bd[nt][c].w);
    }
  }
  const bool b0 = gq & 1, b1 = gq & 2, b2 = gq & 4;
  auto halve = [&](float lo, float hi, bool up, int o) {
    return max_nan(up ? hi : lo, __shfl_xor_sync(0xffffffffu, up ? lo : hi, o));
  };
  auto put_at = [&](int r, int at, float v) {
    worst = max_nan(worst, v);
    if (r < nr && page + at < p1) out[r * row_step + page + at] = (known >> at) & 1u ? v : 0.f;
  };
#pragma unroll
  for (int ke = 0; ke < MT * E / 2; ++ke) {
    const int k = ke / (E / 2), pr = ke % (E / 2), row = r0 + k * (16 / G2);
    auto put = [&](int r, int at, float v) { put_at(r, 16 * pr + at, v); };
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = acc[k][2 * pr + (j >> 2)][j & 3];
    if (G2 == 16) {
#pragma unroll
      for (int j = 0; j < 2; ++j) v[j] = halve(max_nan(v[j], v[j + 2]), max_nan(v[4 + j], v[6 + j]), b0, 4);
      v[0] = halve(v[0], v[1], b1, 8);
      v[0] = max_nan(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
      if (!b2) put(row, b0 * 8 + 2 * tq + b1, v[0]);
    } else if (G2 == 1) {
#pragma unroll
      for (int j = 0; j < 8; ++j) put(row + gq + (j & 2) * 4, (j & 4) * 2 + 2 * tq + (j & 1), v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = halve(v[j], v[j + 4], b0, 4);  // v: half * 2 + odd
      if (G2 == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) put(row + (gq >> 1) + (j & 2) * 2, b0 * 8 + 2 * tq + (j & 1), v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) v[j] = halve(v[j], v[j + 2], b1, 8);
        if (G2 == 4) {
#pragma unroll
          for (int j = 0; j < 2; ++j) put(row + (gq >> 2) + 2 * b1, b0 * 8 + 2 * tq + j, v[j]);
        } else {
          put(row + b1, b0 * 8 + 2 * tq + b2, halve(v[0], v[1], b2, 16));
        }
      }
    }
  }
}

// The scores of a CTA that are NaN once more, term by term: where a bound is infinite
// [q-, q+] . [lo, hi] has products 0 x infinity.  A head that still has no number counts
// for nothing.
template <int D>
__device__ __noinline__ void score_again(const ScoreArgs& a, const int* s_tbl) {
  const int i = blockIdx.z / a.Hkv, g = blockIdx.z % a.Hkv;
  const Window w = window_of(a.bt, i);
  const int rows = kScoreTiles * (16 / a.g2), r0 = w.b + blockIdx.y * rows, nr = min(w.e - r0, rows);
  const int p0 = blockIdx.x * a.per, p1 = min(a.lens[i] / kBlockSize, p0 + a.per);
  for (int p = p0 + (int)threadIdx.x; p < p1; p += kScoreThreads) {
    const int b = s_tbl[p - p0];
    if (b < 0) continue;
    const __nv_bfloat16* lo = a.bounds + ((size_t)b * a.Hkv + g) * 2 * D;
    for (int r = w.cu + r0; r < w.cu + r0 + nr; ++r) {
      float& out = a.scores[((size_t)r * a.Hkv + g) * a.max_pages + p];
      float best = out;
      if (best == best) continue;
      for (int h = 0; h < a.group; ++h) {
        const __nv_bfloat16* q = a.q + ((size_t)r * a.Hq + g * a.group + h) * D;
        float sum = 0.f;
        for (int d = 0; d < D; ++d) {
          const float x = __bfloat162float(q[d]);
          if (x > 0.f) sum += x * __bfloat162float(lo[D + d]);
          else if (x < 0.f) sum += x * __bfloat162float(lo[d]);
        }
        best = fmaxf(best, sum);
      }
      out = best;
    }
  }
}

// For a row's query head h and page t: sum_d max(q lo, q hi) = min(q, 0) . lo +
// max(q, 0) . hi, a product of [q-, q+] with the 2 D contiguous elements [lo,
// hi] of the page: exact bf16 factors, fp32 sums, on mma.sync m16n8k16 (16
// virtual rows x 8 pages x 16 elements).  Virtual row v is row v / G2, head slot
// v % G2 of it, the group's heads in the first slots and some again in the rest
// (the maximum over the slots does not see that).  Where a bound is infinite 0 x infinity
// makes the sum NaN: a CTA that meets NaN takes those again, term by term (noticing it
// costs 1 %; with the second form inside the loop, or what it saw kept in a register,
// 6 to 15 %).  The k order of a product is
// free, so a lane takes 16 consecutive bytes of a page's bounds as the operands
// of two steps: the bounds go from global memory to registers without a stop, 8 E
// pages a warp at once.  q is read again from shared memory for every 8 E pages (264
// rows of 40 heads by 48 contexts of 2000 .. 60000 tokens: E = 1 73 us, 2 54, 4 51, 4.3
// TB/s; small calls take E = 2, whose pages are spread over more warps).  No unit is
// full there: HBM 57 %, in an SM's active cycles the load and store path 61 %, half of
// it shared memory, the products 41 %; 12 warps an SM do not hide the loads (4.5 of 11
// cycles an instruction), and the SMs are active 81 % of the time.
template <int D, int G2, int E>
__global__ void __launch_bounds__(kScoreThreads, E == 4 ? 3 : 4) score_kernel(ScoreArgs a) {
  griddep_entry();
  constexpr int kPairs = 2 * D / 32;  // 16-byte chunks a lane holds of a page, two steps each
  constexpr int kTileRows = 16 / G2;
  extern __shared__ __align__(16) uint4 s_q[];  // [tile][step][lane]
  __shared__ int s_tbl[kMaxPer];
  __shared__ int s_odd[kScoreThreads / 32];
  if (threadIdx.x < kScoreThreads / 32) s_odd[threadIdx.x] = 0;
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
  const int r0 = w.b + blockIdx.y * kScoreTiles * kTileRows;
  const int nr = min(w.e - r0, kScoreTiles * kTileRows);
  const int p0 = blockIdx.x * a.per, p1 = min(n, p0 + a.per);
  if (nr <= 0 || p0 >= p1) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const int tiles = (nr + kTileRows - 1) / kTileRows;
  for (int p = p0 + tid; p < p1; p += kScoreThreads) {
    int b = __ldg(a.tables + (size_t)i * a.max_blocks + p);
    if (b < 0 || b >= a.num_blocks) {
      if (blockIdx.y == 0 && g == 0) flag(a.dev_status, SV_DEV_BAD_BLOCK_ID);
      b = -1;
    }
    s_tbl[p - p0] = b;
  }
  // [q-, q+] of the tiles' rows in the order the products take them: the lower
  // half of the steps is q-, the upper q+, of the same chunks of q
  for (int x = tid; x < tiles * (kPairs / 2) * 32; x += kScoreThreads) {
    const int l = x & 31, c = (x >> 5) % (kPairs / 2), mt = (x >> 5) / (kPairs / 2);
    uint4 dn[2], up[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int slot = (l >> 2) + 8 * k, s = slot % G2;
      const int r = min(mt * kTileRows + slot / G2, nr - 1), h = s < a.group ? s : s - a.group;
      up[k] = __ldg(reinterpret_cast<const uint4*>(
                  a.q + ((size_t)(w.cu + r0 + r) * a.Hq + g * a.group + h) * D) + c * 4 + (l & 3));
      const __nv_bfloat162 z = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        __nv_bfloat162& y = reinterpret_cast<__nv_bfloat162*>(&up[k])[e];
        reinterpret_cast<__nv_bfloat162*>(&dn[k])[e] = __hmin2(y, z);
        y = __hmax2(y, z);
      }
    }
    uint4* to = s_q + (mt * kPairs + c) * 64 + l;
    to[0] = make_uint4(dn[0].x, dn[1].x, dn[0].y, dn[1].y);
    to[32] = make_uint4(dn[0].z, dn[1].z, dn[0].w, dn[1].w);
    to[kPairs * 32] = make_uint4(up[0].x, up[1].x, up[0].y, up[1].y);
    to[kPairs * 32 + 32] = make_uint4(up[0].z, up[1].z, up[0].w, up[1].w);
  }
  __syncthreads();
  float* out = a.scores + ((size_t)(w.cu + r0) * a.Hkv + g) * a.max_pages;
  const size_t row_step = (size_t)a.Hkv * a.max_pages;
  constexpr int kPages = 8 * E;  // of a warp at once
  for (int p = p0 + warp * kPages; p < p1; p += (kScoreThreads / 32) * kPages) {
    uint4 bd[E][kPairs];  // pages p + gq, p + gq + 8, ...
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const int b = s_tbl[min(p + k * 8 + gq, p1 - 1) - p0];
      const uint4* src = reinterpret_cast<const uint4*>(
          a.bounds + ((size_t)max(b, 0) * a.Hkv + g) * 2 * D) + tq;
#pragma unroll
      for (int c = 0; c < kPairs; ++c) bd[k][c] = __ldg(src + c * 4);
    }
    // pages whose block is in the cache
    const unsigned known = __ballot_sync(0xffffffffu, s_tbl[min(p + lane % kPages, p1 - 1) - p0] >= 0);
    constexpr int MT = E == 4 ? 1 : 2;
    int mt = 0;
    float worst = 0.f;
    for (; mt + MT <= tiles; mt += MT)
      score_tiles<D, G2, MT, E>(bd, s_q + mt * kPairs * 64 + lane, mt * kTileRows, nr, p, p1, lane, known,
                                out, row_step, worst);
    if (mt < tiles)
      score_tiles<D, G2, 1, E>(bd, s_q + mt * kPairs * 64 + lane, mt * kTileRows, nr, p, p1, lane, known,
                               out, row_step, worst);
    if (worst != worst) s_odd[warp] = 1;
  }
  __syncthreads();
  if (s_odd[0] | s_odd[1] | s_odd[2] | s_odd[3]) score_again<D>(a, s_tbl);
}

template <int D, int G2, int E>
cudaError_t launch_score(const ScoreArgs& a, dim3 grid, size_t smem, cudaStream_t s) {
  static PerDevice set;
  const size_t most = (size_t)kScoreTiles * (2 * D / 16) * 32 * 16;
  const cudaError_t e = smem_limit_once(set, score_kernel<D, G2, E>, most);
  return e == cudaSuccess ? sv::launch(score_kernel<D, G2, E>, grid, kScoreThreads, smem, s, a) : e;
}
template <int G2>
cudaError_t launch_score(const ScoreArgs& a, int dim, dim3 grid, size_t smem, cudaStream_t s) {
  if (a.per >= 256)
    return dim == 128 ? launch_score<128, G2, 4>(a, grid, smem, s) : launch_score<64, G2, 4>(a, grid, smem, s);
  return dim == 128 ? launch_score<128, G2, 2>(a, grid, smem, s) : launch_score<64, G2, 2>(a, grid, smem, s);
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

// Whole numbers in the order of the scores: NaN below everything, -0 = +0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct SelectRow {
  int r, g, n;
};

// The row and KV head of a CTA; false if it has nothing to choose (every page is
// kept, or the row is left as it is).
__device__ __forceinline__ bool select_row(const SelectArgs& a, SelectRow& s) {
  __shared__ int s_req;
  s.r = blockIdx.x;
  s.g = blockIdx.y;
  const int tid = threadIdx.x;
  // the request that owns the row, asked of all of them at once
  if (tid == 0) s_req = -1;
  __syncthreads();
  for (int i = tid; i < a.bt.n_req; i += blockDim.x)
    if (a.bt.cu_rows[i] <= s.r && s.r < a.bt.cu_rows[i + 1]) atomicMax(&s_req, i);
  __syncthreads();
  const int i = s_req;
  if (i < 0) return false;
  const Window w = window_of(a.bt, i);
  const int ctx = a.lens[i];
  s.n = ctx / kBlockSize;
  if (!w.ok) {
    if (tid == 0 && s.g == 0) flag(a.dev_status, SV_DEV_BAD_WINDOW);
    return false;
  }
  if (ctx < 0 || ctx > (long)a.max_blocks * kBlockSize || s.n > a.max_pages) {
    if (tid == 0 && s.g == 0) flag(a.dev_status, SV_DEV_BAD_LENGTH);
    return false;
  }
  if (s.r < w.cu + w.b || s.r >= w.cu + w.e) return false;
  if (s.n <= a.n_keep) {
    int32_t* out = a.pages + ((size_t)s.r * a.Hkv + s.g) * a.n_keep;
    for (int t = tid; t < a.n_keep; t += blockDim.x) out[t] = t < s.n ? t : -1;
    return false;
  }
  return true;
}

// The score a key stands for (0 is NaN's).
__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

constexpr int kCandidates = 512;
constexpr int kMaxSelect = 49152;  // pages (the call's limit; nothing here is sized by it)

// One CTA a (row, KV head), its scores read from L1 in each pass (kept in shared
// memory they left room for half as many CTAs).  The n_keep-th greatest:
// the keys between the least and the greatest are counted in BINS bins of equal
// width (of the scores; of the keys where the scores' range is no number to
// divide by), the bin that holds the one sought is found from the top, and its
// few keys rank one another.  Where they are many the bin is cut again; equal
// keys need no cut.  Then a bit a page, of those above it and of the first of
// those equal to it, is turned into the list.  Ranges of scores fill equal bins
// better than digits of their bits: few additions meet in one word.  Bound by issue
// slots and barriers (350 rows of 8 heads with 62 .. 6250 pages, 96 kept: 23 us).
template <int THREADS, int BINS>
__global__ void __launch_bounds__(THREADS) select_kernel(SelectArgs a) {
  griddep_entry();
  constexpr int kWarps = THREADS / 32;
  constexpr int kOwn = BINS / THREADS;  // bins a thread adds up
  __shared__ uint32_t s_bin[BINS];
  __shared__ uint32_t s_cand[kCandidates];
  __shared__ uint32_t s_min[kWarps], s_max[kWarps], s_sum[kWarps];
  __shared__ uint32_t s_kth;
  __shared__ int s_found, s_before, s_count, s_above;
  SelectRow sr;
  if (!select_row(a, sr)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = sr.n;
  const float* s = a.scores + ((size_t)sr.r * a.Hkv + sr.g) * a.max_pages;
  // the least and greatest of the keys that are chosen from
  auto range = [&](uint32_t mn, uint32_t mx, uint32_t& lo, uint32_t& hi) {
    mn = __reduce_min_sync(0xffffffffu, mn);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) {
      s_min[warp] = mn;
      s_max[warp] = mx;
    }
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, s_min[lane % kWarps]);
    hi = __reduce_max_sync(0xffffffffu, s_max[lane % kWarps]);
  };
  // before this thread's x of the block's, in the threads' order
  auto scan = [&](uint32_t x) {
    uint32_t y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    if (lane == 31) s_sum[warp] = y;
    __syncthreads();
    uint32_t before = y - x;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (w < warp) before += s_sum[w];
    return before;
  };
  const int t_first = a.n_first, t_last = n - a.n_last;  // the pages chosen from
  uint32_t mn, mx, lo, hi;
  {
    float least = INFINITY, most = -INFINITY;
    bool nan = false;
#pragma unroll 4
    for (int t = t_first + tid; t < t_last; t += THREADS) {
      const float x = __ldg(s + t);
      least = fminf(least, x);
      most = fmaxf(most, x);
      nan |= x != x;
    }
    mn = nan ? 0u : score_key(least);
    mx = score_key(most);
  }
  range(mn, mx, lo, hi);
  int need = a.n_keep - a.n_first - a.n_last;  // keys still sought in lo .. hi
  uint32_t kth = 0xffffffffu;                  // none: the pages that are always kept
  if (need == 0) need = a.n_keep;
  else
    for (bool all = true;; all = false) {
      if (lo == hi) {
        kth = lo;
        break;
      }
      const float xlo = key_score(lo), width = key_score(hi) - xlo;
      const bool linear = lo > 0u && width > 1e-30f && width < 1e38f;
      const float inv = linear ? (float)(BINS - 1) / width : 0.f;
      const bool plain = all && linear;  // the first cut, of numbers: no keys needed
      const int shift = max(0, 32 - __clz(hi - lo) - (31 - __clz(BINS)));
      auto bin = [&](uint32_t k) {  // never falls where k grows
        return linear ? min(BINS - 1, (int)((key_score(k) - xlo) * inv)) : (int)((k - lo) >> shift);
      };
      auto plain_bin = [&](float x) { return min(BINS - 1u, __float2uint_rz(fmaf(x, inv, -xlo * inv))); };
#pragma unroll
      for (int k = 0; k < kOwn; ++k) s_bin[k * THREADS + tid] = 0u;
      if (tid == 0) s_count = s_above = 0;
      __syncthreads();
      if (plain) {
#pragma unroll 4
        for (int t = t_first + tid; t < t_last; t += THREADS) atomicAdd(&s_bin[plain_bin(__ldg(s + t))], 1u);
      } else {
        for (int t = t_first + tid; t < t_last; t += THREADS) {
          const uint32_t k = score_key(__ldg(s + t));
          if (k >= lo && k <= hi) atomicAdd(&s_bin[bin(k)], 1u);
        }
      }
      __syncthreads();
      // thread tid adds up kOwn bins, the highest for thread 0
      uint32_t c[kOwn], sum = 0;
#pragma unroll
      for (int k = 0; k < kOwn; ++k) sum += c[k] = s_bin[BINS - 1 - (tid * kOwn + k)];
      uint32_t before = scan(sum);
      if ((int)before < need && (int)(before + sum) >= need) {
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
          if ((int)before < need && (int)(before + c[k]) >= need) {
            s_found = BINS - 1 - (tid * kOwn + k);
            s_before = (int)before;
          }
          before += c[k];
        }
      }
      __syncthreads();
      const int found = s_found;
      need -= s_before;
      const bool few = s_bin[found] <= (uint32_t)kCandidates;
      mn = 0xffffffffu;
      mx = 0u;
      auto candidate = [&](uint32_t k) {
        mn = min(mn, k);
        mx = max(mx, k);
        if (few) s_cand[atomicAdd(&s_count, 1)] = k;
      };
      if (plain) {
#pragma unroll 4
        for (int t = t_first + tid; t < t_last; t += THREADS) {
          const float x = __ldg(s + t);
          if ((int)plain_bin(x) == found) candidate(score_key(x));
        }
      } else {
        for (int t = t_first + tid; t < t_last; t += THREADS) {
          const uint32_t k = score_key(__ldg(s + t));
          if (k >= lo && k <= hi && bin(k) == found) candidate(k);
        }
      }
      if (!few) {
        __syncwarp();
        range(mn, mx, lo, hi);
        continue;
      }
      __syncthreads();
      // the key with fewer than `need` candidates above it and at least so many at
      // or above it (equal ones find the same)
      const int m = s_count;
      for (int y = tid; y < m; y += THREADS) {
        const uint32_t k = s_cand[y];
        int up = 0, eq = 0;
        for (int z = 0; z < m; ++z) {
          up += s_cand[z] > k;
          eq += s_cand[z] == k;
        }
        if (up < need && up + eq >= need) {
          s_kth = k;
          s_above = up;
        }
      }
      __syncthreads();
      kth = s_kth;
      need -= s_above;
      break;
    }
  // A bit a page: above the threshold, and the first `need` of those equal to it.
  // A word at a time, in the order of the pages, BINS / 2 words at once.
  int32_t* out = a.pages + ((size_t)sr.r * a.Hkv + sr.g) * a.n_keep;
  uint32_t* s_eq = s_bin + BINS / 2;
  const int words = (n + 31) / 32;
  // a threshold between the infinities is compared as a number
  const float xth = key_score(kth);
  const bool numbers = kth > 0x007fffffu && kth < 0xff800000u;
  uint32_t written = 0, equal = 0;  // before these words
  for (int w0 = 0; w0 < words; w0 += BINS / 2) {
    const int nw = min(words - w0, BINS / 2);
    __syncthreads();
    for (int w = warp; w < nw; w += kWarps) {
      const int t = (w0 + w) * 32 + lane;
      bool up, eq;
      if (numbers) {  // NaN is neither
        const float x = t >= t_first && t < t_last ? __ldg(s + t) : t < n ? INFINITY : -INFINITY;
        up = x > xth;
        eq = x == xth;
      } else {
        const uint32_t k = t < t_first || t >= t_last ? 0xffffffffu : score_key(__ldg(s + t));
        up = t < n && k > kth;
        eq = t < n && k == kth;
      }
      const unsigned bu = __ballot_sync(0xffffffffu, up), be = __ballot_sync(0xffffffffu, eq);
      if (lane == 0) {
        s_bin[w] = bu;
        s_eq[w] = be;
      }
    }
    __syncthreads();
    const int per = (nw + THREADS - 1) / THREADS, b0 = min(nw, tid * per), b1 = min(nw, b0 + per);
    uint32_t sum = 0;  // pages above (high half) and equal (low half) in this thread's words
    for (int w = b0; w < b1; ++w) sum += ((uint32_t)__popc(s_bin[w]) << 16) + (uint32_t)__popc(s_eq[w]);
    const uint32_t before = scan(sum);
    uint32_t up = written + (before >> 16), eq = equal + (before & 0xffffu);
    for (int w = b0; w < b1; ++w) {
      const uint32_t above = s_bin[w];
      uint32_t e = s_eq[w];
      const int left = need - (int)eq;  // equal ones still to be taken
      uint32_t take = above;
      if (left >= __popc(e)) take |= e;
      else
        for (int k = 0; k < left; ++k, e &= e - 1) take |= e & (0u - e);
      uint32_t pos = up + min(eq, (uint32_t)need);
      up += __popc(above);
      eq += __popc(s_eq[w]);
      for (; take; take &= take - 1) out[pos++] = (w0 + w) * 32 + __ffs(take) - 1;
    }
    if (w0 + BINS / 2 < words) {  // more words: what came before them
      uint32_t all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) all += s_sum[w];
      written += all >> 16;
      equal += all & 0xffffu;
    }
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
  // enough CTAs for the SMs first, then as many pages as pay for a CTA's start (512: 49
  // us in the case above, 256 51, 128 60, 1024 56)
  a.per = 64;
  while (a.per < pg::kMaxPer && units > 8L * nsm * a.per) a.per *= 2;
  const int per_block = pg::kScoreTiles * 16 / a.g2;
  const int most_rows = std::min(bt->max_rows_per_req, bt->total_rows);
  const dim3 grid((max_pages - 1) / a.per + 1, (most_rows + per_block - 1) / per_block,
                  bt->n_req * kv->n_kv_heads);
  const int tiles = std::min(pg::kScoreTiles, (most_rows * a.g2 + 15) / 16);
  const size_t smem = (size_t)tiles * (2 * kv->head_dim / 16) * 32 * 16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (a.g2) {
    case 1: e = pg::launch_score<1>(a, kv->head_dim, grid, smem, s); break;
    case 2: e = pg::launch_score<2>(a, kv->head_dim, grid, smem, s); break;
    case 4: e = pg::launch_score<4>(a, kv->head_dim, grid, smem, s); break;
    case 8: e = pg::launch_score<8>(a, kv->head_dim, grid, smem, s); break;
    default: e = pg::launch_score<16>(a, kv->head_dim, grid, smem, s); break;
  }
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
  if (n_keep > 1024 || max_pages > pg::kMaxSelect || kv->n_kv_heads > 65535) return SV_ERR_UNSUPPORTED_SHAPE;
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
  const dim3 grid(bt->total_rows, kv->n_kv_heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  // few lists leave SMs idle: more threads for each (350 rows of 8 heads with 62 to
  // 6250 pages: 128 threads a list 40 us, 256 29 us, 512 43 us)
  if ((long)bt->total_rows * kv->n_kv_heads <= sizing_sms())
    e = sv::launch(pg::select_kernel<1024, 2048>, grid, 1024, 0, s, a);
  else
    e = sv::launch(pg::select_kernel<256, 512>, grid, 256, 0, s, a);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
