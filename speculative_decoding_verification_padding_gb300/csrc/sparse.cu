// sparse.cu — sv_page_attend: attention of draft rows over the pages that each
// of them selected.
//
// Source: [SSD] section details (PagedAttention), [SwiftSpec] mechanism 3 (all
// draft rows of a request in one padding-free call); a row's own choice of pages
// is on none of the pages and fixed in the header.
//
// Launches:
//   build  (1 CTA a (tile, KV head)) checks the requests, cuts their rows into tiles
//          of up to 128 virtual rows and makes each list: the union of the rows'
//          page lists as block ids, in page order, with a bit a row and entry for
//          who sees it -- a page that several rows of a tile chose is read once;
//   units, merge (sv_page_units.cuh).

#include "sv_page_units.cuh"

namespace sv {
namespace pu {

constexpr int kMaxTable = 1 << 18;  // table entries a request may have (bits in shared memory)
constexpr int kBuildThreads = 256;
// Entries of the rows' lists that a thread keeps in registers: the first of a tile,
// kHeld x 256 of them; of longer lists it reads the rest again for each step.
constexpr int kHeld = 6;

// Bound by latency, a chain of loads and barriers: what a step needs is asked for as
// soon as its address is known (48 chains of 4000 .. 60000 tokens, 128 pages a row and
// head: 5.2 us after the wait; each step with its own loads, 8.2).
__global__ void __launch_bounds__(kBuildThreads) build_kernel(const __grid_constant__ Args a) {
  griddep_entry();
  extern __shared__ uint32_t s_bits[];  // one bit a page, then the bits before each word
  // (the two scans have a total each: one may still be read when the other begins)
  __shared__ int s_warp[32], s_ntiles, s_npages, s_req, s_k, s_ctx;
  __shared__ Window s_win;
  __shared__ int s_len[kTileRows];
  const int x = blockIdx.x, tile = x / a.Hkv, g = x % a.Hkv, R = a.bt.n_req;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the request that holds the tile, and how many tiles there are
  if (tid == 0) {
    s_ntiles = s_npages = 0;
    if (x == 0 && (a.bt.cu_rows[0] != 0 || a.bt.cu_rows[R] != a.bt.total_rows))
      flag(a.dev_status, SV_DEV_BAD_WINDOW);
  }
  for (int base = 0; base < R; base += kBuildThreads) {
    const int i = base + tid;
    Window w{};
    int nt = 0, ctx = 0;
    if (i < R) {
      w = window_of(a.bt, i);
      ctx = a.lens[i];
      if (w.ok) nt = (max(w.b, w.e) - w.b + a.rt - 1) / a.rt;
      else if (x == 0) flag(a.dev_status, SV_DEV_BAD_WINDOW);
    }
    const int at = block_scan(nt, s_warp, &s_ntiles);
    if (at <= tile && tile < at + nt) {
      s_req = i;
      s_k = tile - at;
      s_win = w;
      s_ctx = ctx;
    }
  }
  __syncthreads();
  // (offsets that overlap could ask for more tiles than there are; such a call is left out)
  const int T = s_ntiles <= a.tiles_cap ? s_ntiles : 0;
  if (x == 0 && tid == 0) {
    if (s_ntiles > a.tiles_cap) flag(a.dev_status, SV_DEV_BAD_WINDOW);
    a.hdr->T = T;
  }
  if (tile >= T) return;
  const int i = s_req, ctx = s_ctx;
  const Window w = s_win;
  const int r0 = w.b + s_k * a.rt, nr = min(a.rt, w.e - r0), n = max(ctx, 0) / kBlockSize;
  // a warp takes 32 entries of a row at once
  constexpr int kWarps = kBuildThreads / 32;
  const int32_t* rows = a.pages + ((size_t)(w.cu + r0) * a.Hkv + g) * a.n_keep;
  const int32_t* table = a.tables + (size_t)i * a.max_blocks;
  const size_t row_step = (size_t)a.Hkv * a.n_keep;
  const int chunks = (a.n_keep + 31) / 32, runs = nr * chunks;
  struct Entry {
    int r, k, page, prev, block;
  };
  auto read = [&](int y) {  // (page and the one before it, where there are any)
    Entry e{0, a.n_keep, -1, -1, -1};
    if (y < runs) {
      e.r = y / chunks;
      e.k = (y - e.r * chunks) * 32 + lane;
      const int32_t* list = rows + e.r * row_step + e.k;
      if (e.k < a.n_keep) e.page = __ldg(list);
      if (e.k < a.n_keep && e.k > 0) e.prev = __ldg(list - 1);
    }
    return e;
  };
  auto block_of = [&](int page) { return page >= 0 && page < a.max_blocks ? __ldg(table + page) : -1; };
  Entry held[kHeld];
#pragma unroll
  for (int q = 0; q < kHeld; ++q) held[q] = read(warp + q * kWarps);
  bool bad = false;
  if (tid < w.rows) {
    const int p = a.bt.parent[w.cu + tid];
    bad = tid == 0 ? p != -1 : (p < 0 || p >= tid);
  }
  const bool fits = ctx >= 0 && (long)ctx + w.rows <= (long)a.max_blocks * kBlockSize;
  const int words = fits ? (n + 31) / 32 : 0;
  uint32_t* s_before = s_bits + words;
  for (int y = tid; y < words; y += kBuildThreads) s_bits[y] = 0u;
  uint32_t* see = a.see + (size_t)x * a.rt * (a.cap / 32);
  for (int y = tid; y < nr * (a.cap / 32); y += kBuildThreads) see[y] = 0u;
  if (tid < nr) s_len[tid] = a.n_keep;
  if (__syncthreads_or(bad) || !fits) {
    // an empty list
    if (tid == 0) {
      a.cnt[2 * x] = a.cnt[2 * x + 1] = 0;
      if (g == 0 && s_k == 0) flag(a.dev_status, fits ? SV_DEV_BAD_PARENT : SV_DEV_BAD_LENGTH);
    }
    return;
  }
  if (g == 0 && tid == 0) {
    Tile t{};
    t.i = i;
    t.cu = w.cu;
    t.ctx = ctx;
    t.r0 = r0;
    t.nr = nr;
    t.rows = w.rows;
    a.tiles[tile] = t;
  }
  const int ntail = (ctx + r0 + nr + kBlockSize - 1) / kBlockSize - n;
  const int tail_block = tid < ntail ? __ldg(table + n + tid) : -1;
#pragma unroll
  for (int q = 0; q < kHeld; ++q) held[q].block = block_of(held[q].page);
  auto entries = [&](auto&& f) {
#pragma unroll
    for (int q = 0; q < kHeld; ++q)
      if (held[q].k < a.n_keep) f(held[q]);
    for (int y = warp + kHeld * kWarps; y < runs; y += kWarps) {
      Entry e = read(y);
      if (e.k < a.n_keep) {
        e.block = block_of(e.page);
        f(e);
      }
    }
  };
  // a row's list ends where its pages stop to ascend
  entries([&](const Entry& e) {
    if (e.page <= e.prev || e.page >= n) atomicMin(&s_len[e.r], e.k);
  });
  __syncthreads();
  entries([&](const Entry& e) {
    if (e.k < s_len[e.r]) atomicOr(&s_bits[e.page >> 5], 1u << (e.page & 31));
    else if (e.k == s_len[e.r] && e.page != -1) flag(a.dev_status, SV_DEV_BAD_PARAM);
  });
  __syncthreads();
  for (int base = 0; base < words; base += kBuildThreads) {
    const int y = base + tid;
    const int before = block_scan(y < words ? __popc(s_bits[y]) : 0, s_warp, &s_npages);
    if (y < words) s_before[y] = (uint32_t)before;
  }
  __syncthreads();
  const int U = s_npages;
  int* blk = a.blk + (size_t)x * a.cap;
  entries([&](const Entry& e) {
    if (e.k >= s_len[e.r]) return;
    const int v = e.page, pos = (int)s_before[v >> 5] + __popc(s_bits[v >> 5] & ((1u << (v & 31)) - 1u));
    blk[pos] = e.block;  // the same from every row that lists it
    atomicOr(see + (size_t)e.r * (a.cap / 32) + (pos >> 5), 1u << (pos & 31));
  });
  if (tid < ntail) blk[U + tid] = tail_block;
  if (tid == 0) {
    a.cnt[2 * x] = U;
    a.cnt[2 * x + 1] = U + ntail;
  }
}

template <int D>
__global__ void __launch_bounds__(unit::kThreads, 1)
    page_unit_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmQ) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(16) unit::Shared sh;
  __shared__ int s_scan[32], s_carry, s_first[2];
  __shared__ uint32_t s_tmem;
  const int c = blockIdx.x, tid = threadIdx.x, warp = tid >> 5;
  // nothing that earlier kernels write is read before griddep_entry()
  if (tid == 0) unit::init(sh);
  if (warp == 8) {
    if ((tid & 31) == 0) {
      prefetch_map(&tmK);
      prefetch_map(&tmV);
      prefetch_map(&tmQ);
    }
    __syncwarp();
    tc5::tmem_alloc(smem_u32(&s_tmem), unit::kCols);
    tc5::tmem_relinquish();
  }
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  const uint32_t tmem = s_tmem;
  griddep_entry();
  // A run of lists a thread: the stages before it, and of all of them
  const int lists = a.hdr->T * a.Hkv, per = (lists + unit::kThreads - 1) / unit::kThreads;
  const int y0 = min(lists, tid * per), y1 = min(lists, y0 + per);
  auto stages = [&](int y) { return (a.cnt[2 * y + 1] + kStagePages - 1) / kStagePages; };
  int sum = 0;
  for (int y = y0; y < y1; ++y) sum += stages(y);
  if (tid == 0) s_carry = 0;
  int at = block_scan(sum, s_scan, &s_carry);
  const int W = s_carry, C = min(a.ctas, W);
  const int s0 = c < C ? share_start(c, W, C) : -1;
  for (int y = y0; y < y1; ++y) {
    if (c == 0) a.off[y] = at;  // for the merge
    const int n = stages(y);
    if (at <= s0 && s0 < at + n) {
      s_first[0] = y;
      s_first[1] = at;
    }
    at += n;
  }
  if (c == 0 && tid == 0) {
    a.off[lists] = W;
    a.hdr->W = W;
    a.hdr->C = C;
  }
  __syncthreads();
  if (c < C)
    unit_share<D, true>(a, tmK, tmV, tmQ, sh, smem_raw + ((1024 - smem_u32(smem_raw)) & 1023), tmem, c, W, C,
                        s_first[0], s_first[1]);
  if (warp == 8) tc5::tmem_dealloc(tmem, unit::kCols);
}

inline Args page_args(const sv_paged_kv* kv, const sv_batch* bt, int32_t Hq, int32_t n_keep,
                      uint8_t* at, size_t& off) {
  Args a = common_args(kv, bt, Hq, at, off);
  a.n_keep = n_keep;
  // the rows' pages, and a tail of at most (15 + 128 + 15) / 16 pages
  const long most = std::min((long)kv->max_blocks_per_req, (long)a.rt * n_keep) + 9;
  a.cap = (int)((most + 31) / 32 * 32);
  const size_t lists = (size_t)a.tiles_cap * a.Hkv;
  a.blk = take<int>(at, off, lists * a.cap);
  a.see = take<uint32_t>(at, off, lists * a.rt * (a.cap / 32));
  a.cnt = take<int>(at, off, lists * 2);
  return a;
}

template <int D>
sv_status page_attend(const Args& a, const void* k, const void* v, cudaStream_t stream) {
  CUtensorMap tmK, tmV, tmQ;
  if (!attn::make_map(&tmK, k, a.num_blocks, a.Hkv, D) || !attn::make_map(&tmV, v, a.num_blocks, a.Hkv, D) ||
      !make_q_map(&tmQ, a, D))
    return SV_ERR_CUDA;
  const size_t words = ((size_t)a.max_blocks + 31) / 32;
  static PerDevice set_build, set_unit;
  if (smem_limit_once(set_build, build_kernel, kMaxTable / 32 * 8) != cudaSuccess ||
      smem_limit_once(set_unit, page_unit_kernel<D>, unit::Smem<D>::kAsk) != cudaSuccess)
    return SV_ERR_CUDA;
  if (sv::launch(build_kernel, a.tiles_cap * a.Hkv, kBuildThreads, words * 8, stream, a) != cudaSuccess ||
      sv::launch(page_unit_kernel<D>, a.ctas, unit::kThreads, unit::Smem<D>::kAsk, stream, a, tmK, tmV, tmQ) !=
          cudaSuccess ||
      launch_merge<D, true>(a, stream) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}

inline sv_status check_pages(const sv_paged_kv* kv, const sv_batch* bt, int32_t Hq, int32_t n_keep) {
  const sv_status st = check(kv, bt, Hq);
  if (st != SV_OK) return st;
  if (n_keep < 0) return SV_ERR_INVALID_ARGUMENT;
  if (n_keep > 1024 || kv->max_blocks_per_req > kMaxTable) return SV_ERR_UNSUPPORTED_SHAPE;
  return SV_OK;
}

}  // namespace pu
}  // namespace sv

using namespace sv;

extern "C" size_t sv_page_attend_workspace(const sv_batch* bt, const sv_paged_kv* kv,
                                           int32_t n_q_heads, int32_t n_keep) {
  if (pu::check_pages(kv, bt, n_q_heads, n_keep) != SV_OK) return 0;
  size_t off = 0;
  const pu::Args a = pu::page_args(kv, bt, n_q_heads, n_keep, nullptr, off);
  return pu::counts_fit((long)a.tiles_cap * a.Hkv, a.max_blocks) ? off : 0;
}

extern "C" sv_status sv_page_attend(const sv_paged_kv* kv, const sv_batch* bt, const void* q,
                                    int32_t n_q_heads, float softmax_scale, const int32_t* pages,
                                    int32_t n_keep, void* out, void* ws, size_t ws_bytes,
                                    int32_t* dev_status, void* stream) {
  SV_TRACE("sv_page_attend");
  const sv_status st = pu::check_pages(kv, bt, n_q_heads, n_keep);
  if (st != SV_OK) return st;
  if (bt->n_req == 0 || bt->total_rows == 0) return SV_OK;
  if (!q || !out || !ws || (n_keep > 0 && !pages)) return SV_ERR_INVALID_ARGUMENT;
  if (((uintptr_t)q | (uintptr_t)out) & 15) return SV_ERR_INVALID_ARGUMENT;
  if ((uintptr_t)ws & 255) return SV_ERR_INVALID_ARGUMENT;
  if (!(softmax_scale > 0.f)) return SV_ERR_INVALID_ARGUMENT;
  size_t need = 0;
  pu::Args a = pu::page_args(kv, bt, n_q_heads, n_keep, static_cast<uint8_t*>(ws), need);
  if (!pu::counts_fit((long)a.tiles_cap * a.Hkv, a.max_blocks)) return SV_ERR_UNSUPPORTED_SHAPE;
  if (pu::overlap(q, out, bt, n_q_heads, kv->head_dim)) return SV_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need) return SV_ERR_WORKSPACE_TOO_SMALL;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.pages = pages;
  a.dev_status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return kv->head_dim == 128 ? pu::page_attend<128>(a, kv->k_cache, kv->v_cache, s)
                             : pu::page_attend<64>(a, kv->k_cache, kv->v_cache, s);
}
