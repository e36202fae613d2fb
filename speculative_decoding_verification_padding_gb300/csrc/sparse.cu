// sparse.cu — sv_page_attend: attention of draft rows over the pages that each
// of them selected.
//
// Source: [SSD] section details (PagedAttention), [SwiftSpec] mechanism 3 (all
// draft rows of a request in one padding-free call); a row's own choice of pages
// is on none of the pages and fixed in the header.
//
// Launches:
//   plan   (1 CTA) checks the requests and cuts their rows into tiles of up to
//          128 virtual rows;
//   build  (1 CTA a (tile, KV head)) the union of the rows' page lists as block
//          ids, in page order, with a bit a row and entry for who sees it: a page
//          that several rows of a tile chose is read once.  The last CTA deals the
//          lists' stages out;
//   units, merge (sv_page_units.cuh).

#include "sv_page_units.cuh"

namespace sv {
namespace pu {

constexpr int kMaxTable = 1 << 18;  // table entries a request may have (bits in shared memory)
constexpr int kBuildThreads = 256;

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const __grid_constant__ Args a) {
  griddep_entry();
  __shared__ int s_warp[32], s_tiles;
  extern __shared__ __align__(16) uint8_t s_mem[];
  const int R = a.bt.n_req, tid = threadIdx.x;
  Req* req = R <= kPlanRequests ? reinterpret_cast<Req*>(s_mem) : a.req;
  if (tid == 0) {
    s_tiles = 0;
    if (a.bt.cu_rows[0] != 0 || a.bt.cu_rows[R] != a.bt.total_rows) flag(a.dev_status, SV_DEV_BAD_WINDOW);
  }
  check_requests(a, req);
  for (int base = 0; base < R; base += blockDim.x) {
    const int i = base + tid;
    const int nt = i < R ? (req[i].e - req[i].b + a.rt - 1) / a.rt : 0;
    const int at = block_scan(nt, s_warp, &s_tiles);
    if (i < R) req[i].tile = at;
  }
  // (offsets that overlap could ask for more tiles than there are; such a call is left out)
  const bool fits = s_tiles <= a.tiles_cap;
  if (tid == 0) {
    if (!fits) flag(a.dev_status, SV_DEV_BAD_WINDOW);
    a.hdr->T = fits ? s_tiles : 0;
    a.hdr->W = 0;
    a.hdr->C = 0;
    a.hdr->ticket = 0;
  }
  __syncthreads();
  if (fits) write_tiles(a, req);
}

__global__ void __launch_bounds__(kBuildThreads) build_kernel(const __grid_constant__ Args a) {
  griddep_entry();
  extern __shared__ uint32_t s_bits[];  // one bit a page, then the bits before each word
  __shared__ int s_warp[32], s_carry, s_last;
  __shared__ int s_len[kTileRows];
  const int x = blockIdx.x;
  const int lists = a.hdr->T * a.Hkv;
  if (x >= lists) return;
  const Tile tl = a.tiles[x / a.Hkv];
  const int g = x % a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = tl.ctx / kBlockSize, words = (n + 31) / 32;
  uint32_t* s_before = s_bits + words;
  for (int y = tid; y < words; y += kBuildThreads) s_bits[y] = 0u;
  if (tid == 0) s_carry = 0;
  __syncthreads();
  const int32_t* rows = a.pages + ((size_t)(tl.cu + tl.r0) * a.Hkv + g) * a.n_keep;
  const size_t row_step = (size_t)a.Hkv * a.n_keep;
  // a row's list ends where its pages stop to ascend
  for (int r = warp; r < tl.nr; r += kBuildThreads / 32) {
    const int32_t* list = rows + r * row_step;
    int last = -1, len = 0;
    for (int k0 = 0; k0 < a.n_keep; k0 += 32) {
      const int k = k0 + lane;
      const int v = k < a.n_keep ? __ldg(list + k) : -1;
      int prev = __shfl_up_sync(0xffffffffu, v, 1);
      if (lane == 0) prev = last;
      const unsigned bad = __ballot_sync(0xffffffffu, v <= prev || v >= n);
      const int good = bad ? __ffs(bad) - 1 : 32;
      if (lane < good) atomicOr(&s_bits[v >> 5], 1u << (v & 31));
      len += good;
      if (bad) {
        if (lane == good && v != -1) flag(a.dev_status, SV_DEV_BAD_PARAM);
        break;
      }
      last = __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) s_len[r] = len;
  }
  __syncthreads();
  for (int base = 0; base < words; base += kBuildThreads) {
    const int y = base + tid;
    const int before = block_scan(y < words ? __popc(s_bits[y]) : 0, s_warp, &s_carry);
    if (y < words) s_before[y] = (uint32_t)before;
  }
  __syncthreads();
  const int U = s_carry;
  int* blk = a.blk + (size_t)x * a.cap;
  uint32_t* see = a.see + (size_t)x * a.rt * (a.cap / 32);
  const int32_t* table = a.tables + (size_t)tl.i * a.max_blocks;
  for (int y = tid; y < words; y += kBuildThreads) {
    uint32_t bits = s_bits[y];
    for (int pos = (int)s_before[y]; bits; bits &= bits - 1, ++pos)
      blk[pos] = __ldg(table + y * 32 + __ffs(bits) - 1);
  }
  for (int y = tid; y < tl.nr * (a.cap / 32); y += kBuildThreads) see[y] = 0u;
  const int ntail = (tl.ctx + tl.r0 + tl.nr + kBlockSize - 1) / kBlockSize - n;
  for (int k = tid; k < ntail; k += kBuildThreads) blk[U + k] = __ldg(table + n + k);
  __syncthreads();
  for (int r = warp; r < tl.nr; r += kBuildThreads / 32) {
    const int32_t* list = rows + r * row_step;
    for (int k = lane; k < s_len[r]; k += 32) {
      const int v = __ldg(list + k);
      const int pos = (int)s_before[v >> 5] + __popc(s_bits[v >> 5] & ((1u << (v & 31)) - 1u));
      atomicOr(see + (size_t)r * (a.cap / 32) + (pos >> 5), 1u << (pos & 31));
    }
  }
  if (tid == 0) {
    a.cnt[2 * x] = U;
    a.cnt[2 * x + 1] = U + ntail;
    s_last = ticket_add(&a.hdr->ticket, 1) == lists - 1;
    s_carry = 0;
  }
  __syncthreads();
  if (!s_last) return;
  // every list is known: their first stages, and the CTAs' shares
  for (int base = 0; base < lists; base += kBuildThreads) {
    const int y = base + tid;
    const int v = y < lists ? (__ldcg(a.cnt + 2 * y + 1) + kStagePages - 1) / kStagePages : 0;
    const int at = block_scan(v, s_warp, &s_carry);
    if (y < lists) a.off[y] = at;
  }
  __syncthreads();
  const int W = s_carry, C = min(a.ctas, W);
  if (tid == 0) {
    a.off[lists] = W;
    a.hdr->W = W;
    a.hdr->C = C;
  }
  __syncthreads();
  for (int y = tid; y < lists; y += kBuildThreads) deal_list(a, y, a.off[y], a.off[y + 1], W, C);
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
  CUtensorMap tmK, tmV;
  if (!attn::make_map(&tmK, k, a.num_blocks, a.Hkv, D) || !attn::make_map(&tmV, v, a.num_blocks, a.Hkv, D))
    return SV_ERR_CUDA;
  const size_t words = ((size_t)a.max_blocks + 31) / 32;
  static PerDevice set;
  if (smem_limit_once(set, build_kernel, kMaxTable / 32 * 8) != cudaSuccess) return SV_ERR_CUDA;
  if (sv::launch(page_plan_kernel, 1, kPlanThreads, plan_smem(a), stream, a) != cudaSuccess ||
      sv::launch(build_kernel, a.tiles_cap * a.Hkv, kBuildThreads, words * 8, stream, a) != cudaSuccess)
    return SV_ERR_CUDA;
  return launch_units<D, true>(a, tmK, tmV, stream);
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
  (void)pu::page_args(kv, bt, n_q_heads, n_keep, nullptr, off);
  return off;
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
