// prefix.cu — sv_prefix_attend: verification attention of a batch whose requests
// share a prefix, the prefix's pages read once for all rows of a group.
//
// Sources: [SwiftSpec] mechanism 3 (one padding-free call for all draft rows),
// [SSD] section details (PagedAttention: requests that share a prompt share its
// pages); computing the shared part once is on none of the pages.
//
// softmax over (prefix, own keys) = the two parts' (max, sum, weighted values)
// joined.  Launches:
//   plan    (1 CTA) checks groups and requests, decides which requests share, lists
//           their rows by group, cuts them into prefix lists and all requests' rows
//           into tiles, divides the CTAs between the two and deals out both;
//   prefix  (tcgen05, one CTA an SM) some CTAs the prefix lists -- 256 virtual rows
//           (rows of all requests of the group x GQA group) by the prefix's pages:
//           (max, sum, O) -- and the others the tiles' own pages (unit_share);
//   merge   (sv_page_units.cuh) a row's parts of both.

#include "sv_page_units.cuh"
#include "sv_tcgen05.cuh"

namespace sv {
namespace pu {

constexpr int kPlanThreads = 1024;
// Requests and groups whose records the plan keeps in shared memory; with more of
// them they are in the workspace.
constexpr int kPlanRequests = 512, kPlanGroups = 256;

struct PlanSmem {
  Req req[kPlanRequests];
  int4 groups[kPlanGroups];
  int cu_groups[kPlanGroups + 1], prefix_len[kPlanGroups], gstage[kPlanGroups + 1];
};

// The time that `rows` virtual rows of a group take on one SM for a prefix of
// `stages` stages, in quarters of an own stage (one tile by 128 tokens, however few
// rows the tile has): a stage of a prefix list takes 5 with two tiles and 3 with one,
// of head_dim 64 (half the copies and products, the same softmax) 4 and 2.5.
__device__ __forceinline__ long prefix_cost(const Args& a, long rows, int stages) {
  const long tiles = (rows + 127) / 128;
  return (a.dim == 128 ? 5 * tiles + 1 : 3 * tiles + 2) * (stages + kListStart) / 2;
}

// Whether a request's rows go with its group's prefix lists (n requests about like it
// in the group), or its own lists read the prefix's pages too.  A row in two parts
// writes and reads both.  Where all own stages are few the SMs are there for them.
// (27 trees of 83 rows, 16 heads a KV head, behind 16 .. 832 tokens: 98 us with own
// lists only, 174 with prefix lists; 62 chains of 2 rows behind 16 tokens 24 and 33; 64
// chains of 7 rows behind 24576 tokens 748 and 293; 30 trees of 41 rows, 7 heads a KV
// head, behind 809, 2024 and 5060 tokens 43.8 and 42.8, by the rule 41.8; 4 chains behind
// 2048 tokens 21.8 and 21.9.)
__device__ __forceinline__ bool shared_pays(const Args& a, int n, int vrows, int tiles, int stages) {
  if ((long)a.bt.n_req * tiles * a.Hkv * stages <= 6L * a.ctas) return false;
  const long rows = (long)n * vrows;
  return 4L * stages * tiles * n > prefix_cost(a, rows, stages) + rows * (5 * a.dim / 64) / 64;
}

__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const __grid_constant__ Args a) {
  griddep_entry();
  extern __shared__ __align__(16) uint8_t s_mem[];
  __shared__ int s_tiles, s_stages, s_rows, s_pstages, s_groups_bad;
  __shared__ long s_pcost;
  PlanSmem& sm = *reinterpret_cast<PlanSmem*>(s_mem);
  const int R = a.bt.n_req, G = a.n_groups, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool small = R <= kPlanRequests && G <= kPlanGroups;  // in shared memory
  Req* req = small ? sm.req : a.req;
  int4* groups = small ? sm.groups : a.groups;
  int* gstage = small ? sm.gstage : a.gstage;
  const int32_t* cu_groups = small ? sm.cu_groups : a.cu_groups;
  const int32_t* prefix_len = small ? sm.prefix_len : a.prefix_len;
  if (tid == 0) s_groups_bad = 0;
  // (asked for ahead of what the requests' rows are read for)
  const int k0 = min(tid, G), cu0 = a.cu_groups[k0], cu1 = a.cu_groups[min(k0 + 1, G)],
            len0 = a.prefix_len[min(k0, G - 1)];
  // windows, parents and lengths, 16 lanes a request; what cannot be attended is
  // reported and left out
  constexpr int kLanes = 16;
  for (int i0 = 0; i0 < R; i0 += kPlanThreads / kLanes) {
    const int i = i0 + tid / kLanes, l = tid % kLanes;
    Window w{};
    int ctx = 0;
    bool bad = false;
    if (i < R) {
      w = window_of(a.bt, i);
      ctx = a.lens[i];
      if (w.ok) {
#pragma unroll
        for (int k = 0; k < kMaxRows / kLanes; ++k) {
          const int j = l + kLanes * k;
          if (j < w.rows) {
            const int p = a.bt.parent[w.cu + j];
            bad |= j == 0 ? p != -1 : (p < 0 || p >= j);
          }
        }
      }
    }
    bad = (__ballot_sync(0xffffffffu, bad) >> (lane & 16)) & 0xffffu;
    if (i >= R || l != 0) continue;
    const bool fits = ctx >= 0 && (long)ctx + w.rows <= (long)a.max_blocks * kBlockSize;
    if (!w.ok) flag(a.dev_status, SV_DEV_BAD_WINDOW);
    else if (bad) flag(a.dev_status, SV_DEV_BAD_PARENT);
    else if (!fits) flag(a.dev_status, SV_DEV_BAD_LENGTH);
    Req r{};
    r.cu = w.cu;
    r.rows = w.rows;
    r.b = w.b;
    r.e = w.ok && !bad && fits ? max(w.b, w.e) : w.b;  // (a window behind the verified rows is empty)
    r.ctx = ctx;
    req[i] = r;
  }
  if (tid == 0 && (a.bt.cu_rows[0] != 0 || a.bt.cu_rows[R] != a.bt.total_rows))
    flag(a.dev_status, SV_DEV_BAD_WINDOW);
  // groups that do not cut the requests into runs: nothing is attended
  auto check = [&](int k, int v, int next) {
    if ((k == 0 && v != 0) || (k < G ? v > next : v != R)) s_groups_bad = 1;
  };
  __syncthreads();
  if (tid <= G) check(tid, cu0, cu1);
  for (int k = tid + kPlanThreads; k <= G; k += kPlanThreads) check(k, a.cu_groups[k], a.cu_groups[min(k + 1, G)]);
  if (small && tid <= G) {
    sm.cu_groups[tid] = cu0;
    if (tid < G) sm.prefix_len[tid] = len0;
  }
  __syncthreads();
  if (s_groups_bad) {
    if (tid == 0) {
      flag(a.dev_status, SV_DEV_BAD_PARAM);
      a.hdr->T = a.hdr->W = a.hdr->C = a.hdr->Wp = a.hdr->Cp = 0;
    }
    return;
  }
  // The last entry at or before v of a table that does not descend (entries of none
  // are as the one behind them).
  auto last_at = [&](int n, int v, auto&& at) {
    int lo = 0;
    for (int hi = n - 1; lo < hi;) {
      const int mid = (lo + hi + 1) >> 1;
      if (at(mid) <= v) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  // the request's group, tiles and stages
  auto stages_of = [&](const Req& r, int k) {  // of its tile k
    return ((r.ctx + min(r.b + (k + 1) * a.rt, r.e) + kBlockSize - 1) / kBlockSize - r.first + kStagePages - 1) /
           kStagePages;
  };
  for (int i = tid; i < R; i += blockDim.x) {
    Req r = req[i];
    const int lo = last_at(G, i, [&](int k) { return cu_groups[k]; }), p = prefix_len[lo];
    if (r.e > r.b && (p < 0 || p % kBlockSize != 0 || p > r.ctx)) {
      flag(a.dev_status, p < 0 || p % kBlockSize != 0 ? SV_DEV_BAD_PARAM : SV_DEV_BAD_LENGTH);
      r.e = r.b;
    }
    const int nt = (r.e - r.b + a.rt - 1) / a.rt, pages = r.e > r.b ? p / kBlockSize : 0;
    const bool share = pages > 0 && shared_pays(a, cu_groups[lo + 1] - cu_groups[lo], (r.e - r.b) * a.group, nt,
                                                (pages + kStagePages - 1) / kStagePages);
    r.grp = lo;
    r.first = share ? pages : 0;
    r.pre = pages - r.first;
    r.tile = nt;  // counts, for now
    r.stage = 0;
    for (int k = 0; k < nt; ++k) r.stage += stages_of(r, k);
    r.arow = share ? r.e - r.b : 0;
    req[i] = r;
  }
  __syncthreads();
  // offsets of all three, by one warp, a run of requests a lane
  if (warp == 0) {
    const int per = (R + 31) / 32, i0 = min(R, lane * per), i1 = min(R, i0 + per);
    int c[3] = {0, 0, 0}, at[3];
    for (int i = i0; i < i1; ++i) {
      c[0] += req[i].tile;
      c[1] += req[i].stage;
      c[2] += req[i].arow;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      int x = c[k];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      at[k] = x - c[k];
      c[k] = __shfl_sync(0xffffffffu, x, 31);
    }
    for (int i = i0; i < i1; ++i) {
      const int t = req[i].tile, s = req[i].stage, n = req[i].arow;
      req[i].tile = at[0];
      req[i].stage = at[1];
      req[i].arow = at[2];
      at[0] += t;
      at[1] += s;
      at[2] += n;
    }
    __syncwarp();
    const int rows = c[2];
    // groups: first row, rows, pages; their lists, one a 256-row tile
    // and KV head, and the lists' stages
    auto arow = [&](int i) { return i < R ? req[i].arow : rows; };
    int lists = 0, stages = 0;
    long cost = 0;
    for (int base = 0; base < G; base += 32) {
      const int k = base + lane;
      int4 gr = make_int4(0, 0, 0, 0);
      int n = 0, s = 0;
      if (k < G) {
        gr.x = arow(cu_groups[k]);
        gr.y = arow(cu_groups[k + 1]) - gr.x;
        gr.z = gr.y > 0 ? prefix_len[k] / kBlockSize : 0;  // checked by its requests
        n = gr.z > 0 ? (gr.y * a.group + kPrefixRows - 1) / kPrefixRows * a.Hkv : 0;
        s = n * ((gr.z + kStagePages - 1) / kStagePages + kListStart);
        if (n > 0) cost += a.Hkv * prefix_cost(a, (long)gr.y * a.group, (gr.z + kStagePages - 1) / kStagePages);
      }
      int x = n, y = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) { x += u; y += v; }
      }
      gr.w = lists + x - n;
      if (k < G) {
        groups[k] = gr;
        gstage[k] = stages + y - s;
        if (small) {
          a.groups[k] = gr;
          a.gstage[k] = stages + y - s;
        }
      }
      lists += __shfl_sync(0xffffffffu, x, 31);
      stages += __shfl_sync(0xffffffffu, y, 31);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) cost += __shfl_xor_sync(0xffffffffu, cost, o);
    if (lane == 0) {
      s_pcost = cost;
      s_tiles = c[0];
      s_stages = c[1];
      s_rows = rows;
      s_pstages = stages;
    }
  }
  __syncthreads();
  // (offsets that overlap could ask for more than there is; such a call is left out)
  if (s_tiles > a.tiles_cap || s_rows > a.bt.total_rows) {
    if (tid == 0) {
      flag(a.dev_status, SV_DEV_BAD_WINDOW);
      a.hdr->T = a.hdr->W = a.hdr->C = a.hdr->Wp = a.hdr->Cp = 0;
    }
    return;
  }
  // The CTAs that take prefix stages and those that take the requests' own: both at
  // once, as one is bound by the tensor cores and the other by memory (448 rows of 64
  // heads behind 24576 tokens, 100 .. 2000 tokens of a request's own: 303 us, one after
  // the other 327).  Divided by what both take, an own list's start 5, so that both
  // kinds end at the same time.
  const int W = s_stages * a.Hkv, Wp = s_pstages;
  int Cp = min(a.ctas, Wp), C = min(a.ctas, W);
  if (Wp > 0 && W > 0) {
    const long all = s_pcost + 4L * W + 5L * s_tiles * a.Hkv;
    Cp = min(Wp, max(1, min(a.ctas - 1, (int)((a.ctas * s_pcost + all / 2) / all))));
    C = min(W, max(1, a.ctas - Cp));
  }
  if (tid == 0) {
    a.hdr->T = s_tiles;
    a.hdr->W = W;
    a.hdr->C = C;
    a.hdr->Wp = Wp;
    a.hdr->Cp = Cp;
    a.off[(size_t)s_tiles * a.Hkv] = W;
    a.gstage[G] = Wp;
  }
  // Each table from a thread of its own on, as most are short.
  auto from = [&](int first) { return (tid - first) & (kPlanThreads - 1); };
  // the list of the first stage of each CTA's share of the own stages
  for (int c = tid; c < C; c += kPlanThreads) {
    int s = share_start(c, W, C), k = 0;
    const int sh = s / a.Hkv;
    const Req r = req[last_at(R, sh, [&](int i) { return req[i].stage; })];
    s -= r.stage * a.Hkv;
    int n = stages_of(r, 0);
    while (s >= n * a.Hkv) {
      s -= n * a.Hkv;
      n = stages_of(r, ++k);
    }
    a.start[c] = (r.tile + k) * a.Hkv + s / n;
  }
  // the last stage of each CTA's share of the prefix stages
  for (int c = from(160); c < Cp; c += kPlanThreads) {
    const int s = share_start(c + 1, Wp, Cp) - 1;
    PEnd ps{};
    ps.k = last_at(G, s, [&](int k) { return gstage[k]; });
    ps.gr = groups[ps.k];
    const int sp = (ps.gr.z + kStagePages - 1) / kStagePages + kListStart;
    ps.list = (s - gstage[ps.k]) / sp;
    ps.at = (s - gstage[ps.k]) - ps.list * sp;
    ps.leader = cu_groups[ps.k];
    a.pend[c] = ps;
  }
  // rows of the prefix lists
  for (int y = from(320); y < s_rows; y += kPlanThreads) {
    const Req r = req[last_at(R, y, [&](int i) { return req[i].arow; })];
    a.arows[y] = r.cu + r.b + y - r.arow;
  }
  // tiles and the first stages of their lists
  for (int x = from(512); x < s_tiles * a.Hkv; x += kPlanThreads) {
    const int tile = x / a.Hkv, g = x - tile * a.Hkv;
    const int i = last_at(R, tile, [&](int j) { return req[j].tile; });
    const Req r = req[i];
    const int k = tile - r.tile;
    int before = 0;
    for (int j = 0; j < k; ++j) before += stages_of(r, j);
    a.off[x] = (r.stage + before) * a.Hkv + g * stages_of(r, k);
    if (g != 0) continue;
    Tile t{};
    t.i = i;
    t.cu = r.cu;
    t.ctx = r.ctx;
    t.r0 = r.b + k * a.rt;
    t.nr = min(a.rt, r.e - t.r0);
    t.rows = r.rows;
    t.first = r.first;
    t.ncomp = r.ctx / kBlockSize - r.first;
    t.nent = (r.ctx + t.r0 + t.nr + kBlockSize - 1) / kBlockSize - r.first;
    t.arow = r.arow + k * a.rt;
    t.grp = r.grp;
    t.pre = r.pre;
    a.tiles[tile] = t;
  }
}

// ------------------------------------------------------------ tcgen05 --
// A list is two tiles of 128 virtual rows of a group by its prefix, 128 tokens a
// stage; all stages are dealt out evenly to the CTAs.  S = Q K^T and O += P V of a
// tile are tcgen05.mma of 128 x 128 (S) and 128 x D (O).  Tensor memory: S in
// columns 0 .. 127, of one tile and then the other, P (bf16) of the tiles in 128 ..
// 191 and 192 .. 255, O in 256 .. 511.
//   A CTA takes the lists of its share from the last to the first.  The last begins
// at stage 0 of the prefix and the first goes on to the prefix's end, so that all
// CTAs move through the prefix together and what one has read is still in L2 for the
// others (first list first, the CTAs were spread over the whole prefix: 1.22 GB from
// HBM for 448 rows of 64 heads behind 24576 tokens, now 0.29, own pages included).
//   warps 0-3, 4-7: the softmax of tile 0 and 1; thread t owns row t (TMEM lane
//     t): S to registers, which frees it for the other tile, running max and sum,
//     P in two halves; O is rescaled in place only where a row's max grows by
//     more than 2^8;
//   warps 8, 9: the copies of K and V (two slots each, refilled as soon as both
//     tiles' products have read them); warp 8 owns the tensor memory;
//   warps 10, 11: issue the products of tile 0 and 1, the next stage's QK^T as
//     soon as the other tile's softmax has read S, before PV of this stage.
// (Measured for 448 rows of 64 heads behind 24576 tokens: one thread that issued
// for both tiles spent as long on waits and a full queue as the tensor cores on
// the products, 343 us; a thread a tile with S and P of each tile in the same
// columns, where the next QK^T waits for PV and both tiles fall into step, 307 us;
// columns as they are, QK^T behind PV, 290 us; QK^T before PV 263 us; with two
// waits at once and one commit a product, 243 us: 1.49 PFLOP/s.)
// Every wait is bounded; a CTA that gives up flags SV_DEV_TIMEOUT, lets copies and
// products land and frees its tensor memory.
namespace pfx {
constexpr int kThreads = 384;
constexpr uint32_t kCols = 512, kColP = 128, kColO = 256;
template <int D>
struct Smem {
  static constexpr int kHalf = kTok * 128;            // 64 elements of d of 128 rows
  static constexpr int kTile = D / 64 * kHalf;        // Q of a tile; K or V of a stage
  static constexpr int kBytes = 2 * kTile + 4 * kTile + 1024;
  // one CTA an SM: two would ask for more tensor memory than there is
  static constexpr int kAsk = kBytes > 120 * 1024 ? kBytes : 120 * 1024;
};
}  // namespace pfx

template <int D>
__global__ void __launch_bounds__(pfx::kThreads, 1)
    prefix_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmQ) {
  using S = pfx::Smem<D>;
  constexpr int kHalves = D / 64;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // of a slot: K, V landed; of a tile and slot: S ready (K read), PV done (V read);
  // of a tile: S read by its softmax, P written, every product landed
  __shared__ __align__(8) unsigned long long s_kfull[2], s_vfull[2], s_sfull[2][2], s_odone[2][2],
      s_sread[2], s_pfull[2], s_qfull[2], s_drain[2], s_zero[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_issued[4];
  __shared__ __align__(16) unit::Shared s_unit;
  const int c = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t ring = base + 2 * S::kTile;  // K slots, then V slots
  const int group = a.group;
  // nothing that earlier kernels write is read before griddep_entry()
  if (tid == 0) {
    s_abort = 0;
    unit::init(s_unit);
  }
  if (warp == 8) {
    if (lane == 0) {
      prefetch_map(&tmK);
      prefetch_map(&tmV);
      prefetch_map(&tmQ);
    }
    __syncwarp();
    tc5::tmem_alloc(smem_u32(&s_tmem), pfx::kCols);
    tc5::tmem_relinquish();
  }
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  const uint32_t tmem = s_tmem;
  griddep_entry();
  const int Wp = a.hdr->Wp, Cp = a.hdr->Cp;
  if (c >= Cp) {
    const int W = a.hdr->W, C = a.hdr->C, x_start = a.start[c - Cp];  // (there are a.ctas of them)
    if (c - Cp < C)
      unit_share<D, false>(a, tmK, tmV, tmQ, s_unit, base_ptr, tmem, c - Cp, W, C, x_start, 0);
    if (warp == 8) tc5::tmem_dealloc(tmem, pfx::kCols);
    return;
  }
  PEnd ps = a.pend[c];
  const int s_begin = share_start(c, Wp, Cp);
  int s_end = share_start(c + 1, Wp, Cp), phase = 0;
  bool again = false;  // a list was worked on
  while (s_end > s_begin) {
  const int4 gr = ps.gr;
  const int list = ps.list, g = list % a.Hkv, sp = (gr.z + kStagePages - 1) / kStagePages;
  const int s_list = s_end - 1 - ps.at;  // where the list's start and stages begin
  const int st0 = max(s_begin - s_list - kListStart, 0), n_stage = s_end - s_list - kListStart - st0;
  const int* table = a.tables + (size_t)ps.leader * a.max_blocks + st0 * kStagePages;
  // on to the list before
  s_end = s_list;
  --ps.list;
  ps.at = sp + kListStart - 1;
  if (ps.list < 0 && s_end > s_begin) {  // of the group before that has stages
    do --ps.k;
    while (a.gstage[ps.k] >= s_end);
    ps.gr = a.groups[ps.k];
    ps.leader = a.cu_groups[ps.k];
    ps.list = (ps.gr.y * group + kPrefixRows - 1) / kPrefixRows * a.Hkv - 1;
    ps.at = (ps.gr.z + kStagePages - 1) / kStagePages + kListStart - 1;
  }
  if (n_stage <= 0) continue;  // the share ends in the list's start
  // stage st of this part is its stage (st + turn) mod n_stage: whole lists go on
  // from the stage where the list before ended
  const int turn = n_stage == sp ? phase % sp : 0;
  phase += n_stage;
  const int v0 = list / a.Hkv * kPrefixRows, vrows = min(kPrefixRows, gr.y * group - v0);
  const int ntile = vrows > 128 ? 2 : 1;
  const int np = min(n_stage * kStagePages, gr.z - st0 * kStagePages);
  const size_t slot_id = (size_t)(c + gr.w + list);
  // block of page `lane` of stage st of the part, -1 past its end or outside the cache
  auto page_of = [&](int st) { return (st + turn - (st + turn >= n_stage ? n_stage : 0)) * kStagePages + lane; };
  auto block_of = [&](int st) {
    const int p = page_of(st);
    if (lane >= kStagePages || st >= n_stage || p >= np) return -1;
    const int b = __ldg(table + p);
    return b >= 0 && b < a.num_blocks ? b : -1;
  };

  if (tid == 0) {
    for (int k = 0; k < 4; ++k) s_issued[k] = -1;
    if (again)
      for (int k = 0; k < 2; ++k) {
        for (unsigned long long* b : {&s_kfull[k], &s_vfull[k], &s_sfull[k][0], &s_sfull[k][1], &s_odone[k][0],
                                      &s_odone[k][1], &s_sread[k], &s_pfull[k], &s_qfull[k], &s_drain[k],
                                      &s_zero[k]})
          mbar_inval(smem_u32(b));
      }
    for (int k = 0; k < 2; ++k) {
      mbar_init(smem_u32(&s_kfull[k]), 1);
      mbar_init(smem_u32(&s_vfull[k]), 1);
      for (int j = 0; j < 2; ++j) {
        mbar_init(smem_u32(&s_sfull[k][j]), 1);
        mbar_init(smem_u32(&s_odone[k][j]), 1);
      }
      mbar_init(smem_u32(&s_sread[k]), 128);
      mbar_init(smem_u32(&s_pfull[k]), 128);
      mbar_init(smem_u32(&s_qfull[k]), 128);
      mbar_init(smem_u32(&s_drain[k]), 1);
      mbar_init(smem_u32(&s_zero[k]), 128);
    }
    fence_mbar_init();
  }
  again = true;
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();

  const bool real = tid < vrows;
  if (warp == 8 || warp == 9) {
    // --------------------------------------------------------- producers --
    const int half = warp - 8;  // 0: K, 1: V
    // a slot is free once both tiles' products have read it
    unsigned long long (*freeb)[2] = half ? s_odone : s_sfull;
    unsigned long long* fullb = half ? s_vfull : s_kfull;
    int next = block_of(0);
    for (int st = 0; st < n_stage; ++st) {
      const int slot = st & 1;
      bool go = true;
      if (st >= 2)
        for (int t = 0; t < ntile; ++t)
          go = go && mbar_wait_bounded(smem_u32(&freeb[t][slot]), (uint32_t)(((st - 2) >> 1) & 1));
      if (!__all_sync(0xffffffffu, go)) {
        s_abort = 1;
        break;
      }
      if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s_abort))) break;
      const int b = next;
      next = block_of(st + 1);
      if (half == 0 && lane < kStagePages && b < 0 && page_of(st) < np)
        flag(a.dev_status, SV_DEV_BAD_BLOCK_ID);
      const uint32_t bar = smem_u32(&fullb[slot]);
      const int n = __popc(__ballot_sync(0xffffffffu, b >= 0));
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, (uint32_t)(n * kHalves * 2048));
        s_issued[2 * half + slot] = st;
      }
      __syncwarp();
      if (b >= 0) {
        const uint32_t dst = ring + (2 * half + slot) * S::kTile + lane * 2048;
        const int y = (b * a.Hkv + g) * kBlockSize;
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          tma_load_2d(dst + h * S::kHalf, half ? &tmV : &tmK, 64 * h, y, bar);
      }
    }
  } else if (warp >= 10) {
    // --------------------------------------------------------- MMA issue --
    const int t = warp - 10;
    if (lane == 0 && t < ntile) {
      constexpr uint32_t idesc_qk = tc5::idesc_bf16_f32(128, kTok, false);
      constexpr uint32_t idesc_pv = tc5::idesc_bf16_f32(128, D, true);
      const uint32_t tp = tmem + pfx::kColP + (uint32_t)(t * 64), to = tmem + pfx::kColO + (uint32_t)(t * 128);
      // descriptors of slot 0, first step: the address field counts 16 bytes
      const uint64_t qd = tc5::sw128_desc(base + t * S::kTile, 16, 1024);
      const uint64_t kd = tc5::sw128_desc(ring, 16, 1024);
      const uint64_t vd = tc5::sw128_desc(ring + 2 * S::kTile, S::kHalf, 1024);
      auto qk = [&](int st) -> bool {
        // K has landed, and the softmax has read the S that was there: tile 1's of
        // the stage before (tile 0's, if it is alone), tile 0's of this stage
        const uint32_t kf = smem_u32(&s_kfull[st & 1]), kp = (uint32_t)((st >> 1) & 1);
        const uint32_t sr = smem_u32(&s_sread[t == 1 ? 0 : ntile - 1]);
        if (!(t == 0 && st == 0 ? mbar_wait_bounded(kf, kp)
                                : mbar_wait2_bounded(kf, kp, sr, (uint32_t)((t == 1 ? st : st - 1) & 1))))
          return false;
        tc5::fence_after_sync();
        const uint64_t bd = kd + (uint64_t)((st & 1) * (S::kTile >> 4));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t o = (uint64_t)(((ks >> 2) * S::kHalf + (ks & 3) * 32) >> 4);
          tc5::mma_bf16(tmem, qd + o, bd + o, idesc_qk, ks > 0 ? 1u : 0u);
        }
        tc5::commit(smem_u32(&s_sfull[t][st & 1]));
        return true;
      };
      bool ok = mbar_wait_bounded(smem_u32(&s_qfull[t]), 0u) && qk(0);
      for (int st = 0; st < n_stage && ok; ++st) {
        if (st + 1 < n_stage && !(ok = qk(st + 1))) break;
        // V has landed, P is there
        ok = mbar_wait2_bounded(smem_u32(&s_vfull[st & 1]), (uint32_t)((st >> 1) & 1),
                                smem_u32(&s_pfull[t]), (uint32_t)(st & 1)) &&
             !*reinterpret_cast<volatile int*>(&s_abort);
        if (!ok) break;
        tc5::fence_after_sync();
        const uint64_t bd = vd + (uint64_t)((st & 1) * (S::kTile >> 4));
#pragma unroll
        for (int ks = 0; ks < kTok / 16; ++ks)
          tc5::mma_bf16_ts(to, tp + ks * 8, bd + (uint64_t)(ks * 2048 >> 4), idesc_pv,
                           (st > 0 || ks > 0) ? 1u : 0u);
        tc5::commit(smem_u32(&s_odone[t][st & 1]));
      }
      // The last PV's barrier has its arrival before the next list sets it up anew (of the
      // others the softmax waits for each phase; nothing says that two commits arrive in
      // their order, so the one below does not stand for it).
      if (ok)
        ok = mbar_wait_bounded(smem_u32(&s_odone[t][(n_stage - 1) & 1]), (uint32_t)(((n_stage - 1) >> 1) & 1));
      if (!ok) s_abort = 1;
      // every product of the tile has landed before the CTA moves on
      tc5::commit(smem_u32(&s_drain[t]));
      mbar_wait_bounded(smem_u32(&s_drain[t]), 0);
    }
  } else if (warp < 4 * ntile) {
    // ----------------------------------------------------- softmax, rows --
    const int t = warp >> 2;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base, tp = ts + pfx::kColP + (uint32_t)(t * 64);
    const uint32_t to = tmem + lane_base + pfx::kColO + (uint32_t)(t * 128);
    const float sc = a.scale_log2;
    {
      // Q row, K-major with the 128-byte swizzle, zeros past the list's rows
      const int v = v0 + min(tid, vrows - 1), row = tid & 127;
      const int4* src = reinterpret_cast<const int4*>(
          a.q + ((size_t)a.arows[gr.x + v / group] * a.Hq + g * group + v % group) * D);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const int4 x = real ? __ldg(src + c) : make_int4(0, 0, 0, 0);
        const uint32_t off = (uint32_t)(t * S::kTile + (c >> 3) * S::kHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4));
        *reinterpret_cast<int4*>(base_ptr + off) = x;
      }
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(&s_qfull[t]));
    }
    // pages of the next stage that are there
    auto there = [&](int st) {
      return __ballot_sync(0xffffffffu, block_of(st) >= 0);
    };
    uint32_t pages1 = there(0);
    float m_ref = -INFINITY, l = 0.f;
    // PV of the stage before has landed: O may be rescaled, P overwritten
    auto pv_done = [&](int st) -> bool {
      const bool got = st == 0 || mbar_wait_bounded(smem_u32(&s_odone[t][(st - 1) & 1]), (uint32_t)(((st - 1) >> 1) & 1));
      if (!__all_sync(0xffffffffu, got)) return false;
      tc5::fence_after_sync();
      return true;
    };
    uint32_t zeroed = 0u;  // parity of the incomplete stages so far in each V slot
    bool ok = true;
    for (int st = 0; st < n_stage; ++st) {
      const uint32_t pages = pages1;
      pages1 = there(st + 1);
      const bool got = mbar_wait_bounded(smem_u32(&s_sfull[t][st & 1]), (uint32_t)((st >> 1) & 1));
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      tc5::fence_after_sync();
      uint32_t s[kTok];
      tc5::tmem_ld_x128(ts, s);
      tc5::fence_before_sync();
      mbar_arrive(smem_u32(&s_sread[t]));
      {
        if (pages != 0xffu) {
#pragma unroll
          for (int j = 0; j < kTok; ++j)
            if (!((pages >> (j / 16)) & 1u)) s[j] = __float_as_uint(-INFINITY);
          // rows of V that were not copied may hold anything: tile 0's warps make
          // them zeros, so that their weights of 0 add nothing; tile 1 waits for it
          // (a barrier a slot: tile 0 gets to a slot's next stage after tile 1's PV)
          const int slot = st & 1;
          const bool gv = t == 0 ? mbar_wait_bounded(smem_u32(&s_vfull[slot]), (uint32_t)((st >> 1) & 1))
                                 : mbar_wait_bounded(smem_u32(&s_zero[slot]), (zeroed >> slot) & 1u);
          if (!__all_sync(0xffffffffu, gv)) {
            ok = false;
            break;
          }
          zeroed ^= 1u << slot;
          if (t == 0) {
            uint8_t* vb = base_ptr + (ring - base) + (2 + (st & 1)) * S::kTile;
            for (int x = tid; x < kTok * (D / 8); x += 128) {
              const int row = x / (D / 8), c = x % (D / 8);
              if (!((pages >> (row / 16)) & 1u))
                *reinterpret_cast<int4*>(vb + (c >> 3) * S::kHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4)) =
                    make_int4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            mbar_arrive(smem_u32(&s_zero[slot]));
          }
        }
      }
      float mx4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) mx4[k] = fmaxf(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1]));
#pragma unroll
      for (int j = 8; j < kTok; j += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mx4[k] = fmaxf(fmaxf(mx4[k], __uint_as_float(s[j + 2 * k])), __uint_as_float(s[j + 2 * k + 1]));
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sc;
      const bool grow = mx > m_ref + 8.f;
      if (__any_sync(0xffffffffu, grow)) {
        const float m_new = grow ? mx : m_ref;
        const float alpha = grow ? ex2(m_ref - m_new) : 1.f;  // 0 while m_ref is -inf
        if (!pv_done(st)) {
          ok = false;
          break;
        }
        if (st > 0) {
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t ov[16];
            tc5::tmem_ld_x16(to + c, ov);
#pragma unroll
            for (int k = 0; k < 16; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * alpha);
            tc5::tmem_st_x16(to + c, ov);
          }
        }
        l *= alpha;
        m_ref = m_new;
      }
      const float mb = m_ref == -INFINITY ? 0.f : m_ref;
      const uint64_t sc2 = pair(sc, sc), mb2 = pair(-mb, -mb);
      uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int e = h * 64 + 2 * j;
          const float2 x = unpair(fma2(pair(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2, mb2));
          const float e0 = ex2(x.x), e1 = ex2(x.y);
          sum[j & 3] = add2(sum[j & 3], pair(e0, e1));
          pk[j] = pack_bf16(e0, e1);
        }
        if (h == 0 && !pv_done(st)) {
          ok = false;
          break;
        }
        tc5::tmem_st_x32(tp + h * 32, pk);
      }
      if (!ok) break;
      tc5::fence_before_sync();
      mbar_arrive(smem_u32(&s_pfull[t]));
      const float2 r = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
      l += r.x + r.y;
    }
    if (ok) {
      const bool g3 = mbar_wait_bounded(smem_u32(&s_drain[t]), 0u);
      if (!__all_sync(0xffffffffu, g3)) ok = false;
    }
    if (!ok) {
      s_abort = 1;
    } else {
      tc5::fence_after_sync();
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t ov[32];
        tc5::tmem_ld_x32(to + c, ov);
        if (!real) continue;
        float4* dst = reinterpret_cast<float4*>(a.po) + (slot_id * (D / 4) + c / 4) * kPrefixRows + tid;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          dst[k * kPrefixRows] = make_float4(__uint_as_float(ov[4 * k]), __uint_as_float(ov[4 * k + 1]),
                                             __uint_as_float(ov[4 * k + 2]), __uint_as_float(ov[4 * k + 3]));
      }
      if (real) reinterpret_cast<float2*>(a.pml)[slot_id * kPrefixRows + tid] = make_float2(m_ref, l);
    }
  }

  // every role is done with tensor memory and the ring
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  if (s_abort) break;
  }
  if (s_abort) {
    // copies in flight land before the CTA leaves (bounded waits)
    if (tid == 0) {
      flag(a.dev_status, SV_DEV_TIMEOUT);
      for (int k = 0; k < 4; ++k)
        if (s_issued[k] >= 0)
          mbar_wait_bounded(smem_u32(k < 2 ? &s_kfull[k] : &s_vfull[k - 2]),
                            (uint32_t)((s_issued[k] >> 1) & 1));
    }
    __syncthreads();
  }
  if (warp == 8) tc5::tmem_dealloc(tmem, pfx::kCols);
}

inline Args prefix_args(const sv_paged_kv* kv, const sv_batch* bt, const sv_shared_prefix* sp,
                        int32_t Hq, uint8_t* at, size_t& off) {
  Args a = common_args(kv, bt, Hq, at, off);
  a.n_groups = sp->n_groups;
  a.cu_groups = sp->cu_groups;
  a.prefix_len = sp->prefix_len;
  a.arows = take<int>(at, off, bt->total_rows);
  a.req = take<Req>(at, off, bt->n_req);
  a.groups = take<int4>(at, off, sp->n_groups);
  a.gstage = take<int>(at, off, sp->n_groups + 1);
  a.pend = take<PEnd>(at, off, a.ctas);
  // the row tiles of all groups
  a.plists = (int)std::min(((long)bt->total_rows * a.group / kPrefixRows + sp->n_groups) * a.Hkv, (long)INT32_MAX);
  a.pml = take<float>(at, off, (size_t)(a.plists + a.ctas) * kPrefixRows * 2);
  a.po = take<float>(at, off, (size_t)(a.plists + a.ctas) * kPrefixRows * kv->head_dim);
  return a;
}

template <int D>
sv_status prefix_attend(const Args& a, const void* k, const void* v, cudaStream_t stream) {
  CUtensorMap tmK, tmV, tmQ;
  if (!attn::make_map(&tmK, k, a.num_blocks, a.Hkv, D) || !attn::make_map(&tmV, v, a.num_blocks, a.Hkv, D) ||
      !make_q_map(&tmQ, a, D))
    return SV_ERR_CUDA;
  static PerDevice set;
  if (smem_limit_once(set, prefix_kernel<D>, pfx::Smem<D>::kAsk) != cudaSuccess) return SV_ERR_CUDA;
  if (sv::launch(prefix_plan_kernel, 1, kPlanThreads, sizeof(PlanSmem), stream, a) != cudaSuccess ||
      sv::launch(prefix_kernel<D>, a.ctas, pfx::kThreads, pfx::Smem<D>::kAsk, stream, a, tmK, tmV, tmQ) !=
          cudaSuccess ||
      launch_merge<D, false>(a, stream) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}

inline sv_status check_prefix(const sv_paged_kv* kv, const sv_batch* bt, const sv_shared_prefix* sp,
                              int32_t Hq) {
  const sv_status st = check(kv, bt, Hq);
  if (st != SV_OK) return st;
  if (!sp || sp->n_groups < 0) return SV_ERR_INVALID_ARGUMENT;
  if (bt->n_req == 0) return SV_OK;
  if (sp->n_groups < 1 || sp->n_groups > bt->n_req) return SV_ERR_INVALID_ARGUMENT;
  return SV_OK;
}

}  // namespace pu
}  // namespace sv

using namespace sv;

extern "C" size_t sv_prefix_attend_workspace(const sv_batch* bt, const sv_paged_kv* kv,
                                             const sv_shared_prefix* prefix, int32_t n_q_heads) {
  if (pu::check_prefix(kv, bt, prefix, n_q_heads) != SV_OK) return 0;
  size_t off = 0;
  const pu::Args a = pu::prefix_args(kv, bt, prefix, n_q_heads, nullptr, off);
  return pu::counts_fit((long)a.tiles_cap * a.Hkv, a.max_blocks) && pu::counts_fit(a.plists, a.max_blocks) ? off : 0;
}

extern "C" sv_status sv_prefix_attend(const sv_paged_kv* kv, const sv_batch* bt,
                                      const sv_shared_prefix* prefix, const void* q,
                                      int32_t n_q_heads, float softmax_scale, void* out, void* ws,
                                      size_t ws_bytes, int32_t* dev_status, void* stream) {
  SV_TRACE("sv_prefix_attend");
  const sv_status st = pu::check_prefix(kv, bt, prefix, n_q_heads);
  if (st != SV_OK) return st;
  if (bt->n_req == 0 || bt->total_rows == 0) return SV_OK;
  if (!q || !out || !ws || !prefix->cu_groups || !prefix->prefix_len) return SV_ERR_INVALID_ARGUMENT;
  if (((uintptr_t)q | (uintptr_t)out) & 15) return SV_ERR_INVALID_ARGUMENT;
  if ((uintptr_t)ws & 255) return SV_ERR_INVALID_ARGUMENT;
  if (!(softmax_scale > 0.f)) return SV_ERR_INVALID_ARGUMENT;
  size_t need = 0;
  pu::Args a = pu::prefix_args(kv, bt, prefix, n_q_heads, static_cast<uint8_t*>(ws), need);
  if (!pu::counts_fit((long)a.tiles_cap * a.Hkv, a.max_blocks) || !pu::counts_fit(a.plists, a.max_blocks))
    return SV_ERR_UNSUPPORTED_SHAPE;
  if (pu::overlap(q, out, bt, n_q_heads, kv->head_dim)) return SV_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need) return SV_ERR_WORKSPACE_TOO_SMALL;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.dev_status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return kv->head_dim == 128 ? pu::prefix_attend<128>(a, kv->k_cache, kv->v_cache, s)
                             : pu::prefix_attend<64>(a, kv->k_cache, kv->v_cache, s);
}
