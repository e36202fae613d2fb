// sv_page_units.cuh — attention of tiles of draft rows over lists of pages, and
// the merge of its parts: what sv_page_attend and sv_prefix_attend share.
//
// A tile is up to 64 virtual rows (query rows x GQA group) of one request.  For
// every (tile, KV head) there is a list of cache pages: complete pages of the
// context first, of which each row sees all or none of the slots (a bit of the
// page's row mask), then the tail, the pages from the one that holds slot ctx
// on, whose slots a row sees up to the context's end and where its ancestors
// lie.  The lists are cut into stages of four pages; all stages of a call, in
// (tile, KV head) order, are dealt out evenly to C CTAs, so that a CTA's share
// is one run of stages over one or several lists.  A list that lies in one
// CTA's share is written to the output there; the parts of the others meet in
// merge_kernel.  Part c of list x has the slot c + x: the runs and the lists
// both only move on, so no two parts share a slot and C + lists slots do.
#pragma once

#include <algorithm>

#include "sv_attend_common.cuh"
#include "sv_internal.cuh"

namespace sv {
namespace pu {

constexpr int kTB = 64;         // tokens of a stage (four pages)
constexpr int kStages = 3;      // TMA ring depth
constexpr int kThreads = 128;   // four warps
constexpr int kTileRows = 64;   // virtual rows of a tile
constexpr int kIds = 8;         // stages whose block ids and masks wait in shared memory

struct __align__(16) Tile {
  int i, cu, ctx, r0;      // request, its first packed row, context, first local row
  int nr, rows, first, ncomp;  // rows of the tile and of the request; first table
                               // entry and complete pages of its list (prefix calls)
  int nent, arow, grp, pad;    // entries of the list; the tile's first row among all
                               // active rows, its group (prefix calls)
};

struct Header {
  int T;       // tiles
  int W;       // stages of all lists
  int C;       // CTAs that share them (at most W)
  int ticket;
  int np_pages;  // pages of a prefix unit
  int units;     // prefix units
  int pad[58];
};

struct Args {
  sv_batch bt;
  int num_blocks, Hkv, max_blocks;
  const int32_t* tables;
  const int32_t* lens;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int Hq, group;
  int rt;             // rows of a tile
  int tile_vr;        // virtual rows of a part: rt * group, at most what a request has
  int tiles_cap, ctas;
  float scale_log2;
  int32_t* dev_status;
  Header* hdr;
  Tile* tiles;
  int* off;           // [lists + 1] first stage of each list
  int* start;         // [ctas] list of each CTA's first stage
  float* ml;          // [slots][tile_vr][2]
  float* o;           // [slots][tile_vr][D]
  // page lists (sv_page_attend)
  const int32_t* pages;
  int n_keep;
  int cap;            // entries of a list, a multiple of four
  int* blk;           // [lists][cap]
  unsigned long long* mask;  // [lists][cap]
  int* cnt;           // [lists][2] complete pages, all entries
  // shared prefix (sv_prefix_attend)
  int n_groups;
  const int32_t* cu_groups;
  const int32_t* prefix_len;
  int* arows;         // [total_rows] packed rows of the active rows
  int* aoff;          // [n_req + 1] first active row of each request
  int4* groups;       // [n_groups] first active row, active rows, pages, first unit
  int4* punits;       // group, KV head, row tile, split
  int punits_cap;
  float* pml;
  float* po;
};

// Stage s of W belongs to the CTA c of C <= W with start(c) <= s < start(c + 1).
__device__ __forceinline__ int share_start(int c, int W, int C) { return (int)((long)c * W / C); }
__device__ __forceinline__ int share_of(int s, int W, int C) { return (int)((((long)s + 1) * C - 1) / W); }

// ------------------------------------------------------------------ lists --

// The list of each CTA's first stage, from the lists' first stages off[0 ..
// lists] (global memory, written by this block before a barrier).
__device__ __forceinline__ void deal_stages(const Args& a, int lists, int W) {
  const int C = min(a.ctas, W);
  for (int c = threadIdx.x; c < C; c += blockDim.x) {
    const int s = share_start(c, W, C);
    int lo = 0, hi = lists - 1;
    while (lo < hi) {  // the last list that starts at or before s; empty lists are passed over
      const int mid = (lo + hi + 1) >> 1;
      if (a.off[mid] <= s) lo = mid; else hi = mid - 1;
    }
    a.start[c] = lo;
  }
  if (threadIdx.x == 0) {
    a.hdr->W = W;
    a.hdr->C = C;
  }
}

// A request's window, parents and length; false (and reported) if it cannot be
// attended.
__device__ __forceinline__ bool request_rows(const Args& a, int i, Window& w, int& ctx) {
  w = window_of(a.bt, i);
  ctx = a.lens[i];
  bool bad = false;
  if (w.ok)
    for (int j0 = 0; j0 < w.rows; j0 += 8) {  // eight loads in flight, then the checks
      int pp[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) pp[k] = j0 + k < w.rows ? a.bt.parent[w.cu + j0 + k] : 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = j0 + k;
        if (j < w.rows) bad |= (j == 0) ? (pp[k] != -1) : (pp[k] < 0 || pp[k] >= j);
      }
    }
  if (!w.ok) flag(a.dev_status, SV_DEV_BAD_WINDOW);
  if (bad) flag(a.dev_status, SV_DEV_BAD_PARENT);
  if (!w.ok || bad) return false;
  if (ctx < 0 || (long)ctx + w.rows > (long)a.max_blocks * kBlockSize) {
    flag(a.dev_status, SV_DEV_BAD_LENGTH);
    return false;
  }
  return true;
}

// Exclusive scan over the block's threads of v, on top of *carry (shared),
// which moves on by the total.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = *carry;
  for (int w = 0; w < warp; ++w) before += s_warp[w];
  __syncthreads();
  if (threadIdx.x == blockDim.x - 1) *carry = before + x;
  __syncthreads();
  return before + x - v;
}

// ------------------------------------------------------------------ units --

template <int D>
struct Frag {
  float o[D / 8][4];
  float m_a, m_b, l_a, l_b;
};

// NT * 8 tokens from stage row s0 on for this warp's two rows; bit t of vis_*
// says whether the row sees token t of the stage.
template <int D, int NT>
__device__ __forceinline__ void slice_compute(Frag<D>& f, const uint32_t (&qf)[D / 16][4],
                                              uint32_t kbase, uint32_t vbase, int s0,
                                              unsigned long long vis_a, unsigned long long vis_b,
                                              float scale_log2, int lane) {
  using SL = attn::StageLayout<D>;
  const int tq = lane & 3;
  float sc[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ks += 2) {
      const int trow = s0 + nt * 8 + (lane & 7);
      const int chunk = 2 * ks + (lane >> 3);
      uint32_t r[4];
      ldsm_x4(r, kbase + SL::off(trow, chunk));
      mma16816(sc[nt], qf[ks], r[0], r[1]);
      mma16816(sc[nt], qf[ks + 1], r[2], r[3]);
    }
  }
  constexpr uint32_t kAll = NT == 4 ? 0xffffffffu : (1u << (NT * 8 & 31)) - 1u;
  const uint32_t va = (uint32_t)(vis_a >> s0) & kAll, vb = (uint32_t)(vis_b >> s0) & kAll;
  const bool need_mask = __any_sync(0xffffffffu, va != kAll || vb != kAll);
  float mx_a = -INFINITY, mx_b = -INFINITY;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = sc[nt][e] * scale_log2;
      if (need_mask && !(((e < 2 ? va : vb) >> (nt * 8 + 2 * tq + (e & 1))) & 1u)) v = -INFINITY;
      sc[nt][e] = v;
      if (e < 2) mx_a = fmaxf(mx_a, v); else mx_b = fmaxf(mx_b, v);
    }
  }
  mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 1));
  mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 2));
  mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 1));
  mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 2));
  const float nm_a = fmaxf(f.m_a, mx_a), nm_b = fmaxf(f.m_b, mx_b);
  const float base_a = nm_a == -INFINITY ? 0.f : nm_a;
  const float base_b = nm_b == -INFINITY ? 0.f : nm_b;
  const float al_a = ex2(f.m_a - base_a), al_b = ex2(f.m_b - base_b);
  f.m_a = nm_a;
  f.m_b = nm_b;
  float ps_a = 0.f, ps_b = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    sc[nt][0] = ex2(sc[nt][0] - base_a);
    sc[nt][1] = ex2(sc[nt][1] - base_a);
    sc[nt][2] = ex2(sc[nt][2] - base_b);
    sc[nt][3] = ex2(sc[nt][3] - base_b);
    ps_a += sc[nt][0] + sc[nt][1];
    ps_b += sc[nt][2] + sc[nt][3];
  }
  f.l_a = f.l_a * al_a + ps_a;
  f.l_b = f.l_b * al_b + ps_b;
  // a row's factor is 1 once its maximum has settled: O is then left alone
  if (__any_sync(0xffffffffu, al_a != 1.f || al_b != 1.f)) {
#pragma unroll
    for (int dn = 0; dn < D / 8; ++dn) {
      f.o[dn][0] *= al_a;
      f.o[dn][1] *= al_a;
      f.o[dn][2] *= al_b;
      f.o[dn][3] *= al_b;
    }
  }
  // P is rounded to bf16 for the tensor cores (2^-9 of each weight at most, in
  // the sum of many; the normaliser keeps fp32)
#pragma unroll
  for (int kk = 0; kk < NT / 2; ++kk) {
    uint32_t pa[4];
    pa[0] = pack_bf16(sc[2 * kk][0], sc[2 * kk][1]);
    pa[1] = pack_bf16(sc[2 * kk][2], sc[2 * kk][3]);
    pa[2] = pack_bf16(sc[2 * kk + 1][0], sc[2 * kk + 1][1]);
    pa[3] = pack_bf16(sc[2 * kk + 1][2], sc[2 * kk + 1][3]);
#pragma unroll
    for (int dn = 0; dn < D / 8; dn += 2) {
      const int trow = s0 + 16 * kk + (lane & 7) + ((lane >> 3) & 1) * 8;
      const int chunk = dn + (lane >> 4);
      uint32_t r[4];
      ldsm_x4_t(r, vbase + SL::off(trow, chunk));
      mma16816(f.o[dn], pa, r[0], r[1]);
      mma16816(f.o[dn + 1], pa, r[2], r[3]);
    }
  }
}

// Slots m0 .. m0 + 15 relative to the context's end that a row sees: those
// before it, and its ancestors-or-self (bits of mk1:mk0).
__device__ __forceinline__ uint32_t tail_visible(int m0, unsigned long long mk0,
                                                 unsigned long long mk1) {
  if (m0 >= 128) return 0u;
  if (m0 >= 64) return (uint32_t)(mk1 >> (m0 - 64)) & 0xffffu;
  if (m0 >= 0) return (uint32_t)((mk0 >> m0) | (m0 ? mk1 << (64 - m0) : 0ull)) & 0xffffu;
  if (m0 <= -16) return 0xffffu;
  return ((uint32_t)(mk0 << -m0) | ((1u << -m0) - 1u)) & 0xffffu;
}

template <int D, bool SPARSE>
__global__ void __launch_bounds__(kThreads, 2)
    unit_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV) {
  griddep_entry();
  using SL = attn::StageLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int s_par[kMaxRows];
  __shared__ unsigned long long s_anc[kTileRows][2];
  __shared__ int s_id[kIds][4];
  __shared__ unsigned long long s_row[kIds][4];  // rows that see the page
  __shared__ __align__(8) unsigned long long s_full[kStages];
  __shared__ int s_abort;
  const int W = a.hdr->W, C = a.hdr->C;
  const int c = blockIdx.x;
  if (c >= C) return;
  const int s_end = share_start(c + 1, W, C);
  int s_at = share_start(c, W, C);
  int x = a.start[c];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
  if (tid == 0) {
    s_abort = 0;
    for (int k = 0; k < kStages; ++k) mbar_init(smem_u32(&s_full[k]), 4);
    fence_mbar_init();
  }
  int it = 0;  // stages issued to the ring by earlier lists of this share
  for (; s_at < s_end; ++x) {
    const int off0 = a.off[x], off1 = a.off[x + 1];
    const int e_first = 4 * (s_at - off0);  // first entry of the list in this share
    const int n_stage = min(s_end, off1) - s_at;
    if (n_stage <= 0) continue;  // an empty list
    const bool whole = s_at == off0 && s_at + n_stage == off1;
    s_at += n_stage;
    const int g = x % a.Hkv;
    const Tile tl = a.tiles[x / a.Hkv];
    const int ncomp = SPARSE ? a.cnt[2 * x] : tl.ncomp;
    const int nent = SPARSE ? a.cnt[2 * x + 1] : tl.nent;
    const int group = a.group, Mu = tl.nr * group;
    const int tail0 = tl.ctx / kBlockSize * kBlockSize - tl.ctx;  // first tail slot
    const int lim = tl.r0 + tl.nr;  // staged rows that may be attended
    const bool tail = min(nent, e_first + 4 * n_stage) > ncomp;

    // block ids (and row masks) of stage st, entry p: thread p loads them
    auto entry_id = [&](int st) {
      const int e = e_first + 4 * st + (tid & 3);
      int b = -1;
      if (st < n_stage && e < nent) {
        b = SPARSE ? __ldg(a.blk + (size_t)x * a.cap + e)
                   : __ldg(a.tables + (size_t)tl.i * a.max_blocks + tl.first + e);
        if (b < 0 || b >= a.num_blocks) {
          flag(a.dev_status, SV_DEV_BAD_BLOCK_ID);
          b = -1;
        }
      }
      return b;
    };
    auto entry_rows = [&](int st) {
      const int e = e_first + 4 * st + (tid & 3);
      if (!SPARSE || st >= n_stage || e >= ncomp) return ~0ull;
      return __ldg(a.mask + (size_t)x * a.cap + e);
    };
    __syncthreads();  // the list before is done with the shared arrays
    if (tid < 4 * kStages) {
      s_id[tid >> 2][tid & 3] = entry_id(tid >> 2);
      s_row[tid >> 2][tid & 3] = entry_rows(tid >> 2);
    }
    if (tail)
      for (int j = tid; j < tl.rows; j += kThreads) s_par[j] = a.bt.parent[tl.cu + j];
    fence_proxy_async_smem();  // the ring held parts of the list before
    __syncthreads();
    // lane 0 of warp p copies page p of a stage and announces its bytes
    auto issue = [&](int st) {
      if (lane != 0 || st >= n_stage) return;
      const int slot = (it + st) % kStages;
      const uint32_t bar = smem_u32(&s_full[slot]);
      const uint32_t kdst = ring + slot * SL::kStageBytes;
      const int b = s_id[st % kIds][warp];
      mbar_arrive_expect_tx(bar, b >= 0 ? 2u * SL::kHalves * SL::kBoxBytes : 0u);
      if (b < 0) return;
      const int y = (b * a.Hkv + g) * kBlockSize;
#pragma unroll
      for (int h = 0; h < SL::kHalves; ++h) {
        const uint32_t o = (uint32_t)((warp * SL::kHalves + h) * SL::kBoxBytes);
        tma_load_2d(kdst + o, &tmK, 64 * h, y, bar);
        tma_load_2d(kdst + SL::kTensorBytes + o, &tmV, 64 * h, y, bar);
      }
    };
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st) issue(st);
    if (tail) {
      for (int t = tid; t < tl.nr; t += kThreads) {
        unsigned long long lo = 0ull, hi = 0ull;
        int m = tl.r0 + t;
        for (int steps = 0; m >= 0 && steps <= kMaxRows; ++steps) {  // parents were checked
          if (m < 64) lo |= 1ull << m; else hi |= 1ull << (m - 64);
          m = s_par[m];
        }
        s_anc[t][0] = lo;
        s_anc[t][1] = hi;
      }
      __syncthreads();
    }

    // m-tile mt and token slice ts of TS of this warp
    const int MT = (Mu + 15) >> 4;
    const int TS = MT == 1 ? 4 : MT == 2 ? 2 : 1;
    const int mt = MT == 3 ? warp : warp % MT;
    const int ts = MT == 3 ? 0 : warp / MT;
    const bool active = mt < MT;
    const int vl_a = mt * 16 + gq, vl_b = vl_a + 8;
    const bool real_a = active && vl_a < Mu, real_b = active && vl_b < Mu;
    const int lr_a = real_a ? vl_a / group : 0, lr_b = real_b ? vl_b / group : 0;
    const size_t qrow_a = (size_t)(tl.cu + tl.r0 + lr_a) * a.Hq + g * group + (real_a ? vl_a % group : 0);
    const size_t qrow_b = (size_t)(tl.cu + tl.r0 + lr_b) * a.Hq + g * group + (real_b ? vl_b % group : 0);
    unsigned long long ka0 = 0, ka1 = 0, kb0 = 0, kb1 = 0;
    if (tail) {
      ka0 = s_anc[lr_a][0]; ka1 = s_anc[lr_a][1];
      kb0 = s_anc[lr_b][0]; kb1 = s_anc[lr_b][1];
    }
    uint32_t qf[D / 16][4];
    {
      const uint32_t* qa = reinterpret_cast<const uint32_t*>(a.q + qrow_a * D);
      const uint32_t* qb = reinterpret_cast<const uint32_t*>(a.q + qrow_b * D);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qf[ks][0] = real_a ? __ldg(qa + ks * 8 + tq) : 0u;
        qf[ks][1] = real_b ? __ldg(qb + ks * 8 + tq) : 0u;
        qf[ks][2] = real_a ? __ldg(qa + ks * 8 + 4 + tq) : 0u;
        qf[ks][3] = real_b ? __ldg(qb + ks * 8 + 4 + tq) : 0u;
      }
    }
    Frag<D> f;
#pragma unroll
    for (int dn = 0; dn < D / 8; ++dn) f.o[dn][0] = f.o[dn][1] = f.o[dn][2] = f.o[dn][3] = 0.f;
    f.m_a = f.m_b = -INFINITY;
    f.l_a = f.l_b = 0.f;

    int issued = min(kStages - 1, n_stage), abort_at = -1;
    for (int st = 0; st < n_stage; ++st) {
      issue(st + kStages - 1);
      if (st + kStages - 1 < n_stage) issued = st + kStages;
      // ids of the stage after those in flight: loaded now, stored at the end
      int id_next = -1;
      unsigned long long row_next = ~0ull;
      if (tid < 4) {
        id_next = entry_id(st + kStages);
        row_next = entry_rows(st + kStages);
      }
      const int slot = (it + st) % kStages;
      unsigned long long vis_a = 0ull, vis_b = 0ull;
      int valid = 0;  // sixteens of slots of the stage that hold something, 5 bits each
      const int e0 = e_first + 4 * st;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        unsigned long long wa = 0ull, wb = 0ull;
        int n = 0;
        if (s_id[st % kIds][p] >= 0) {
          if (e0 + p < ncomp) {
            n = 16;
            wa = wb = 0xffffull;
            if (SPARSE) {
              const unsigned long long rows = s_row[st % kIds][p];
              wa = (rows >> lr_a) & 1ull ? 0xffffull : 0ull;
              wb = (rows >> lr_b) & 1ull ? 0xffffull : 0ull;
            }
          } else {
            const int m0 = tail0 + (e0 + p - ncomp) * kBlockSize;
            n = max(0, min(16, lim - m0));
            wa = tail_visible(m0, ka0, ka1);
            wb = tail_visible(m0, kb0, kb1);
          }
        }
        vis_a |= wa << (16 * p);
        vis_b |= wb << (16 * p);
        valid |= n << (8 * p);
      }
      // rows of no query take what their neighbours need no mask for
      if (!real_a) vis_a = ~0ull;
      if (!real_b) vis_b = ~0ull;
      // a wait that gives up marks the CTA; all threads stop after the barrier
      if (!mbar_wait_bounded(smem_u32(&s_full[slot]), (uint32_t)(((it + st) / kStages) & 1))) s_abort = 1;
      const uint32_t kbase = ring + slot * SL::kStageBytes;
      const uint32_t vbase = kbase + SL::kTensorBytes;
      if (valid != 0x10101010) {
        // slots that nothing was written to may hold anything: V = 0 there, so
        // that their weights of 0 add nothing
        for (int y = tid; y < kTB * (D / 8); y += kThreads) {
          const int t = y / (D / 8), ch = y % (D / 8);
          if ((t & 15) >= ((valid >> (8 * (t >> 4))) & 31))
            *reinterpret_cast<int4*>(ring_ptr + (vbase - ring) + SL::off(t, ch)) = make_int4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // before later copies into the slot
        __syncthreads();
      }
      if (active) {
        if (TS == 4) {
          slice_compute<D, 2>(f, qf, kbase, vbase, ts * 16, vis_a, vis_b, a.scale_log2, lane);
        } else if (TS == 2) {
          slice_compute<D, 4>(f, qf, kbase, vbase, ts * 32, vis_a, vis_b, a.scale_log2, lane);
        } else {
          slice_compute<D, 4>(f, qf, kbase, vbase, 0, vis_a, vis_b, a.scale_log2, lane);
          slice_compute<D, 4>(f, qf, kbase, vbase, 32, vis_a, vis_b, a.scale_log2, lane);
        }
      }
      if (tid < 4) {
        s_id[(st + kStages) % kIds][tid] = id_next;
        s_row[(st + kStages) % kIds][tid] = row_next;
      }
      __syncthreads();  // the slot is free
      if (s_abort) {
        abort_at = st;
        if (tid == 0) flag(a.dev_status, SV_DEV_TIMEOUT);
        break;
      }
    }
    if (abort_at >= 0) {
      // copies in flight land before the CTA leaves (bounded waits)
      if (tid == 0)
        for (int st = abort_at; st < issued; ++st)
          mbar_wait_bounded(smem_u32(&s_full[(it + st) % kStages]),
                            (uint32_t)(((it + st) / kStages) & 1));
      __syncthreads();
      return;
    }
    it += n_stage;

    // warps that shared an m-tile meet through shared memory (the ring is idle)
    float* xch = reinterpret_cast<float*>(ring_ptr);
    constexpr int kFragFloats = D / 2 + 4;
    if (TS > 1) {
      if (active && ts > 0) {
        float* dst = xch + ((size_t)warp * kFragFloats) * 32 + lane;
#pragma unroll
        for (int dn = 0; dn < D / 8; ++dn)
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[(dn * 4 + e) * 32] = f.o[dn][e];
        dst[(D / 2 + 0) * 32] = f.m_a;
        dst[(D / 2 + 1) * 32] = f.m_b;
        dst[(D / 2 + 2) * 32] = f.l_a;
        dst[(D / 2 + 3) * 32] = f.l_b;
      }
      __syncthreads();
      if (active && ts == 0) {
        for (int t = 1; t < TS; ++t) {
          const float* src = xch + ((size_t)(warp + t * MT) * kFragFloats) * 32 + lane;
          const float m2a = src[(D / 2 + 0) * 32], m2b = src[(D / 2 + 1) * 32];
          const float l2a = src[(D / 2 + 2) * 32], l2b = src[(D / 2 + 3) * 32];
          const float na = fmaxf(f.m_a, m2a), nb = fmaxf(f.m_b, m2b);
          const float ba = na == -INFINITY ? 0.f : na, bb = nb == -INFINITY ? 0.f : nb;
          const float s1a = exp2f(f.m_a - ba), s2a = exp2f(m2a - ba);
          const float s1b = exp2f(f.m_b - bb), s2b = exp2f(m2b - bb);
#pragma unroll
          for (int dn = 0; dn < D / 8; ++dn) {
            f.o[dn][0] = f.o[dn][0] * s1a + src[(dn * 4 + 0) * 32] * s2a;
            f.o[dn][1] = f.o[dn][1] * s1a + src[(dn * 4 + 1) * 32] * s2a;
            f.o[dn][2] = f.o[dn][2] * s1b + src[(dn * 4 + 2) * 32] * s2b;
            f.o[dn][3] = f.o[dn][3] * s1b + src[(dn * 4 + 3) * 32] * s2b;
          }
          f.l_a = f.l_a * s1a + l2a * s2a;
          f.l_b = f.l_b * s1b + l2b * s2b;
          f.m_a = na;
          f.m_b = nb;
        }
      }
    }
    if (!active || ts != 0) continue;
    f.l_a += __shfl_xor_sync(0xffffffffu, f.l_a, 1);
    f.l_a += __shfl_xor_sync(0xffffffffu, f.l_a, 2);
    f.l_b += __shfl_xor_sync(0xffffffffu, f.l_b, 1);
    f.l_b += __shfl_xor_sync(0xffffffffu, f.l_b, 2);
    if (whole && (SPARSE || a.groups[tl.grp].z == 0)) {
      const float inv_a = f.l_a > 0.f ? 1.f / f.l_a : 0.f;
      const float inv_b = f.l_b > 0.f ? 1.f / f.l_b : 0.f;
      uint32_t* oa = reinterpret_cast<uint32_t*>(a.out + qrow_a * D);
      uint32_t* ob = reinterpret_cast<uint32_t*>(a.out + qrow_b * D);
#pragma unroll
      for (int dn = 0; dn < D / 8; ++dn) {
        if (real_a) oa[dn * 4 + tq] = pack_bf16(f.o[dn][0] * inv_a, f.o[dn][1] * inv_a);
        if (real_b) ob[dn * 4 + tq] = pack_bf16(f.o[dn][2] * inv_b, f.o[dn][3] * inv_b);
      }
      continue;
    }
    const size_t part = (size_t)(c + x) * a.tile_vr;
    if (tq == 0) {
      if (real_a) reinterpret_cast<float2*>(a.ml)[part + vl_a] = make_float2(f.m_a, f.l_a);
      if (real_b) reinterpret_cast<float2*>(a.ml)[part + vl_b] = make_float2(f.m_b, f.l_b);
    }
#pragma unroll
    for (int dn = 0; dn < D / 8; ++dn) {
      if (real_a)
        *reinterpret_cast<float2*>(a.o + (part + vl_a) * D + dn * 8 + 2 * tq) = make_float2(f.o[dn][0], f.o[dn][1]);
      if (real_b)
        *reinterpret_cast<float2*>(a.o + (part + vl_b) * D + dn * 8 + 2 * tq) = make_float2(f.o[dn][2], f.o[dn][3]);
    }
  }
}

// ------------------------------------------------------------------ merge --

// One CTA a list: the parts of its rows -- of the CTAs that shared it and, in
// prefix calls, of the prefix units of the row's group -- in one online pass.
// SL neighbouring lanes share four columns of a row, lane s of them the parts
// s, s + SL, ..., kLoads of them in flight at once; shuffles join the lanes.
constexpr int kMergeThreads = 256;
constexpr int kPrefixRows = 256;  // virtual rows of a prefix unit
template <int D, bool SPARSE>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ Args a) {
  griddep_entry();
  constexpr int kQuads = D / 4, kLoads = 8;
  const int x = blockIdx.x;
  const int T = a.hdr->T, W = a.hdr->W, C = a.hdr->C;
  if (x >= T * a.Hkv) return;
  const int off0 = a.off[x], off1 = a.off[x + 1];
  if (off0 == off1) return;
  const Tile tl = a.tiles[x / a.Hkv];
  const int g = x % a.Hkv, group = a.group;
  const int c0 = share_of(off0, W, C), ns = share_of(off1 - 1, W, C) - c0 + 1;
  int np = 0;
  int4 grp = make_int4(0, 0, 0, 0);
  if (!SPARSE) {
    grp = a.groups[tl.grp];
    np = grp.z > 0 ? (grp.z + a.hdr->np_pages - 1) / a.hdr->np_pages : 0;
  }
  const int n = ns + np;
  if (n == 1) return;  // written by the CTA that had it whole
  int SL = 1;
  while (SL < 32 && SL * kLoads < n) SL <<= 1;
  const int items = tl.nr * group * kQuads * SL;
  for (int x0 = 0; x0 < items; x0 += kMergeThreads) {
    const int y = x0 + threadIdx.x;
    const bool live = y < items;
    const int sl = y % SL, qd = y / SL;
    const int vr = qd / kQuads, c4 = qd % kQuads;
    float Mx = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
      size_t prow = 0;
      if (!SPARSE && np > 0) {
        const int v = (tl.arow - grp.x) * group + vr;  // among the group's virtual rows
        prow = ((size_t)(grp.w + (v / kPrefixRows * a.Hkv + g) * np)) * kPrefixRows + v % kPrefixRows;
      }
      for (int k0 = sl; k0 < n; k0 += kLoads * SL) {
        float2 ml2[kLoads];
        float4 o4[kLoads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int s = min(k0 + k * SL, n - 1);
          const float* ml = a.ml;
          const float* o = a.o;
          size_t row = (size_t)(c0 + s + x) * a.tile_vr + vr;
          if (!SPARSE && s >= ns) {
            ml = a.pml;
            o = a.po;
            row = prow + (size_t)(s - ns) * kPrefixRows;
          }
          ml2[k] = __ldcg(reinterpret_cast<const float2*>(ml) + row);
          o4[k] = __ldcg(reinterpret_cast<const float4*>(o + row * D) + c4);
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const float nm = fmaxf(Mx, ml2[k].x);
          if (k0 + k * SL >= n || nm == -INFINITY) continue;
          const float s_old = exp2f(Mx - nm), s_new = exp2f(ml2[k].x - nm);
          L = L * s_old + ml2[k].y * s_new;
          acc.x = acc.x * s_old + o4[k].x * s_new;
          acc.y = acc.y * s_old + o4[k].y * s_new;
          acc.z = acc.z * s_old + o4[k].z * s_new;
          acc.w = acc.w * s_old + o4[k].w * s_new;
          Mx = nm;
        }
      }
    }
    for (int o = SL >> 1; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, Mx, o);
      const float l2 = __shfl_xor_sync(0xffffffffu, L, o);
      float4 a2;
      a2.x = __shfl_xor_sync(0xffffffffu, acc.x, o);
      a2.y = __shfl_xor_sync(0xffffffffu, acc.y, o);
      a2.z = __shfl_xor_sync(0xffffffffu, acc.z, o);
      a2.w = __shfl_xor_sync(0xffffffffu, acc.w, o);
      const float nm = fmaxf(Mx, m2);
      if (nm != -INFINITY) {
        const float s_old = exp2f(Mx - nm), s_new = exp2f(m2 - nm);
        L = L * s_old + l2 * s_new;
        acc.x = acc.x * s_old + a2.x * s_new;
        acc.y = acc.y * s_old + a2.y * s_new;
        acc.z = acc.z * s_old + a2.z * s_new;
        acc.w = acc.w * s_old + a2.w * s_new;
        Mx = nm;
      }
    }
    if (!live || sl != 0) continue;
    const float inv = L > 0.f ? 1.f / L : 0.f;
    const size_t row = (size_t)(tl.cu + tl.r0 + vr / group) * a.Hq + g * group + vr % group;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * D + c4 * 4);
    dst[0] = pack_bf16(acc.x * inv, acc.y * inv);
    dst[1] = pack_bf16(acc.z * inv, acc.w * inv);
  }
}

// ------------------------------------------------------------- host side --

inline sv_status check(const sv_paged_kv* kv, const sv_batch* bt, int32_t Hq) {
  if (!kv || !bt) return SV_ERR_INVALID_ARGUMENT;
  if (bt->n_req < 0 || bt->total_rows < 0 || bt->max_rows_per_req < 1) return SV_ERR_INVALID_ARGUMENT;
  if (bt->n_req > 0 && (!bt->cu_rows || !bt->parent)) return SV_ERR_INVALID_ARGUMENT;
  if (bt->max_rows_per_req > kMaxRows) return SV_ERR_UNSUPPORTED_SHAPE;
  if (kv->block_size != kBlockSize) return SV_ERR_UNSUPPORTED_SHAPE;
  if (kv->head_dim != 64 && kv->head_dim != 128) return SV_ERR_UNSUPPORTED_SHAPE;
  if (kv->n_kv_heads < 1 || Hq < 1 || Hq % kv->n_kv_heads != 0) return SV_ERR_INVALID_ARGUMENT;
  if (Hq / kv->n_kv_heads > 16) return SV_ERR_UNSUPPORTED_SHAPE;
  if (kv->num_blocks < 0 || kv->max_blocks_per_req < 0) return SV_ERR_INVALID_ARGUMENT;
  // rows of the cache are counted in 32 bits by the copies
  if ((long)kv->num_blocks * kv->n_kv_heads >= (1L << 31) / kBlockSize) return SV_ERR_UNSUPPORTED_SHAPE;
  if (bt->n_req > 0 && (!kv->k_cache || !kv->v_cache || !kv->block_tables || !kv->cache_lens))
    return SV_ERR_INVALID_ARGUMENT;
  if (((uintptr_t)kv->k_cache | (uintptr_t)kv->v_cache) & 15) return SV_ERR_INVALID_ARGUMENT;
  return SV_OK;
}

// The part of the arguments and of the workspace that both calls have; `at`
// is the workspace's address or null, `off` moves on by what is taken.
template <class T>
inline T* take(uint8_t* at, size_t& off, size_t n) {
  T* p = reinterpret_cast<T*>(at + off);
  off += align256(sizeof(T) * n);
  return p;
}

inline Args common_args(const sv_paged_kv* kv, const sv_batch* bt, int32_t Hq, uint8_t* at, size_t& off) {
  Args a{};
  a.bt = *bt;
  a.num_blocks = kv->num_blocks;
  a.Hkv = kv->n_kv_heads;
  a.max_blocks = kv->max_blocks_per_req;
  a.tables = kv->block_tables;
  a.lens = kv->cache_lens;
  a.Hq = Hq;
  a.group = Hq / kv->n_kv_heads;
  const int most = std::max(1, std::min(bt->max_rows_per_req, bt->total_rows));
  a.rt = std::min(kTileRows / a.group, most);
  a.tile_vr = a.rt * a.group;
  // ceil(rows / rt) tiles a request
  a.tiles_cap = bt->total_rows / a.rt + bt->n_req;
  a.ctas = 2 * sizing_sms();
  const size_t lists = (size_t)a.tiles_cap * a.Hkv, slots = lists + a.ctas;
  a.hdr = take<Header>(at, off, 1);
  a.tiles = take<Tile>(at, off, a.tiles_cap);
  a.off = take<int>(at, off, lists + 1);
  a.start = take<int>(at, off, a.ctas);
  a.ml = take<float>(at, off, slots * a.tile_vr * 2);
  a.o = take<float>(at, off, slots * a.tile_vr * kv->head_dim);
  return a;
}

template <int D, bool SPARSE>
inline sv_status launch_units(const Args& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                              cudaStream_t stream) {
  constexpr size_t smem = (size_t)kStages * attn::StageLayout<D>::kStageBytes + 1024;
  static PerDevice set;
  if (smem_limit_once(set, unit_kernel<D, SPARSE>, smem) != cudaSuccess) return SV_ERR_CUDA;
  if (sv::launch(unit_kernel<D, SPARSE>, a.ctas, kThreads, smem, stream, a, tmK, tmV) != cudaSuccess)
    return SV_ERR_CUDA;
  if (sv::launch(merge_kernel<D, SPARSE>, a.tiles_cap * a.Hkv, kMergeThreads, 0, stream, a) !=
      cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}

}  // namespace pu
}  // namespace sv
