// sv_page_units.cuh — attention of tiles of draft rows over lists of pages, and
// the merge of its parts: what sv_page_attend and sv_prefix_attend share.
//
// A tile is up to 128 virtual rows (query rows x GQA group) of one request.  For
// every (tile, KV head) there is a list of cache pages: complete pages of the
// context first, of which each row sees all or none of the slots, then the tail,
// the pages from the one that holds slot ctx on, whose slots a row sees up to the
// context's end and where its ancestors lie.  The lists are cut into stages of
// eight pages; all stages of a call, in (tile, KV head) order, are dealt out
// evenly to C CTAs, so that a CTA's share is one run of stages over one or several
// lists.  A list that lies in one CTA's share is written to the output there; the
// parts of the others meet in merge_kernel.  Part c of list x has the slot c + x:
// the runs and the lists both only move on, so no two parts share a slot and C +
// lists slots do.
#pragma once

#include <algorithm>

#include "sv_attend_common.cuh"
#include "sv_internal.cuh"
#include "sv_tcgen05.cuh"

namespace sv {
namespace pu {

constexpr int kTok = 128;        // tokens of a stage
constexpr int kStagePages = 8;   // pages of a stage
constexpr int kTileRows = 128;   // virtual rows of a tile
// Beginning a prefix list (its Q, the first copies, nothing yet to overlap with, and
// writing out the one before) takes a CTA as long as about four stages: a list
// counts so many more, before its own, when the stages are dealt out (30 draft trees
// behind three prompts: 57.5 us without, 51.7 with two, 50.6 with four and with six).
constexpr int kListStart = 4;

struct __align__(16) Tile {
  int i, cu, ctx, r0;      // request, its first packed row, context, first local row
  int nr, rows, first, ncomp;  // rows of the tile and of the request; first table
                               // entry and complete pages of its list (prefix calls)
  int nent, arow, grp, pre;    // entries of the list; the tile's first row among those
                               // of the prefix lists, its group, and the entries that
                               // are read from its group's first request (prefix calls)
};

struct Header {
  int T;       // tiles
  int W;       // stages of all lists
  int C;       // CTAs that share them (at most W)
  int Wp;      // stages of all prefix lists, their starts included
  int Cp;      // CTAs that share them
  int pad[59];
};

// The last stage of a CTA's share of the prefix stages: the group's record, the
// group, the list among the group's, the stage behind the list's start (kListStart
// counted, at), the group's first request.
struct __align__(16) PEnd {
  int4 gr;
  int k, list, at, leader;
};

struct Req;
struct Args {
  sv_batch bt;
  int num_blocks, Hkv, max_blocks;
  const int32_t* tables;
  const int32_t* lens;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int Hq, group, dim;
  int rt;             // rows of a tile
  int tile_vr;        // virtual rows of a part: rt * group, at most what a request has
  int tiles_cap, ctas;
  float scale_log2;
  int32_t* dev_status;
  Header* hdr;
  Tile* tiles;
  int* off;           // [lists + 1] first stage of each list
  int* start;         // [ctas] list of each CTA's first stage (prefix calls)
  float* ml;          // [slots][tile_vr][2]
  float* o;           // [slots][D / 4][tile_vr][4]: neighbouring rows in neighbouring lanes
  // page lists (sv_page_attend)
  const int32_t* pages;
  int n_keep;
  int cap;            // entries of a list, a multiple of 32
  int* blk;           // [lists][cap]
  uint32_t* see;      // [lists][rt][cap / 32] pages a row sees, a bit an entry
  int* cnt;           // [lists][2] complete pages, all entries
  // shared prefix (sv_prefix_attend)
  int n_groups;
  const int32_t* cu_groups;
  const int32_t* prefix_len;
  int* arows;         // [total_rows] packed rows of the prefix lists' rows
  Req* req;           // [n_req]
  int4* groups;       // [n_groups] first of these rows, rows, pages, first prefix list
  int* gstage;        // [n_groups + 1] first stage of each group's prefix lists, starts included
  PEnd* pend;         // [ctas]
  int plists;         // prefix lists at most: 256-row tiles x KV heads
  float* pml;         // [plists + ctas][kPrefixRows][2]
  float* po;          // [plists + ctas][D / 4][kPrefixRows][4]
};

// Stage s of W belongs to the CTA c of C <= W with start(c) <= s < start(c + 1).
__device__ __forceinline__ int share_start(int c, int W, int C) { return (int)((long)c * W / C); }
__device__ __forceinline__ int share_of(int s, int W, int C) { return (int)((((long)s + 1) * C - 1) / W); }

// ------------------------------------------------------------------ lists --

// What the plan of a prefix call keeps of a request.
struct Req {
  int cu, rows, b, e;  // e = b: left out
  int ctx, first, grp, tile;  // prefix pages, group, first tile
  int stage, arow;     // first stage of the request's lists of one KV head, its first row
                       // among those of the prefix lists
  int pre, pad;        // pages of the prefix that its own lists read
};

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

// Bits m0 .. m0 + 31 of what a row sees behind the context's end: ones before it
// (m0 < 0), then its ancestors-or-self (bits of mk1:mk0).
__device__ __forceinline__ uint32_t tail_visible(int m0, unsigned long long mk0,
                                                 unsigned long long mk1) {
  if (m0 >= 128) return 0u;
  if (m0 <= -32) return 0xffffffffu;
  if (m0 < 0) return ((uint32_t)mk0 << -m0) | ((1u << -m0) - 1u);
  const int w = m0 >> 5;
  const uint32_t a[5] = {(uint32_t)mk0, (uint32_t)(mk0 >> 32), (uint32_t)mk1, (uint32_t)(mk1 >> 32), 0u};
  uint32_t lo = a[3], hi = 0u;
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (w == k) {
      lo = a[k];
      hi = a[k + 1];
    }
  return __funnelshift_r(lo, hi, m0 & 31);
}

// One CTA an SM works through its share as one sequence of stages, n = 0, 1, ...
// over all its lists (L = 0, 1, ...), so that the copies and products of a list
// begin while the one before is still being finished:
//   warps 0-3, 4-7: the softmax of every other list; thread t owns row t of the tile
//     (TMEM lane t): S to registers, what the row does not see masked, running max
//     and sum, P (bf16) back over S; O is rescaled only where a row's max grows by
//     more than 2^8; at a list's end O to the output or to a part, while the other
//     warps begin the next list (one set of warps for all lists: 57 us for the own
//     pages of 64 requests, five stages a list, where two take 51);
//   warp 8: the copies of Q and K, warp 9 of V (two slots each);
//   warp 10: one thread issues S = Q K^T (128 x 128) and O += P V (128 x D) as
//     tcgen05.mma, QK^T of the next stage before PV of this one;
//   warp 11: reads the lists ahead (a ring of kLists records in shared memory).
// Tensor memory: S of two stages in columns 0 .. 255, O of two lists in 256 .. 511.
// Bound by the pages' bytes where all SMs do this: a stage of 64 KB (head_dim 128) is
// 1.5 us of one SM's share of HBM, its products 0.7 us, its softmax 0.6 us (the own
// choices of 48 chains: 97 us, 6.25 TB/s); an SM among others that do not read as
// much takes 1.1 us.
// Every wait is bounded; a CTA that gives up flags SV_DEV_TIMEOUT, lets copies and
// products land and frees its tensor memory.
namespace unit {
constexpr int kThreads = 384;
constexpr int kLists = 4;
constexpr uint32_t kCols = 512, kColO = 256;
template <int D>
struct Smem {
  static constexpr int kHalf = kTok * 128;         // 64 elements of d of 128 rows
  static constexpr int kTile = D / 64 * kHalf;     // Q of a list; K or V of a stage
  static constexpr int kBytes = 6 * kTile + 1024;  // two each
  // one CTA an SM: two would ask for more tensor memory than there is
  static constexpr int kAsk = kBytes > 120 * 1024 ? kBytes : 120 * 1024;
};
// A list's part in the share.
struct Rec {
  int x, g, n_stage, e_first;   // n_stage 0: the end
  int i, row0, nr, ctx;         // request; first packed row of the tile, its rows
  int first, ncomp, nent, r0;   // table entry and entries of the list; first local row
  int whole, bad, pre, lead;    // all of the list; some block outside the cache; entries
                                // read from another request
};
struct Shared {
  Rec rec[kLists];
  ulonglong2 anc[kLists][kTileRows];  // ancestors-or-self of the tile's rows
  int ids[kLists][kStagePages];       // blocks of a list's first stage
  int par[kMaxRows];
  // records there / free; K, V landed, PV done (V read), P written of a stage's slot;
  // S ready (K read) of a set of softmax warps and slot: a set counts its own stages
  // there, as a wait for a phase must not begin before the one before is over; Q
  // landed, O complete, O read of a list
  unsigned long long lfull[kLists], lfree[kLists], kfull[2], vfull[2], sfull[2][2], odone[2], pfull[2],
      qfull[2], olast[2], ofree[2], drain;
  int abort;
  int issued[6];  // phases begun of kfull, vfull, qfull
};

// By one thread, before the CTA's first barrier.
__device__ __forceinline__ void init(Shared& sh) {
  sh.abort = 0;
  for (int k = 0; k < 6; ++k) sh.issued[k] = 0;
  for (int k = 0; k < kLists; ++k) {
    mbar_init(smem_u32(&sh.lfull[k]), 1);
    mbar_init(smem_u32(&sh.lfree[k]), 11);  // eight softmax warps, two producers, the issuing thread
  }
  for (int k = 0; k < 2; ++k) {
    mbar_init(smem_u32(&sh.kfull[k]), 1);
    mbar_init(smem_u32(&sh.vfull[k]), 1);
    mbar_init(smem_u32(&sh.sfull[k][0]), 1);
    mbar_init(smem_u32(&sh.sfull[k][1]), 1);
    mbar_init(smem_u32(&sh.odone[k]), 1);
    mbar_init(smem_u32(&sh.pfull[k]), 128);
    mbar_init(smem_u32(&sh.qfull[k]), 1);
    mbar_init(smem_u32(&sh.olast[k]), 1);
    mbar_init(smem_u32(&sh.ofree[k]), 128);
  }
  mbar_init(smem_u32(&sh.drain), 1);
  fence_mbar_init();
}
}  // namespace unit

// The work of CTA c of C: its share of W stages, the first of them of list x_start,
// whose stages begin at off_start.  Q of two lists, then K slots and V slots from
// `base` on (1024-byte aligned).
template <int D, bool SPARSE>
__device__ __forceinline__ void unit_share(const Args& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                           const CUtensorMap& tmQ, unit::Shared& sh, uint8_t* base_ptr,
                                           uint32_t tmem, int c, int W, int C, int x_start, int off_start) {
  using unit::kLists;
  using unit::Rec;
  using S = unit::Smem<D>;
  constexpr int kHalves = D / 64;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = smem_u32(base_ptr), ring = base + 2 * S::kTile;
  auto gone = [&] { return *reinterpret_cast<volatile int*>(&sh.abort) != 0; };
  // the record of list L, by a whole warp (or by one thread); null: gave up
  auto list_at = [&](int L) -> const Rec* {
    if (!mbar_wait_bounded(smem_u32(&sh.lfull[L % kLists]), (uint32_t)((L / kLists) & 1))) return nullptr;
    return &sh.rec[L % kLists];
  };
  auto list_done = [&](int L) { mbar_arrive(smem_u32(&sh.lfree[L % kLists])); };
  // block of entry e of a list, -1 past its end or outside the cache
  auto block_of = [&](const Rec& r, int e) {
    if (e >= r.nent) return -1;
    const int b = SPARSE ? __ldg(a.blk + (size_t)r.x * a.cap + e)
                         : __ldg(a.tables + (size_t)(e < r.pre ? r.lead : r.i) * a.max_blocks + r.first + e);
    return b >= 0 && b < a.num_blocks ? b : -1;
  };

  if (warp == 11) {
    // ------------------------------------------------------- lists ahead --
    const int s_end = share_start(c + 1, W, C);
    int s_at = share_start(c, W, C), x = x_start, off1 = off_start, L = 0;
    bool ok = true;
    for (;; ++x) {
      Rec r{};
      if (s_at < s_end) {
        const Tile tl = a.tiles[x / a.Hkv];
        r.ncomp = SPARSE ? a.cnt[2 * x] : tl.ncomp;
        r.nent = SPARSE ? a.cnt[2 * x + 1] : tl.nent;
        const int off0 = SPARSE ? off1 : a.off[x];
        off1 = off0 + (r.nent + kStagePages - 1) / kStagePages;
        r.n_stage = min(s_end, off1) - s_at;
        if (r.n_stage <= 0) continue;  // an empty list
        r.x = x;
        r.g = x % a.Hkv;
        r.e_first = kStagePages * (s_at - off0);
        r.whole = s_at == off0 && s_at + r.n_stage == off1;
        r.i = tl.i;
        r.row0 = tl.cu + tl.r0;
        r.nr = tl.nr;
        r.ctx = tl.ctx;
        r.first = tl.first;
        r.r0 = tl.r0;
        r.pre = SPARSE ? 0 : tl.pre;
        r.lead = r.pre > 0 ? a.cu_groups[tl.grp] : 0;
        s_at += r.n_stage;
        const int e_end = min(r.nent, r.e_first + r.n_stage * kStagePages);
        const bool tail = e_end > r.ncomp;  // the tail is among it
        int par[kMaxRows / 32];
#pragma unroll
        for (int k = 0; k < kMaxRows / 32; ++k)
          par[k] = tail && lane + 32 * k < tl.rows ? a.bt.parent[tl.cu + lane + 32 * k] : -1;
        const int b0 = block_of(r, r.e_first + lane);
        if (L >= kLists &&
            !mbar_wait_bounded(smem_u32(&sh.lfree[L % kLists]), (uint32_t)((L / kLists - 1) & 1)))
          ok = false;
        if (!__all_sync(0xffffffffu, ok) || __any_sync(0xffffffffu, gone())) {
          ok = false;
          break;
        }
        if (lane < kStagePages) sh.ids[L % kLists][lane] = b0;
        bool bad = r.e_first + lane < e_end && b0 < 0;
        for (int e = r.e_first + 32 + lane; e < e_end; e += 32) bad |= block_of(r, e) < 0;
        if (bad) flag(a.dev_status, SV_DEV_BAD_BLOCK_ID);
        r.bad = __any_sync(0xffffffffu, bad);
        if (tail) {
#pragma unroll
          for (int k = 0; k < kMaxRows / 32; ++k) sh.par[lane + 32 * k] = par[k];
          __syncwarp();
          for (int t = lane; t < tl.nr; t += 32) {
            unsigned long long lo = 0ull, hi = 0ull;
            int m = tl.r0 + t;
            for (int steps = 0; m >= 0 && steps <= kMaxRows; ++steps) {  // parents were checked
              if (m < 64) lo |= 1ull << m; else hi |= 1ull << (m - 64);
              m = sh.par[m];
            }
            sh.anc[L % kLists][t] = make_ulonglong2(lo, hi);
          }
        }
      } else if (L >= kLists &&
                 !mbar_wait_bounded(smem_u32(&sh.lfree[L % kLists]), (uint32_t)((L / kLists - 1) & 1))) {
        ok = false;
        break;
      }
      __syncwarp();
      if (lane == 0) {
        sh.rec[L % kLists] = r;
        mbar_arrive(smem_u32(&sh.lfull[L % kLists]));
      }
      ++L;
      if (r.n_stage == 0) break;
    }
    if (!ok) sh.abort = 1;
  } else if (warp == 8 || warp == 9) {
    // --------------------------------------------------------- producers --
    const bool isV = warp == 9;
    bool ok = true;
    int n = 0;
    uint32_t held = 0u, phase = 0u, count = 0u;  // bits of the slots, of the sets and slots
    for (int L = 0; ok; ++L) {
      const Rec* rp = list_at(L);
      if (!__all_sync(0xffffffffu, rp != nullptr)) {
        ok = false;
        break;
      }
      const Rec r = *rp;
      if (r.n_stage == 0) break;
      int b = lane < kStagePages ? sh.ids[L % kLists][lane] : -1;
      __syncwarp();
      if (lane == 0) list_done(L);
      for (int st = 0; st < r.n_stage; ++st, ++n) {
        // blocks of the next stage on their way
        const int e1 = r.e_first + (st + 1) * kStagePages + lane;
        const int b1 = st + 1 < r.n_stage && lane < kStagePages ? block_of(r, e1) : -1;
        const int slot = n & 1;
        // the slot is free once the products of stage n - 2 have read it
        bool go = n < 2 || (isV ? mbar_wait_bounded(smem_u32(&sh.odone[slot]), (uint32_t)(((n - 2) >> 1) & 1))
                                : mbar_wait_bounded(smem_u32(&sh.sfull[(held >> slot) & 1][slot]),
                                                    (phase >> slot) & 1u));
        // the set and phase that will free the slot again
        const int set = L & 1;
        held = (held & ~(1u << slot)) | (uint32_t)set << slot;
        phase = (phase & ~(1u << slot)) | ((count >> (2 * set + slot)) & 1u) << slot;
        count ^= 1u << (2 * set + slot);
        if (!__all_sync(0xffffffffu, go) || __any_sync(0xffffffffu, gone())) {
          ok = false;
          break;
        }
        if (!isV && st == 0 && lane == 0) {
          // Q of the list: its buffer's last reader was a list before stage n - 2
          const uint32_t bar = smem_u32(&sh.qfull[L & 1]), dst = base + (L & 1) * S::kTile;
          mbar_arrive_expect_tx(bar, (uint32_t)(kHalves * a.rt * a.group * 128));
          sh.issued[4 + (L & 1)] += 1;
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            tma_load_3d(dst + h * S::kHalf, &tmQ, 64 * h, r.g * a.group, r.row0, bar);
        }
        const uint32_t bar = smem_u32(isV ? &sh.vfull[slot] : &sh.kfull[slot]);
        const int cnt = __popc(__ballot_sync(0xffffffffu, b >= 0));
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, (uint32_t)(cnt * kHalves * 2048));
          sh.issued[2 * isV + slot] += 1;
        }
        __syncwarp();
        if (b >= 0) {
          const uint32_t dst = ring + (2 * isV + slot) * S::kTile + lane * 2048;
          const int y = (b * a.Hkv + r.g) * kBlockSize;
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            tma_load_2d(dst + h * S::kHalf, isV ? &tmV : &tmK, 64 * h, y, bar);
        }
        b = b1;
      }
    }
    if (!ok) sh.abort = 1;
  } else if (warp == 10) {
    // --------------------------------------------------------- MMA issue --
    if (lane == 0) {
      constexpr uint32_t idesc_qk = tc5::idesc_bf16_f32(128, kTok, false);
      constexpr uint32_t idesc_pv = tc5::idesc_bf16_f32(128, D, true);
      const uint64_t qd = tc5::sw128_desc(base, 16, 1024);
      const uint64_t kd = tc5::sw128_desc(ring, 16, 1024);
      const uint64_t vd = tc5::sw128_desc(ring + 2 * S::kTile, S::kHalf, 1024);
      bool ok = true;
      // the lists of the next QK^T and of the next PV: PV follows a stage behind
      int Lq = 0, sq = 0, nq = 0, n_q = 0, Lp = 0, sp = 0, np = 0;
      const Rec* rq = list_at(0);
      ok = rq != nullptr;
      if (ok) nq = np = rq->n_stage;
      auto qk = [&]() -> bool {  // stage n_q
        const int n = n_q, slot = n & 1;
        if (sq == 0 && !mbar_wait_bounded(smem_u32(&sh.qfull[Lq & 1]), (uint32_t)((Lq >> 1) & 1))) return false;
        // K has landed; PV of stage n - 2 is through with its P, where S goes
        const uint32_t kf = smem_u32(&sh.kfull[slot]), kp = (uint32_t)((n >> 1) & 1);
        if (!(n < 2 ? mbar_wait_bounded(kf, kp)
                    : mbar_wait2_bounded(kf, kp, smem_u32(&sh.odone[slot]), (uint32_t)(((n - 2) >> 1) & 1))))
          return false;
        tc5::fence_after_sync();
        const uint64_t ad = qd + (uint64_t)((Lq & 1) * (S::kTile >> 4));
        const uint64_t bd = kd + (uint64_t)(slot * (S::kTile >> 4));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t o = (uint64_t)(((ks >> 2) * S::kHalf + (ks & 3) * 32) >> 4);
          tc5::mma_bf16(tmem + (uint32_t)(slot * kTok), ad + o, bd + o, idesc_qk, ks > 0 ? 1u : 0u);
        }
        tc5::commit(smem_u32(&sh.sfull[Lq & 1][slot]));
        ++n_q;
        if (++sq == nq) {
          ++Lq;
          sq = 0;
          const Rec* r = list_at(Lq);
          if (!r) return false;
          nq = r->n_stage;
        }
        return true;
      };
      if (ok && nq > 0) ok = qk();
      for (int n = 0; ok && np > 0; ++n) {
        if (nq > 0 && !(ok = qk())) break;
        const int slot = n & 1;
        // V has landed, P is there; at a list's first stage O of the list two before
        // has been read
        ok = mbar_wait2_bounded(smem_u32(&sh.vfull[slot]), (uint32_t)((n >> 1) & 1),
                                smem_u32(&sh.pfull[slot]), (uint32_t)((n >> 1) & 1)) &&
             (sp > 0 || Lp < 2 ||
              mbar_wait_bounded(smem_u32(&sh.ofree[Lp & 1]), (uint32_t)(((Lp >> 1) - 1) & 1))) &&
             !gone();
        if (!ok) break;
        tc5::fence_after_sync();
        const uint64_t bd = vd + (uint64_t)(slot * (S::kTile >> 4));
        const uint32_t to = tmem + unit::kColO + (uint32_t)((Lp & 1) * 128);
#pragma unroll
        for (int ks = 0; ks < kTok / 16; ++ks)
          tc5::mma_bf16_ts(to, tmem + (uint32_t)(slot * kTok) + ks * 8, bd + (uint64_t)(ks * 2048 >> 4),
                           idesc_pv, (sp > 0 || ks > 0) ? 1u : 0u);
        tc5::commit(smem_u32(&sh.odone[slot]));
        if (++sp == np) {
          // (the next lists may run on before this one's O is read: a barrier of its own)
          tc5::commit(smem_u32(&sh.olast[Lp & 1]));
          list_done(Lp);
          ++Lp;
          sp = 0;
          const Rec* r = list_at(Lp);
          if (!r) {
            ok = false;
            break;
          }
          np = r->n_stage;
        }
      }
      if (!ok) sh.abort = 1;
      // every product has landed before the CTA moves on
      tc5::commit(smem_u32(&sh.drain));
      mbar_wait_bounded(smem_u32(&sh.drain), 0);
    }
  } else {
    // ----------------------------------------------------- softmax, rows --
    const int row_t = tid & 127;  // this thread's row
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float sc = a.scale_log2;
    const uint64_t sc2 = pair(sc, sc);
    const int group = a.group;
    bool ok = true;
    int n = 0;
    uint32_t count = 0u;  // parity of this set's stages so far in each slot
    for (int L = 0; ok; ++L) {
      const Rec* rp = list_at(L);
      if (!__all_sync(0xffffffffu, rp != nullptr)) {
        ok = false;
        break;
      }
      const Rec r = *rp;
      if (r.n_stage == 0) break;
      if ((L & 1) != warp >> 2) {  // the other warps' list
        __syncwarp();
        if (lane == 0) list_done(L);
        n += r.n_stage;
        continue;
      }
      const int vrows = r.nr * group;
      const bool real = row_t < vrows;
      const int lr = real ? row_t / group : 0, head = r.g * group + (real ? row_t % group : 0);
      const bool some = (warp & 3) * 32 < vrows;  // rows in this warp at all
      ulonglong2 anc = make_ulonglong2(0ull, 0ull);
      const int e_end = min(r.nent, r.e_first + r.n_stage * kStagePages);
      if (e_end > r.ncomp) anc = sh.anc[L % kLists][lr];
      __syncwarp();
      if (lane == 0) list_done(L);
      const uint32_t* see = SPARSE ? a.see + ((size_t)r.x * a.rt + lr) * (a.cap / 32) : nullptr;
      uint32_t bits = SPARSE ? __ldg(see + (r.e_first >> 5)) : 0u, bits1 = 0u;
      const int tail0 = r.ctx / kBlockSize * kBlockSize - r.ctx;  // first tail slot
      const uint32_t to = tmem + lane_base + unit::kColO + (uint32_t)((L & 1) * 128);
      float m_ref = -INFINITY, l = 0.f;
      for (int st = 0; st < r.n_stage; ++st, ++n) {
        const int slot = n & 1;
        const int e0 = r.e_first + st * kStagePages;
        if (SPARSE && (e0 & 31) == 0 && st > 0) bits = bits1;
        if (SPARSE && (e0 & 31) == 24 && st + 1 < r.n_stage) bits1 = __ldg(see + (e0 >> 5) + 1);
        const uint32_t vis = SPARSE ? bits >> (e0 & 31) : 0xffu;  // pages of the stage the row sees
        const bool got = mbar_wait_bounded(smem_u32(&sh.sfull[L & 1][slot]), (count >> slot) & 1u);
        count ^= 1u << slot;
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        const bool odd = r.bad || e0 + kStagePages > r.ncomp;  // not all complete and there
        uint32_t there = 0xffu;
        if (odd) {
          there = e0 + kStagePages <= r.nent ? 0xffu : (1u << (r.nent - e0)) - 1u;
          if (r.bad) there &= __ballot_sync(0xffffffffu, lane < kStagePages && block_of(r, e0 + lane) >= 0);
        }
        tc5::fence_after_sync();
        if (some) {
          const uint32_t ts = tmem + lane_base + (uint32_t)(slot * kTok);
          // In an odd stage: the tokens of quarter q (32 tokens) that the row sees.
          const int m0 = tail0 + (e0 - r.ncomp) * kBlockSize;  // slot of the stage's first token
          auto seen = [&](int q) {
            const uint32_t w = tail_visible(m0 + 32 * q, anc.x, anc.y);
            uint32_t x = 0u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int p = 2 * q + h;
              const uint32_t whole = (vis >> p) & 1u ? 0xffffu : 0u;
              const uint32_t y = e0 + p < r.ncomp ? whole : (w >> (16 * h)) & 0xffffu;
              x |= ((there >> p) & 1u ? y : 0u) << (16 * h);
            }
            return x;
          };
          // S is read twice, for the maxima and for P: its 128 values would not leave
          // two sets of softmax warps registers enough
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if (!odd) {
            uint32_t s[2][32];
            tc5::tmem_ld_x32_begin(ts, s[0]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              tc5::tmem_ld_wait(s[q & 1]);
              if (q < 3) tc5::tmem_ld_x32_begin(ts + 32 * (q + 1), s[(q + 1) & 1]);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float m2[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const uint32_t* v = s[q & 1] + 16 * h + 8 * k;
                  m2[k] = fmaxf(fmaxf(fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1])), __uint_as_float(v[2])),
                                fmaxf(__uint_as_float(v[3]), __uint_as_float(v[4])));
                  m2[k] = fmaxf(fmaxf(m2[k], __uint_as_float(v[5])), fmaxf(__uint_as_float(v[6]), __uint_as_float(v[7])));
                }
                if ((vis >> (2 * q + h)) & 1u) mx4[q] = fmaxf(fmaxf(mx4[q], m2[0]), m2[1]);
              }
            }
          } else {
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t s[32];
              tc5::tmem_ld_x32(ts + 32 * q, s);
              const uint32_t w = seen(q);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (w & (1u << k)) mx4[k & 3] = fmaxf(mx4[k & 3], __uint_as_float(s[k]));
            }
          }
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sc;
          const bool grow = mx > m_ref + 8.f;
          if (__any_sync(0xffffffffu, grow)) {
            const float m_new = grow ? mx : m_ref;
            const float alpha = grow ? ex2(m_ref - m_new) : 1.f;  // 0 while m_ref is -inf
            if (st > 0) {
              const bool g2 = mbar_wait_bounded(smem_u32(&sh.odone[(n - 1) & 1]), (uint32_t)(((n - 1) >> 1) & 1));
              if (!__all_sync(0xffffffffu, g2)) {
                ok = false;
                break;
              }
              tc5::fence_after_sync();
#pragma unroll 1
              for (int k = 0; k < D; k += 16) {
                uint32_t ov[16];
                tc5::tmem_ld_x16(to + k, ov);
#pragma unroll
                for (int j = 0; j < 16; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
                tc5::tmem_st_x16(to + k, ov);
              }
            }
            l *= alpha;
            m_ref = m_new;
          }
          const float mb = m_ref == -INFINITY ? 0.f : m_ref;
          uint64_t sum[4] = {0, 0, 0, 0};
          // P is rounded to bf16 for the tensor cores (2^-8 of each weight at most, in
          // a sum of many; the normaliser keeps fp32); a page that the row does not
          // see gets its -inf with the maximum's subtraction.  P of a quarter goes
          // over columns of S that have been read.
          auto weights = [&](const uint32_t (&s)[32], int q, float off0, float off1) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float off = k < 8 ? off0 : off1;
              const float2 x = unpair(fma2(pair(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), sc2,
                                           pair(off, off)));
              const float w0 = ex2(x.x), w1 = ex2(x.y);
              sum[k & 3] = add2(sum[k & 3], pair(w0, w1));
              pk[k] = pack_bf16(w0, w1);
            }
            tc5::tmem_st_x16(ts + 16 * q, pk);
          };
          if (!odd) {
            uint32_t s[2][32];
            tc5::tmem_ld_x32_begin(ts, s[0]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              tc5::tmem_ld_wait(s[q & 1]);
              if (q < 3) tc5::tmem_ld_x32_begin(ts + 32 * (q + 1), s[(q + 1) & 1]);
              weights(s[q & 1], q, (vis >> (2 * q)) & 1u ? -mb : -INFINITY, (vis >> (2 * q + 1)) & 1u ? -mb : -INFINITY);
            }
          } else {
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t s[32];
              tc5::tmem_ld_x32(ts + 32 * q, s);
              const uint32_t w = seen(q);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(w & (1u << k))) s[k] = __float_as_uint(-INFINITY);
              weights(s, q, -mb, -mb);
            }
          }
          const float2 z = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
          l += z.x + z.y;
        }
        if (odd) {
          // rows of V that nothing was written to may hold anything: zeros, so that
          // their weights of 0 add nothing
          const bool gv = mbar_wait_bounded(smem_u32(&sh.vfull[slot]), (uint32_t)((n >> 1) & 1));
          if (!__all_sync(0xffffffffu, gv)) {
            ok = false;
            break;
          }
          uint8_t* vb = base_ptr + (ring - base) + (2 + slot) * S::kTile;
          auto zero = [&](int t0, int t1) {  // rows t0 .. t1 - 1 of V
#pragma unroll 1
            for (int y = row_t; y < (t1 - t0) * (D / 8); y += 128) {
              const int t = t0 + y / (D / 8), ch = y % (D / 8);
              *reinterpret_cast<int4*>(vb + (ch >> 3) * S::kHalf + t * 128 + (((ch & 7) ^ (t & 7)) << 4)) =
                  make_int4(0, 0, 0, 0);
            }
          };
          // behind the last staged slot, and (where a block is missing) whole pages
          zero(min(kTok, max(0, (r.ncomp - e0) * kBlockSize + r.r0 + r.nr - tail0)), kTok);
#pragma unroll 1
          for (int p = 0; p < (r.bad ? kStagePages : 0); ++p)
            if (!((there >> p) & 1u)) zero(16 * p, 16 * p + 16);
          fence_proxy_async_smem();
        }
        tc5::fence_before_sync();
        mbar_arrive(smem_u32(&sh.pfull[slot]));
      }
      if (!ok) break;
      // the list's last PV has landed: O, normalised, to the output or to a part
      const bool last = mbar_wait_bounded(smem_u32(&sh.olast[L & 1]), (uint32_t)((L >> 1) & 1));
      if (!__all_sync(0xffffffffu, last)) {
        ok = false;
        break;
      }
      tc5::fence_after_sync();
      if (some) {
        const bool out = r.whole && (SPARSE || r.first == 0);
        const size_t row = (size_t)(r.row0 + lr) * a.Hq + head, part = (size_t)(c + r.x);
        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
          uint32_t ov[32];
          tc5::tmem_ld_x32(to + k, ov);
          if (!real) continue;
          if (out) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + k);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int z = 0; z < 4; ++z)
                w[z] = pack_bf16(__uint_as_float(ov[8 * j + 2 * z]) * inv, __uint_as_float(ov[8 * j + 2 * z + 1]) * inv);
              dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(a.o) + (part * (D / 4) + k / 4) * a.tile_vr + row_t;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              dst[(size_t)j * a.tile_vr] =
                  make_float4(__uint_as_float(ov[4 * j]), __uint_as_float(ov[4 * j + 1]),
                              __uint_as_float(ov[4 * j + 2]), __uint_as_float(ov[4 * j + 3]));
          }
        }
        if (real && !out) reinterpret_cast<float2*>(a.ml)[part * a.tile_vr + row_t] = make_float2(m_ref, l);
      }
      tc5::fence_before_sync();
      mbar_arrive(smem_u32(&sh.ofree[L & 1]));
    }
    if (!ok) sh.abort = 1;
  }

  // every role is done with tensor memory and the ring
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  if (sh.abort) {
    // copies in flight land before the CTA leaves (bounded waits)
    if (tid == 0) {
      flag(a.dev_status, SV_DEV_TIMEOUT);
      for (int k = 0; k < 6; ++k)
        if (sh.issued[k] > 0)
          mbar_wait_bounded(smem_u32(k < 2 ? &sh.kfull[k] : k < 4 ? &sh.vfull[k - 2] : &sh.qfull[k - 4]),
                            (uint32_t)((sh.issued[k] - 1) & 1));
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ merge --

// One CTA takes 32 rows of a list, a lane a row, a warp D / 8 columns: the parts of
// the row -- of the CTAs that shared its list and, in prefix calls, those that
// shared its group's prefix -- in one online pass, kLoads of them in flight.  Where
// there are at most 16 rows, `slices` lanes share a row, each with every so many-th
// part, and join by shuffles.  Bound by latency: 8 us for the lists of 48 chains, 20
// for 28672 virtual rows with three parts each (with two parts in flight and 3 CTAs an
// SM, or 4, a call of few rows takes 24 and 32 us where it takes 22).
constexpr int kMergeThreads = 256;
constexpr int kPrefixRows = 256;  // virtual rows of a prefix list
template <int D, bool SPARSE>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ Args a) {
  griddep_entry();
  constexpr int kQuads = D / 32;  // of a warp
  constexpr int kLoads = 4;
  const int x = blockIdx.x;
  const int T = a.hdr->T, W = a.hdr->W, C = a.hdr->C, Wp = a.hdr->Wp, Cp = a.hdr->Cp;
  const int off0 = a.off[x], off1 = a.off[x + 1];  // (anything past the last list)
  const Tile tl = a.tiles[x / a.Hkv];
  if (x >= T * a.Hkv || off0 == off1) return;
  const int g = x % a.Hkv, group = a.group;
  const int vr0 = blockIdx.y * 32, vrows = tl.nr * group;
  if (vr0 >= vrows) return;
  const int lane = threadIdx.x & 31, c4 = (threadIdx.x >> 5) * kQuads;
  int rows2 = 1;  // rows of the block, rounded up to a power of two
  while (rows2 < 32 && rows2 < vrows - vr0) rows2 *= 2;
  const int slices = 32 / rows2, slice = lane / rows2;
  const int vr = vr0 + lane % rows2, vs = min(vr, vrows - 1);
  const int c0 = share_of(off0, W, C), ns = share_of(off1 - 1, W, C) - c0 + 1;
  int np = 0, p0 = 0, pv = 0;
  if (!SPARSE) {
    if (tl.first > 0) {
      const int4 grp = a.groups[tl.grp];
      const int v = (tl.arow - grp.x) * group + vs;  // among the group's virtual rows
      const int list = v / kPrefixRows * a.Hkv + g, sp = (grp.z + kStagePages - 1) / kStagePages;
      const int s0 = a.gstage[tl.grp] + list * (sp + kListStart) + kListStart;
      const int cp = share_of(s0, Wp, Cp);
      np = share_of(s0 + sp - 1, Wp, Cp) - cp + 1;
      p0 = cp + grp.w + list;
      pv = v % kPrefixRows;
    }
  }
  const int n = ns + np;  // (rows of a block may lie in two prefix lists)
  if (SPARSE ? n == 1 : np == 0 && ns == 1) return;  // written by the CTA that had it whole
  float Mx = -INFINITY, L = 0.f;
  float4 acc[kQuads];
#pragma unroll
  for (int j = 0; j < kQuads; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto join = [&](float m2, float l2, const float4 (&o2)[kQuads]) {
    const float nm = fmaxf(Mx, m2);
    if (nm == -INFINITY) return;
    const float s_old = exp2f(Mx - nm), s_new = exp2f(m2 - nm);
    L = L * s_old + l2 * s_new;
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      acc[j].x = acc[j].x * s_old + o2[j].x * s_new;
      acc[j].y = acc[j].y * s_old + o2[j].y * s_new;
      acc[j].z = acc[j].z * s_old + o2[j].z * s_new;
      acc[j].w = acc[j].w * s_old + o2[j].w * s_new;
    }
    Mx = nm;
  };
  for (int k0 = slice; k0 < n; k0 += kLoads * slices) {
    float2 ml2[kLoads];
    float4 o4[kLoads][kQuads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int s = k0 + k * slices;
      if (s >= n) break;
      const bool own = SPARSE || s < ns;
      const size_t slot = own ? (size_t)(c0 + s + x) : (size_t)(p0 + s - ns);
      const int rows = own ? a.tile_vr : kPrefixRows, row = own ? vs : pv;
      ml2[k] = __ldcg(reinterpret_cast<const float2*>(own ? a.ml : a.pml) + slot * rows + row);
      const float4* o = reinterpret_cast<const float4*>(own ? a.o : a.po) + (slot * (D / 4) + c4) * rows + row;
#pragma unroll
      for (int j = 0; j < kQuads; ++j) o4[k][j] = __ldcg(o + (size_t)j * rows);
    }
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      if (k0 + k * slices >= n) break;
      join(ml2[k].x, ml2[k].y, o4[k]);
    }
  }
  __syncwarp();
  for (int o = rows2; o < 32; o <<= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, Mx, o), l2 = __shfl_xor_sync(0xffffffffu, L, o);
    float4 o2[kQuads];
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      o2[j].x = __shfl_xor_sync(0xffffffffu, acc[j].x, o);
      o2[j].y = __shfl_xor_sync(0xffffffffu, acc[j].y, o);
      o2[j].z = __shfl_xor_sync(0xffffffffu, acc[j].z, o);
      o2[j].w = __shfl_xor_sync(0xffffffffu, acc[j].w, o);
    }
    join(m2, l2, o2);
  }
  if (vr >= vrows || slice != 0) return;
  const float inv = L > 0.f ? 1.f / L : 0.f;
  const size_t row = (size_t)(tl.cu + tl.r0 + vr / group) * a.Hq + g * group + vr % group;
  uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + c4 * 4);
#pragma unroll
  for (int j = 0; j < kQuads; j += 2)
    dst[j / 2] = make_uint4(pack_bf16(acc[j].x * inv, acc[j].y * inv), pack_bf16(acc[j].z * inv, acc[j].w * inv),
                            pack_bf16(acc[j + 1].x * inv, acc[j + 1].y * inv),
                            pack_bf16(acc[j + 1].z * inv, acc[j + 1].w * inv));
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
  if (bt->n_req > 0 && kv->num_blocks < 1) return SV_ERR_INVALID_ARGUMENT;
  if (bt->n_req > 0 && (!kv->k_cache || !kv->v_cache || !kv->block_tables || !kv->cache_lens))
    return SV_ERR_INVALID_ARGUMENT;
  if (((uintptr_t)kv->k_cache | (uintptr_t)kv->v_cache) & 15) return SV_ERR_INVALID_ARGUMENT;
  return SV_OK;
}

// Lists and their stages, starts included, are counted in 32 bits.
inline bool counts_fit(long lists, int max_blocks) {
  return lists < INT32_MAX && lists * (max_blocks / kStagePages + 3L + kListStart) < INT32_MAX;
}

// Whether the rows of q and out (bf16) share memory.
inline bool overlap(const void* q, const void* out, const sv_batch* bt, int32_t Hq, int D) {
  const uintptr_t n = (uintptr_t)bt->total_rows * Hq * D * 2, x = (uintptr_t)q, y = (uintptr_t)out;
  return x < y + n && y < x + n;
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
  a.dim = kv->head_dim;
  const int most = std::max(1, std::min(bt->max_rows_per_req, bt->total_rows));
  a.rt = std::min(kTileRows / a.group, most);
  a.tile_vr = a.rt * a.group;
  // ceil(rows / rt) tiles a request
  a.tiles_cap = (int)std::min((long)bt->total_rows / a.rt + bt->n_req, (long)INT32_MAX);
  a.ctas = std::max(2, sizing_sms());  // (a prefix call has CTAs of two kinds)
  const size_t lists = (size_t)a.tiles_cap * a.Hkv, slots = lists + a.ctas;
  a.hdr = take<Header>(at, off, 1);
  a.tiles = take<Tile>(at, off, a.tiles_cap);
  a.off = take<int>(at, off, lists + 1);
  a.start = take<int>(at, off, a.ctas);
  a.ml = take<float>(at, off, slots * a.tile_vr * 2);
  a.o = take<float>(at, off, slots * a.tile_vr * kv->head_dim);
  return a;
}

// The query rows as boxes of a tile: 64 elements x the heads of a KV head's group
// x the tile's rows.
inline bool make_q_map(CUtensorMap* map, const Args& a, int D) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = attn::encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)a.bt.total_rows};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.Hq * D * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)a.rt};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(a.q), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool SPARSE>
inline cudaError_t launch_merge(const Args& a, cudaStream_t stream) {
  const dim3 grid(a.tiles_cap * a.Hkv, (a.tile_vr + 31) / 32);
  return sv::launch(merge_kernel<D, SPARSE>, grid, kMergeThreads, 0, stream, a);
}

}  // namespace pu
}  // namespace sv
