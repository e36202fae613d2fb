// stage.cu — sv_stage_qkv: the draft rows' Q, K and V on their way from the
// projection to sv_tree_attend, in one pass: RMS norm of every Q and K head,
// rotation by the row's position(s), Q to its packed rows, K and V into the
// cache pages of the row's slot.
//
//   y = x * rsqrt(mean(x^2) + eps) * w        (fp32; without weights y = x)
//   angle_j = position[axis_j] * inv_freq_j,  j < rotary_dim / 2
//   (a, b) -> scale * (a cos - b sin, b cos + a sin)
//   with (a, b) elements (j, j + rotary_dim / 2) or (2j, 2j + 1) of the head.
// One rounding, to bf16, at the store: the norm, the angle and the rotation
// are fp32, so that a rounding of the normalised head is not rotated along.
//
// Angles of far positions: position * inv_freq in fp32 is off by up to 2^-24
// of itself, 0.06 rad at a million.  The turn inv_freq / (2 pi) is kept as a
// 64-bit binary fraction instead, and position * turn modulo one turn is a
// 64-bit integer product: what wraps away is whole turns.  The fraction is
// the fp32 mantissa times 2^64 / (2 pi), shifted by the exponent, good to a
// few units of 2^-64 for frequencies up to 1; no fp64, which this GPU has
// little of.
//
// Bound: HBM for many rows (each element read once and written once), launch
// and one load latency for few.  A piece is 16 elements of a head, two 16-byte
// vectors chosen so that both elements of every pair are the same thread's (8
// elements of the first half and their 8 partners of the second, or whole
// pairs of neighbours), and it lies at the same place of every head a thread works on:
// the rotation needs no exchange between lanes, and a row's sine and cosine
// are read from shared memory once for all its heads.  (With 8 elements per
// lane and shuffles for the partners, shared-memory and shuffle traffic
// bounded the kernel at 43 % of HBM.)  A norm is two or three shuffles.
// Many rows: each (or each half of one) goes to a warp, which loads kVecs
// pieces per lane ahead of the kVecs it works on, over the end of the row; the
// next row's sines are computed under its last loads.  Few: a CTA for each, all
// its loads at once.
// 20000 rows of 80 heads of 128: 134 us, 6.12 TB/s, 0.90 of the measured copy
// rate; six rows of 48 heads: 2.8 us.

#include <limits.h>
#include <math.h>

#include "sv_internal.cuh"

namespace sv {
namespace stg {

struct Args {
  const __nv_bfloat16 *q, *k, *v;
  long q_stride, k_stride, v_stride;  // elements between rows
  const int32_t* slots;
  const int32_t* positions;
  long axis_stride;          // elements between a row's positions on two axes
  const int32_t* freq_axis;  // null: axis 0
  const float* inv_freq;
  const float *qw, *kw;      // null: no norm
  __nv_bfloat16* out;
  __nv_bfloat16 *kc, *vc;
  int32_t* dev_status;
  long n_slots;
  int N, Hq, Hkv, rd, n_axes, inter;
  float eps, scale;
};

constexpr int kVecs = 3;          // pieces of a thread's round; two rounds are in flight
constexpr int kMaxThreads = 512;
constexpr int kStreamWarps = 16;  // warps of stream_kernel on an SM
// A CTA takes a row as long as all rows are on the SMs at once, or there are no
// more than kFewRows an SM; then a warp takes several in turn.  stream_kernel /
// row_kernel: 56 heads of 128, 1000 rows 9.1 / 7.6 us, 1500 rows 12.9 / 10.6,
// 1800 rows 13.3 / 13.4; 18 heads of 64, 4099 rows 8.0 / 6.5; rows too wide to be
// there together, 160 heads of 128: 700 rows (five an SM) 15.1 / 15.0, 1000 rows
// 22.0 / 23.9.
constexpr int kFewRows = 4;
constexpr int kMaxHalf = 64;      // rotated pairs of a head at most

// f / (2 pi) modulo one turn, in units of 2^-64 of a turn.
__device__ __forceinline__ unsigned long long turn_fraction(float f) {
  const unsigned long long kInv2Pi = 2935890503282001226ull;  // floor(2^64 / (2 pi))
  const uint32_t u = __float_as_uint(f);
  const int ex = (int)(u >> 23 & 255u);
  const unsigned long long m = (u & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int s = 150 - (ex ? ex : 1);  // f = m 2^-s
  const unsigned long long lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  unsigned long long t;
  if (s <= 0) t = s > -64 ? lo << -s : 0ull;
  else if (s < 64) t = lo >> s | hi << (64 - s);
  else t = s < 128 ? hi >> (s - 64) : 0ull;
  return u >> 31 ? 0ull - t : t;
}

__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Head h of row r: queries, then keys, then values.
template <int D>
__device__ __forceinline__ const __nv_bfloat16* piece_of(const Args& a, long r, int h) {
  if (h < a.Hq) return a.q + (size_t)r * a.q_stride + (size_t)h * D;
  if (h < a.Hq + a.Hkv) return a.k + (size_t)r * a.k_stride + (size_t)(h - a.Hq) * D;
  return a.v + (size_t)r * a.v_stride + (size_t)(h - a.Hq - a.Hkv) * D;
}

// (cos, sin) of pos turns of frac, times the scale.
__device__ __forceinline__ float2 turn_by(const Args& a, int pos, unsigned long long frac) {
  const long long turn = (long long)((unsigned long long)(long)pos * frac);
  float sn, co;
  sincospif((float)turn * 0x1p-63f, &sn, &co);  // signed: +- half a turn
  return make_float2(co * a.scale, sn * a.scale);
}

// An axis that there is.
__device__ __forceinline__ int checked_axis(const Args& a, int axis, bool used) {
  if (!used || (axis >= 0 && axis < a.n_axes)) return used ? axis : 0;
  flag(a.dev_status, SV_DEV_BAD_PARAM);
  return 0;
}

// Piece c of head h of row r (its elements at g0 and g1 of the head): norm,
// rotation, store.  Every lane of the warp calls it; `live` ones store.
template <int D>
__device__ __forceinline__ void finish(const Args& a, uint4 y0, uint4 y1, int h, bool live, int g0,
                                       int g1, bool rot, const float4 (&cs)[4], long r,
                                       size_t page) {
  constexpr int kLanes = D / 16;
  float f[16] = {lo_f(y0.x), hi_f(y0.x), lo_f(y0.y), hi_f(y0.y), lo_f(y0.z), hi_f(y0.z),
                 lo_f(y0.w), hi_f(y0.w), lo_f(y1.x), hi_f(y1.x), lo_f(y1.y), hi_f(y1.y),
                 lo_f(y1.z), hi_f(y1.z), lo_f(y1.w), hi_f(y1.w)};
  const bool turns = h < a.Hq + a.Hkv;
  const float* w = h < a.Hq ? a.qw : a.kw;
  if (a.qw || a.kw) {
    // (a head's lanes share a warp; those of V heads and past the row
    // take part in the shuffles and keep their elements)
    float ss = 0.f;
#pragma unroll
    for (int t = 0; t < 16; ++t) ss = fmaf(f[t], f[t], ss);
#pragma unroll
    for (int o = kLanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (turns && w) {
      const float rs = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float4 ww = __ldg(reinterpret_cast<const float4*>(w + (t < 2 ? g0 : g1)) + (t & 1));
        f[4 * t] *= rs * ww.x;
        f[4 * t + 1] *= rs * ww.y;
        f[4 * t + 2] *= rs * ww.z;
        f[4 * t + 3] *= rs * ww.w;
      }
    }
  }
  if (rot && turns) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const float co = t & 1 ? cs[t >> 1].z : cs[t >> 1].x;
      const float sn = t & 1 ? cs[t >> 1].w : cs[t >> 1].y;
      if (a.inter) {
        const float p0 = f[2 * t], p1 = f[2 * t + 1];
        f[2 * t] = p0 * co - p1 * sn;
        f[2 * t + 1] = p1 * co + p0 * sn;
      } else {
        const float p0 = f[t], p1 = f[t + 8];
        f[t] = p0 * co - p1 * sn;
        f[t + 8] = p1 * co + p0 * sn;
      }
    }
  }
  if (turns) {
    y0 = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
    y1 = make_uint4(pack_bf16(f[8], f[9]), pack_bf16(f[10], f[11]), pack_bf16(f[12], f[13]),
                    pack_bf16(f[14], f[15]));
  }
  if (live) {
    __nv_bfloat16* d;
    if (h < a.Hq) d = a.out + ((size_t)r * a.Hq + h) * D;
    else if (turns) d = a.kc + (page + (size_t)(h - a.Hq) * kBlockSize) * D;
    else d = a.vc + (page + (size_t)(h - a.Hq - a.Hkv) * kBlockSize) * D;
    *reinterpret_cast<uint4*>(d + g0) = y0;
    *reinterpret_cast<uint4*>(d + g1) = y1;
  }
}

// A warp's unit of work: a row (sh = 0) or half of one (sh = 1), `span` heads.
template <int D>
__global__ void __launch_bounds__(32) stream_kernel(Args a, int sh, int span) {
  griddep_entry();
  constexpr int kLanes = D / 16;  // lanes of a head
  __shared__ __align__(16) float2 s_cs[2][kMaxHalf];  // (cos, sin) of this row and the next
  const int tid = threadIdx.x;
  constexpr int nt = 32;
  const int half = a.rd >> 1;
  const int heads = a.Hq + 2 * a.Hkv;
  const int c = tid % kLanes, hs = tid / kLanes, hstep = nt / kLanes;
  const bool rot = 16 * c < a.rd;  // rotary_dim is a multiple of 16: whole pieces
  // A piece's two vectors lie half of the rotated (or of the other) elements
  // apart, whichever make a pair: neighbouring lanes read neighbouring vectors
  // (20000 rows with a norm alone 137 us; two neighbours a lane 160).
  const int g0 = rot ? 8 * c : a.rd + 8 * (c - a.rd / 16);
  const int g1 = g0 + (rot ? half : (D - a.rd) >> 1);
  const int t0 = (a.inter ? 4 : 8) * c, t1 = t0 + (a.inter ? half >> 1 : 4);  // their pairs
  // The frequencies this lane turns every row's position by, as loaded; what
  // they make is computed behind the first row's loads.
  constexpr int kFreqs = kMaxHalf / 32;
  float freq[kFreqs];
  int axis[kFreqs];
#pragma unroll
  for (int i = 0; i < kFreqs; ++i) {
    const int j = tid + i * nt;
    freq[i] = j < half ? a.inv_freq[j] : 0.f;
    axis[i] = j < half && a.freq_axis ? a.freq_axis[j] : 0;
  }
  const long units = (long)a.N << sh;
  // The slot of a unit's row and the positions its angles need, as loaded.
  struct Ahead {
    int slot;
    int pos[kFreqs];
  };
  unsigned long long frac[kFreqs];
  auto look = [&](long x, Ahead& n) {
    n.slot = -1;
    const long r = x >> sh;
    if (r < a.N) {
      n.slot = a.slots[r];
#pragma unroll
      for (int i = 0; i < kFreqs; ++i)
        if (tid + i * nt < half) n.pos[i] = a.positions[(size_t)axis[i] * a.axis_stride + r];
    }
  };
  // The first unit from x on (in steps of the grid) that is not skipped.
  auto settle = [&](long& x, Ahead& n) {
    while (x < units && (n.slot < 0 || n.slot >= a.n_slots)) {  // the same for the whole CTA
      if (n.slot != -1 && tid == 0) flag(a.dev_status, SV_DEV_BAD_SLOT);
      x += gridDim.x;
      look(x, n);
    }
  };
  auto turn_table = [&](const Ahead& n, float2* table) {
#pragma unroll
    for (int i = 0; i < kFreqs; ++i) {
      const int j = tid + i * nt;
      if (j < half) {
        table[j] = turn_by(a, n.pos[i], frac[i]);
      }
    }
  };
  auto from = [&](long x) { return sh ? ((int)x & 1) * span : 0; };  // its heads
  auto upto = [&](long x) { return min(heads, from(x) + span); };
  struct Round {
    uint4 x[kVecs][2];
  };
  auto fetch = [&](long x, int h0, Round& n) {
    const long r = x >> sh;
    const int to = upto(x);
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int h = h0 + u * hstep + hs;
      if (h < to) {
        const __nv_bfloat16* p = piece_of<D>(a, r, h);
        n.x[u][0] = *reinterpret_cast<const uint4*>(p + g0);
        n.x[u][1] = *reinterpret_cast<const uint4*>(p + g1);
      }
    }
  };
  long x = blockIdx.x;
  Ahead now;
  Round next;
  now.slot = a.slots[x >> sh];
  fetch(x, from(x), next);  // (a row that turns out to be skipped was read in vain)
#pragma unroll
  for (int i = 0; i < kFreqs; ++i) {
    axis[i] = checked_axis(a, axis[i], tid + i * nt < half);
    now.pos[i] = 0;
    if (tid + i * nt < half) now.pos[i] = a.positions[(size_t)axis[i] * a.axis_stride + (x >> sh)];
    frac[i] = turn_fraction(freq[i]);
  }
  if (now.slot < 0 || now.slot >= a.n_slots) {
    settle(x, now);
    if (x >= units) return;
    fetch(x, from(x), next);
  }
  turn_table(now, s_cs[0]);
  for (int par = 0; x < units; par ^= 1) {
    const long r = x >> sh;
    const int end = upto(x);
    const long slot = now.slot;
    const size_t page = (size_t)(slot / kBlockSize) * a.Hkv * kBlockSize + (size_t)(slot % kBlockSize);
    long xn = x + gridDim.x;
    look(xn, now);
    __syncwarp();  // the row's table is there, the other one is free
    float4 cs[4];     // this piece's eight pairs: (cos, sin, cos, sin)
    if (rot) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        cs[t] = *reinterpret_cast<const float4*>(&s_cs[par][(t < 2 ? t0 : t1) + 2 * (t & 1)]);
    }
    for (int h0 = from(x); h0 < end; h0 += kVecs * hstep) {
      const Round cur = next;
      if (h0 + kVecs * hstep < end) {
        fetch(x, h0 + kVecs * hstep, next);
      } else {
        settle(xn, now);
        if (xn < units) {
          fetch(xn, from(xn), next);
          turn_table(now, s_cs[par ^ 1]);
        }
      }
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        if (h0 + u * hstep >= end) break;  // the same for the whole CTA
        const int h = h0 + u * hstep + hs;
        finish<D>(a, cur.x[u][0], cur.x[u][1], h, h < end, g0, g1, rot, cs, r, page);
      }
    }
    x = xn;
  }
}

// Few rows: a CTA for each, every load the row needs in flight at once.  The
// pieces come to shared memory by asynchronous copies, each to a place that
// only the thread that asked for it reads, so no barrier stands between; a
// thread works on its first while the others are on their way.  (Two pieces of
// a thread at a time in registers: 1280 rows of 56 heads 11.8 us, so 10.2.)
constexpr int kRowVecs = 8;                  // pieces of a thread in flight at most
constexpr size_t kMaxRowSmem = 40 * 1024;
// Waits until all but the last n of this thread's copies are there.
__device__ __forceinline__ void wait_all_but(int n) {
  switch (n) {
    case 0: cp_async_wait<0>(); break;
    case 1: cp_async_wait<1>(); break;
    case 2: cp_async_wait<2>(); break;
    case 3: cp_async_wait<3>(); break;
    case 4: cp_async_wait<4>(); break;
    case 5: cp_async_wait<5>(); break;
    case 6: cp_async_wait<6>(); break;
    default: cp_async_wait<7>(); break;
  }
}
template <int D>
__global__ void __launch_bounds__(kMaxThreads, 2) row_kernel(Args a, int vecs) {
  griddep_entry();
  constexpr int kLanes = D / 16;
  __shared__ __align__(16) float2 s_cs[kMaxHalf];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int half = a.rd >> 1;
  const int heads = a.Hq + 2 * a.Hkv;
  const int c = tid % kLanes, hs = tid / kLanes, hstep = nt / kLanes;
  const bool rot = 16 * c < a.rd;
  // (the places that stream_kernel takes cost 1 us of 10 here)
  const int g0 = rot && !a.inter ? 8 * c : 16 * c;
  const int g1 = rot && !a.inter ? half + 8 * c : 16 * c + 8;
  const long r = blockIdx.x;
  const long slot = a.slots[r];
  constexpr int kFreqs = kMaxHalf / 32;
  float freq[kFreqs];
  int pos[kFreqs];
#pragma unroll
  for (int i = 0; i < kFreqs; ++i) {
    const int j = tid + i * nt;
    if (j < half) {
      freq[i] = a.inv_freq[j];
      const int axis = a.freq_axis ? checked_axis(a, a.freq_axis[j], true) : 0;
      pos[i] = a.positions[(size_t)axis * a.axis_stride + r];
    }
  }
  extern __shared__ __align__(16) uint4 s_x[];  // [vecs][2][nt]
  auto fetch = [&](int h0) {
    for (int u = 0; u < vecs; ++u) {
      const int h = h0 + u * hstep + hs;
      uint4* to = s_x + (size_t)u * 2 * nt + tid;
      if (h < heads) {
        const __nv_bfloat16* p = piece_of<D>(a, r, h);
        cp_async16(smem_u32(to), p + g0, 16);
        cp_async16(smem_u32(to + nt), p + g1, 16);
      } else {
        to[0] = to[nt] = make_uint4(0u, 0u, 0u, 0u);
      }
      cp_async_commit();
    }
  };
  fetch(0);  // (a row that turns out to be skipped was read in vain)
  if (slot < 0 || slot >= a.n_slots) {  // the same for the whole CTA
    if (slot != -1 && tid == 0) flag(a.dev_status, SV_DEV_BAD_SLOT);
    cp_async_wait<0>();
    return;
  }
#pragma unroll
  for (int i = 0; i < kFreqs; ++i) {
    const int j = tid + i * nt;
    if (j < half) s_cs[j] = turn_by(a, pos[i], turn_fraction(freq[i]));
  }
  __syncthreads();
  float4 cs[4];
  if (rot) {
#pragma unroll
    for (int t = 0; t < 4; ++t) cs[t] = *reinterpret_cast<const float4*>(&s_cs[8 * c + 2 * t]);
  }
  const size_t page = (size_t)(slot / kBlockSize) * a.Hkv * kBlockSize + (size_t)(slot % kBlockSize);
  for (int h0 = 0; h0 < heads; h0 += vecs * hstep) {
    if (h0 > 0) fetch(h0);
    for (int u = 0; u < vecs; ++u) {
      if (h0 + u * hstep >= heads) break;  // the same for the whole CTA
      const int h = h0 + u * hstep + hs;
      wait_all_but(vecs - 1 - u);
      const uint4* x = s_x + (size_t)u * 2 * nt + tid;
      finish<D>(a, x[0], x[nt], h, h < heads, g0, g1, rot, cs, r, page);
    }
  }
}

}  // namespace stg
}  // namespace sv

using namespace sv;

extern "C" sv_status sv_stage_qkv(const sv_paged_kv* kv, int32_t n_rows, const void* q,
                                  int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                  int64_t v_stride, int32_t n_q_heads, const int32_t* slots,
                                  const int32_t* positions, int64_t axis_stride,
                                  const sv_rotary* rotary, const float* q_weight,
                                  const float* k_weight, float eps, void* q_out,
                                  int32_t* dev_status, void* stream) {
  SV_TRACE("sv_stage_qkv");
  if (!kv || n_rows < 0 || n_q_heads < 1 || kv->n_kv_heads < 1 || kv->num_blocks < 0)
    return SV_ERR_INVALID_ARGUMENT;
  if (kv->block_size != kBlockSize || (kv->head_dim != 64 && kv->head_dim != 128) ||
      n_q_heads > 65536 || kv->n_kv_heads > 65536)
    return SV_ERR_UNSUPPORTED_SHAPE;
  const int D = kv->head_dim;
  stg::Args a{};
  if (rotary) {
    if (rotary->rotary_dim < 0 || rotary->rotary_dim > D || rotary->n_axes < 1 ||
        !(fabsf(rotary->scale) < INFINITY))
      return SV_ERR_INVALID_ARGUMENT;
    if (rotary->rotary_dim % 16) return SV_ERR_UNSUPPORTED_SHAPE;
    a.rd = rotary->rotary_dim;
    a.n_axes = rotary->n_axes;
    a.inter = rotary->interleaved ? 1 : 0;
    a.scale = rotary->scale;
    a.inv_freq = rotary->inv_freq;
    a.freq_axis = rotary->freq_axis;
    if (a.rd > 0 && (!a.inv_freq || (a.n_axes > 1 && !a.freq_axis)))
      return SV_ERR_INVALID_ARGUMENT;
  }
  // the negations refuse NaN too
  if ((q_weight || k_weight) && !(eps >= 0.f && eps < INFINITY)) return SV_ERR_INVALID_ARGUMENT;
  const int64_t qw = (int64_t)n_q_heads * D, kw = (int64_t)kv->n_kv_heads * D;
  if (n_rows > 1 && (q_stride < qw || k_stride < kw || v_stride < kw))
    return SV_ERR_INVALID_ARGUMENT;
  if (n_rows == 0) return SV_OK;
  if (!q || !k || !v || !slots || !q_out || !kv->k_cache || !kv->v_cache ||
      (a.rd > 0 && !positions) || axis_stride < 0)
    return SV_ERR_INVALID_ARGUMENT;
  // 16-byte vectors everywhere
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out | (uintptr_t)kv->k_cache |
       (uintptr_t)kv->v_cache | (uintptr_t)q_weight | (uintptr_t)k_weight) & 15)
    return SV_ERR_INVALID_ARGUMENT;
  if (n_rows > 1 && ((q_stride | k_stride | v_stride) & 7)) return SV_ERR_INVALID_ARGUMENT;
  // q_out is q itself (each vector is read by the thread that writes it) or apart
  const auto span = [&](const void* p, int64_t stride, int64_t width) {
    return (uintptr_t)p + ((uintptr_t)(n_rows - 1) * (uintptr_t)stride + (uintptr_t)width) * 2;
  };
  const uintptr_t o0 = (uintptr_t)q_out, o1 = span(q_out, qw, qw);
  const auto meets = [&](const void* p, int64_t stride, int64_t width) {
    return (uintptr_t)p < o1 && o0 < span(p, stride, width);
  };
  const bool in_place = q == q_out && (n_rows == 1 || q_stride == qw);
  if ((!in_place && meets(q, q_stride, qw)) || meets(k, k_stride, kw) || meets(v, v_stride, kw))
    return SV_ERR_INVALID_ARGUMENT;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slots = slots;
  a.positions = positions;
  a.axis_stride = axis_stride;
  a.qw = q_weight;
  a.kw = k_weight;
  a.out = static_cast<__nv_bfloat16*>(q_out);
  a.kc = static_cast<__nv_bfloat16*>(kv->k_cache);
  a.vc = static_cast<__nv_bfloat16*>(kv->v_cache);
  a.dev_status = dev_status;
  a.n_slots = (long)kv->num_blocks * kBlockSize;
  a.N = n_rows;
  a.Hq = n_q_heads;
  a.Hkv = kv->n_kv_heads;
  a.eps = eps;
  const int lanes = D / 16;
  const long pieces = (long)(n_q_heads + 2 * kv->n_kv_heads) * lanes;
  const int nsm = num_sms();
  if (nsm < 1) return SV_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  const long per_sm = ((long)n_rows + nsm - 1) / nsm;
  // a CTA's own shared memory: its table and what the system takes
  const bool resident = per_sm <= 32 && per_sm * (pieces * 32 + 1536) <= 227 * 1024L;
  if (!resident && per_sm > stg::kFewRows) {
    const int heads = n_q_heads + 2 * kv->n_kv_heads, round = stg::kVecs * (32 / lanes);
    const int rounds = (heads + round - 1) / round;
    // Halves of rows where the last wave would hold few whole ones (2600 rows of
    // 80 heads 25.0 us against 26.9; of 160 heads 42.7 against 49.2).  Rows of
    // one round are never halved: no half is empty.
    const long wave = (long)nsm * stg::kStreamWarps;
    const auto cost = [&](int parts, int each) {
      return (n_rows * (long)parts + wave - 1) / wave * (2 * each + 1);
    };
    const int sh = cost(2, (rounds + 1) / 2) < cost(1, rounds) ? 1 : 0;
    const int span = ((rounds + (1 << sh) - 1) >> sh) * round;
    e = sv::launch(D == 64 ? stg::stream_kernel<64> : stg::stream_kernel<128>,
                   (unsigned)min((long)n_rows << sh, 2 * wave), 32, 0, s, a, sh, span);
  } else {
    // a thread for every piece while that leaves an SM's rows side by side
    // (1280 rows of 56 heads of 128, nine an SM: 96 threads 10.4 us, 64 13.0,
    // 128 12.6; 300 rows, two an SM: 448 threads 4.1 us, 384 4.4)
    const long most = min((long)stg::kMaxThreads, 1024 / per_sm / 32 * 32);
    const unsigned threads = (unsigned)max(32L, min(most, (pieces + 31) / 32 * 32));
    const long each = (pieces + threads - 1) / threads;
    const long room = (long)(stg::kMaxRowSmem / (32 * threads));
    const int vecs = (int)max(1L, min(min(each, (long)stg::kRowVecs), room));
    e = sv::launch(D == 64 ? stg::row_kernel<64> : stg::row_kernel<128>, (unsigned)n_rows, threads,
                   (size_t)vecs * threads * 32, s, a, vecs);
  }
  if (e != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}
