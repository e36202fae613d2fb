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
// good to 2^-53 of a turn of inv_freq / (2 pi), so a position of 2^31 still
// has an angle good to 2^-20; fp64 is used once per thread, not per row.
//
// Bound: HBM for many rows (each element read once and written once), launch
// and one load latency for few.  A CTA takes whole rows, so that the row's
// sines are computed once for all its heads; a thread holds up to kVecs
// 16-byte vectors of the row, all loaded before the sines are computed.
// Eight or sixteen neighbouring lanes hold one head (64 or 128 elements), so
// a norm is three or four shuffles, and a pair's partner is in another lane
// of the same head (halves) or in the same vector (pairs side by side).

#include <limits.h>

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

constexpr int kVecs = 4;          // vectors of a row in flight per thread
constexpr int kMaxThreads = 320;
constexpr int kMaxHalf = 64;      // rotated pairs of a head at most

// inv_freq / (2 pi) modulo one turn, in units of 2^-64 of a turn.
__device__ __forceinline__ unsigned long long turn_fraction(float f) {
  const double t = (double)f * 0.15915494309189533577;  // 1 / (2 pi)
  const double frac = t - floor(t);
  return (unsigned long long)(frac * 18446744073709551616.0);  // 2^64; frac <= 1 - 2^-53
}

__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

template <int D>
__global__ void __launch_bounds__(kMaxThreads) stage_kernel(Args a) {
  griddep_entry();
  constexpr int kLanes = D / 8;  // lanes of a head
  __shared__ float2 s_cs[2][kMaxHalf];  // (cos, sin) of this row and the next
  const int tid = threadIdx.x, nt = blockDim.x;
  const int half = a.rd >> 1;
  const int heads = a.Hq + 2 * a.Hkv;
  const int nvec = heads * kLanes;
  // the frequency this thread turns every row's position by
  unsigned long long frac = 0;
  int axis = 0;
  if (tid < half) {
    frac = turn_fraction(a.inv_freq[tid]);
    if (a.freq_axis) {
      axis = a.freq_axis[tid];
      if (axis < 0 || axis >= a.n_axes) {
        flag(a.dev_status, SV_DEV_BAD_PARAM);
        axis = 0;
      }
    }
  }
  int par = 0;
  for (int r = blockIdx.x; r < a.N; r += gridDim.x) {
    const long slot = a.slots[r];
    if (slot < 0 || slot >= a.n_slots) {  // the same for the whole CTA
      if (slot != -1 && tid == 0) flag(a.dev_status, SV_DEV_BAD_SLOT);
      continue;
    }
    const __nv_bfloat16* src[3] = {a.q + (size_t)r * a.q_stride, a.k + (size_t)r * a.k_stride,
                                   a.v + (size_t)r * a.v_stride};
    bool turned = half == 0;
    for (int v0 = 0; v0 < nvec; v0 += kVecs * nt) {
      uint4 x[kVecs];
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const int vec = v0 + u * nt + tid;
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        if (vec < nvec) {
          int h = vec / kLanes, which = 0;
          if (h >= a.Hq) { h -= a.Hq; which = 1; }
          if (which && h >= a.Hkv) { h -= a.Hkv; which = 2; }
          const __nv_bfloat16* p = which == 0 ? src[0] : which == 1 ? src[1] : src[2];
          x[u] = *reinterpret_cast<const uint4*>(p + (size_t)h * D + (vec % kLanes) * 8);
        }
      }
      if (!turned) {
        // the row's sines, behind the loads; two rows' tables alternate, so
        // one barrier per row is enough
        if (tid < half) {
          const long pos = a.positions[(size_t)axis * a.axis_stride + r];
          const long long turn = (long long)((unsigned long long)pos * frac);  // signed: +- half a turn
          float s, c;
          sincospif((float)turn * 0x1p-63f, &s, &c);
          s_cs[par][tid] = make_float2(c * a.scale, s * a.scale);
        }
        __syncthreads();
        turned = true;
      }
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const int vec = v0 + u * nt + tid;
        if (v0 + u * nt >= nvec) break;  // the same for the whole CTA
        const int c = vec % kLanes;      // this lane's eighth of the head
        int h = vec / kLanes, which = 0;
        if (h >= a.Hq) { h -= a.Hq; which = 1; }
        if (which && h >= a.Hkv) { h -= a.Hkv; which = 2; }
        uint4 y = x[u];
        float f[8] = {lo_f(y.x), hi_f(y.x), lo_f(y.y), hi_f(y.y),
                      lo_f(y.z), hi_f(y.z), lo_f(y.w), hi_f(y.w)};
        const float* w = which == 0 ? a.qw : a.kw;
        // (a head's lanes always share a warp; lanes of V heads and past the
        // row take part in the shuffles and keep their elements)
        float ss = 0.f;
#pragma unroll
        for (int t = 0; t < 8; ++t) ss = fmaf(f[t], f[t], ss);
#pragma unroll
        for (int o = kLanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (w && which < 2) {
          const float rs = rsqrtf(ss * (1.f / D) + a.eps);
          const float4 w0 = *reinterpret_cast<const float4*>(w + c * 8);
          const float4 w1 = *reinterpret_cast<const float4*>(w + c * 8 + 4);
          f[0] = f[0] * rs * w0.x; f[1] = f[1] * rs * w0.y;
          f[2] = f[2] * rs * w0.z; f[3] = f[3] * rs * w0.w;
          f[4] = f[4] * rs * w1.x; f[5] = f[5] * rs * w1.y;
          f[6] = f[6] * rs * w1.z; f[7] = f[7] * rs * w1.w;
        }
        if (half) {
          if (a.inter) {
            if (c * 8 < a.rd && which < 2) {
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const float2 cs = s_cs[par][c * 4 + t];
                const float p0 = f[2 * t], p1 = f[2 * t + 1];
                f[2 * t] = p0 * cs.x - p1 * cs.y;
                f[2 * t + 1] = p1 * cs.x + p0 * cs.y;
              }
            }
          } else {
            // element e < half pairs with e + half, half a multiple of 8:
            // the partner is the same element of the lane half / 8 away
            const int hl = half >> 3;
            const int lane0 = (tid & 31) - c;
            const int mate = c < hl ? c + hl : c < 2 * hl ? c - hl : c;
            const float sgn = c < hl ? -1.f : 1.f;
            const bool rot = c < 2 * hl && which < 2;
            const int j0 = (c < hl ? c : c - hl) * 8;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
              const float o = __shfl_sync(0xffffffffu, f[t], lane0 + mate);
              if (rot) {
                const float2 cs = s_cs[par][j0 + t];
                f[t] = f[t] * cs.x + sgn * o * cs.y;
              }
            }
          }
        }
        if (which < 2) {
          y.x = pack_bf16(f[0], f[1]);
          y.y = pack_bf16(f[2], f[3]);
          y.z = pack_bf16(f[4], f[5]);
          y.w = pack_bf16(f[6], f[7]);
        }
        if (vec < nvec) {
          __nv_bfloat16* dst;
          if (which == 0) {
            dst = a.out + ((size_t)r * a.Hq + h) * D;
          } else {
            const size_t page = (size_t)(slot / kBlockSize) * a.Hkv + h;
            dst = (which == 1 ? a.kc : a.vc) + (page * kBlockSize + (size_t)(slot % kBlockSize)) * D;
          }
          *reinterpret_cast<uint4*>(dst + c * 8) = y;
        }
      }
    }
    par ^= 1;
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
        !(rotary->scale == rotary->scale))
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
  if ((q_weight || k_weight) && !(eps >= 0.f)) return SV_ERR_INVALID_ARGUMENT;
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
  const int nvec = (n_q_heads + 2 * kv->n_kv_heads) * (D / 8);
  // threads: the fewest vectors each that keep the CTA at kMaxThreads, evenly
  int per = 1;
  while ((nvec + per - 1) / per > stg::kMaxThreads) ++per;
  int threads = ((nvec + per - 1) / per + 31) / 32 * 32;
  threads = max(threads, stg::kMaxHalf);  // a thread for every rotated pair
  const int nsm = num_sms();
  if (nsm < 1) return SV_ERR_CUDA;
  const unsigned grid = (unsigned)min((long)n_rows, (long)nsm * (2048 / threads));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (sv::launch(D == 64 ? stg::stage_kernel<64> : stg::stage_kernel<128>, grid, (unsigned)threads,
                 0, s, a) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}
