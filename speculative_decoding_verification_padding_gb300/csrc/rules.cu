// rules.cu — sv_shape_logits: each draft node's logits under its request's
// rules: penalties for the tokens seen on the way to the node, biases, and a
// grammar mask, in one pass from the head's output to the logits sv_accept
// reads.
//
//   c(v) = occurrences of v in history[prompt_len ..] and among the drafts on
//          the node's path (the root's token is the history's last)
//   seen = c(v) > 0 or v in history[.. prompt_len)
//   y = seen ? (x > 0 ? x / repetition : x * repetition) : x
//   y = y - (frequency * c + presence * [c > 0]) + bias(v)
//   y = -inf where the node's mask has a zero
//
// Bound: HBM, 4 bytes written and 2 or 4 read per logit; a barred logit is
// not read.  Few tokens of a row are touched by a rule, and they are the same
// for all rows of a request but for their paths.  So a CTA takes kSlice
// entries of the vocabulary and up to kGroup packed rows, counts the
// request's history into shared memory once (every CTA reads the whole
// history from L2 and keeps what falls in its slice: no workspace, no global
// atomics, no order that could change a result), marks the touched tokens in
// a bit map, and streams the rows: four entries cost one nibble test unless
// one of them is marked.  A row's path tokens are added to the counts before
// the row and taken out after it, which needs a barrier only in the rare
// slices that hold one.

#include "sv_internal.cuh"

namespace sv {
namespace rul {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlice = 4096;   // vocabulary entries of a CTA
constexpr int kGroup = kWarps; // packed rows of a CTA (a warp prepares each)
constexpr int kQuads = kSlice / (4 * kThreads);

struct Args {
  sv_batch bt;
  const void* logits;
  long stride;
  float* out;
  sv_logit_rules ru;
  int32_t* dev_status;
  int V, slices;
};

struct Smem {
  unsigned cnt[kSlice];        // occurrences; the top bit: seen in the prompt
  unsigned bits[kSlice / 32];  // tokens of the slice that a rule touches
  int tok[kMaxRows];
  int8_t par[kMaxRows];
  int owner[kGroup];
  int npath[kGroup];           // drafts of the row's path inside the slice
  int masked[kGroup];          // the row's mask row, -1: none
  uint16_t path[kGroup][kMaxRows];
};
// Behind it, with biases: the lowest list position of each token.
constexpr size_t kBiasAt = (sizeof(Smem) + 15) / 16 * 16;
constexpr size_t kBiasBytes = kSlice * sizeof(unsigned);

constexpr unsigned kSeen = 0x80000000u;

struct Rule {
  float rho, freq, pres;
  const float* bias;  // values of the request's list
  bool pen;
};

__device__ __forceinline__ float apply(float x, int o, const Rule& ru, const Smem& sm,
                                       const unsigned* first) {
  if (ru.pen) {
    const unsigned c = sm.cnt[o];
    if (c) {
      x = x > 0.f ? __fdiv_rn(x, ru.rho) : x * ru.rho;
      const unsigned n = c & ~kSeen;
      if (n) x -= ru.freq * (float)n + ru.pres;
    }
  }
  if (first) {
    const unsigned k = first[o];
    if (k != 0xffffffffu) x += ru.bias[k];
  }
  return x;
}

__device__ __forceinline__ float load1(const float* p) { return __ldcs(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float4 load4(const float* p) {
  return __ldcs(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// The words of mask row m that overlap entries [lo, lo + n): any bit set?  By
// one warp; bits past the vocabulary do not count.
__device__ __forceinline__ bool any_bit(const int32_t* m, int lo, int n, int V) {
  const int lane = threadIdx.x & 31;
  const int w0 = lo >> 5, w1 = (lo + n + 31) >> 5, last = (V - 1) >> 5;
  for (int w = w0; w < w1; w += 32 * 8) {
    unsigned x = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int at = w + 32 * k + lane;
      if (at < w1) {
        unsigned b = (unsigned)__ldg(m + at);
        if (at == last && (V & 31)) b &= (1u << (V & 31)) - 1u;
        x |= b;
      }
    }
    if (__any_sync(0xffffffffu, x != 0)) return true;
  }
  return false;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) rules_kernel(Args a) {
  griddep_entry();
  extern __shared__ __align__(16) uint8_t s_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(s_raw);
  unsigned* s_first = a.ru.bias_begin
                          ? reinterpret_cast<unsigned*>(s_raw + kBiasAt)
                          : nullptr;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int slice = (int)(blockIdx.x % (unsigned)a.slices);
  const int r0 = (int)(blockIdx.x / (unsigned)a.slices) * kGroup;
  const int r1 = min(a.bt.total_rows, r0 + kGroup);
  const int lo = slice * kSlice, n = min(kSlice, a.V - lo);
  const sv_logit_rules& ru = a.ru;

  // owners of the group's rows
  if (tid < kGroup) sm.owner[tid] = -1;
  __syncthreads();
  for (int i = tid; i < a.bt.n_req; i += kThreads) {
    const int c0 = a.bt.cu_rows[i], c1 = a.bt.cu_rows[i + 1];
    for (int r = max(c0, r0); r < min(c1, r1); ++r) sm.owner[r - r0] = i;
  }
  __syncthreads();

  for (int r = r0; r < r1;) {
    const int i = sm.owner[r - r0];
    int end = r + 1;
    while (end < r1 && sm.owner[end - r0] == i) ++end;
    const int first_row = r;
    r = end;
    if (i < 0) continue;  // padding rows
    const Window w = window_of(a.bt, i);
    if (!w.ok) {
      if (tid == 0) flag(a.dev_status, SV_DEV_BAD_WINDOW);
      continue;
    }
    const int ra = max(first_row, w.cu + w.b), rb = min(end, w.cu + w.e);
    if (ra >= rb) continue;
    Rule rule;
    rule.rho = ru.repetition ? ru.repetition[i] : 1.f;
    rule.freq = ru.frequency ? ru.frequency[i] : 0.f;
    rule.pres = ru.presence ? ru.presence[i] : 0.f;
    rule.pen = rule.rho != 1.f || rule.freq != 0.f || rule.pres != 0.f;
    const int hlen = ru.history ? ru.history_len[i] : 0;
    const int plen = ru.history && ru.prompt_len ? ru.prompt_len[i] : 0;
    int b0 = 0, b1 = 0;
    if (s_first) {
      b0 = ru.bias_begin[i];
      b1 = ru.bias_begin[i + 1];
    }
    int finding = 0;
    if (!(rule.rho > 0.f && rule.rho < INFINITY) || !(fabsf(rule.freq) < INFINITY) ||
        !(fabsf(rule.pres) < INFINITY) || b0 < 0 || b1 < b0 || b1 > ru.n_bias)
      finding = SV_DEV_BAD_PARAM;
    else if (hlen < 0 || hlen > ru.max_history || plen < 0 || plen > hlen)
      finding = SV_DEV_BAD_LENGTH;
    if (finding) {  // the request's rows are left as they were
      if (tid == 0) flag(a.dev_status, finding);
      continue;
    }
    rule.bias = s_first ? ru.bias_value + b0 : nullptr;

    // ---- the request's counts, biases and tree in shared memory ----
    __syncthreads();  // the last request's are no longer read
    if (tid < kSlice / 32) sm.bits[tid] = 0;
    bool bad = false;
    if (rule.pen) {
      for (int o = tid; o < kSlice / 4; o += kThreads)
        reinterpret_cast<uint4*>(sm.cnt)[o] = make_uint4(0u, 0u, 0u, 0u);
      for (int j = tid; j < w.rows; j += kThreads) {
        const int p = a.bt.parent[w.cu + j];
        sm.tok[j] = a.bt.tokens[w.cu + j];
        sm.par[j] = (int8_t)(p >= 0 && p < j ? p : 0);
        if (j == 0 ? p != -1 : (p < 0 || p >= j)) bad = true;
      }
    }
    if (b1 > b0)
      for (int o = tid; o < kSlice; o += kThreads) s_first[o] = 0xffffffffu;
    if (__syncthreads_or(bad)) {
      if (tid == 0) flag(a.dev_status, SV_DEV_BAD_PARENT);
      continue;
    }
    if (rule.pen) {
      const int32_t* h = ru.history + (size_t)i * ru.max_history;
      for (int t = tid; t < hlen; t += kThreads) {
        const unsigned o = (unsigned)(h[t] - lo);
        if (o < (unsigned)n) {
          if (t < plen) atomicOr(&sm.cnt[o], kSeen);
          else atomicAdd(&sm.cnt[o], 1u);
          atomicOr(&sm.bits[o >> 5], 1u << (o & 31));
        }
      }
    }
    for (int t = b0 + tid; t < b1; t += kThreads) {
      const unsigned o = (unsigned)(ru.bias_token[t] - lo);
      if (o < (unsigned)n) {
        atomicMin(&s_first[o], (unsigned)(t - b0));
        atomicOr(&sm.bits[o >> 5], 1u << (o & 31));
      }
    }
    // a warp for each row: its path's drafts in the slice, its mask
    if (ra + wid < rb) {
      const int row = ra + wid;
      int np = 0;
      if (rule.pen && lane == 0) {
        for (int p = row - w.cu; p > 0; p = sm.par[p]) {
          const unsigned o = (unsigned)(sm.tok[p] - lo);
          if (o < (unsigned)n) {
            sm.path[wid][np++] = (uint16_t)o;
            atomicOr(&sm.bits[o >> 5], 1u << (o & 31));
          }
        }
      }
      int m = -1;
      if (ru.mask) {
        m = ru.mask_row ? ru.mask_row[row] : row;
        if (m < -1 || m >= ru.n_masks) {
          if (lane == 0) flag(a.dev_status, SV_DEV_BAD_PARAM);
          m = -1;
        }
        if (m >= 0) {
          const int32_t* words = ru.mask + (size_t)m * ru.mask_stride;
          // a mask that lets nothing through would leave no distribution
          if (!any_bit(words, lo, n, a.V) && !any_bit(words, 0, a.V, a.V)) {
            if (lane == 0) flag(a.dev_status, SV_DEV_EMPTY_MASK);
            m = -1;
          }
        }
      }
      if (lane == 0) {
        sm.npath[wid] = np;
        sm.masked[wid] = m;
      }
    }
    __syncthreads();

    // ---- the rows ----
    const unsigned* first = b1 > b0 ? s_first : nullptr;
    int added = -1;  // the row whose path is in the counts
    for (int k = 0; k < rb - ra; ++k) {
      const int np = sm.npath[k];
      if (np > 0 || added >= 0) {  // the same for the whole CTA
        __syncthreads();
        if (added >= 0)
          for (int t = tid; t < sm.npath[added]; t += kThreads)
            atomicSub(&sm.cnt[sm.path[added][t]], 1u);
        for (int t = tid; t < np; t += kThreads) atomicAdd(&sm.cnt[sm.path[k][t]], 1u);
        added = np > 0 ? k : -1;
        __syncthreads();
      }
      const T* src = static_cast<const T*>(a.logits) + (size_t)(ra + k) * a.stride + lo;
      float* dst = a.out + (size_t)(ra + k) * a.V + lo;
      const int m = sm.masked[k];
      const int32_t* words = m >= 0 ? ru.mask + (size_t)m * ru.mask_stride + (lo >> 5) : nullptr;
      if (VEC) {
        float4 x[kQuads];
        unsigned let[kQuads];
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
          const int o = 4 * (q * kThreads + tid);
          let[q] = 15u;
          if (words && o < n) let[q] = ((unsigned)__ldg(words + (o >> 5)) >> (o & 31)) & 15u;
        }
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
          const int o = 4 * (q * kThreads + tid);
          x[q] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (o < n && let[q]) x[q] = load4(src + o);
        }
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
          const int o = 4 * (q * kThreads + tid);
          if (o >= n) break;
          const unsigned hit = (sm.bits[o >> 5] >> (o & 31)) & let[q];
          if (hit) {
            if (hit & 1u) x[q].x = apply(x[q].x, o, rule, sm, first);
            if (hit & 2u) x[q].y = apply(x[q].y, o + 1, rule, sm, first);
            if (hit & 4u) x[q].z = apply(x[q].z, o + 2, rule, sm, first);
            if (hit & 8u) x[q].w = apply(x[q].w, o + 3, rule, sm, first);
          }
          if (!(let[q] & 1u)) x[q].x = -INFINITY;
          if (!(let[q] & 2u)) x[q].y = -INFINITY;
          if (!(let[q] & 4u)) x[q].z = -INFINITY;
          if (!(let[q] & 8u)) x[q].w = -INFINITY;
          *reinterpret_cast<float4*>(dst + o) = x[q];
        }
      } else {
        float x[4 * kQuads];
        unsigned let = 0;
#pragma unroll
        for (int q = 0; q < 4 * kQuads; ++q) {
          const int o = q * kThreads + tid;
          unsigned l = 1u;
          if (words && o < n) l = ((unsigned)__ldg(words + (o >> 5)) >> (o & 31)) & 1u;
          let |= l << q;
        }
#pragma unroll
        for (int q = 0; q < 4 * kQuads; ++q) {
          const int o = q * kThreads + tid;
          x[q] = 0.f;
          if (o < n && (let >> q & 1u)) x[q] = load1(src + o);
        }
#pragma unroll
        for (int q = 0; q < 4 * kQuads; ++q) {
          const int o = q * kThreads + tid;
          if (o >= n) break;
          if (!(let >> q & 1u)) x[q] = -INFINITY;
          else if (sm.bits[o >> 5] >> (o & 31) & 1u) x[q] = apply(x[q], o, rule, sm, first);
          dst[o] = x[q];
        }
      }
    }
  }
}

}  // namespace rul
}  // namespace sv

using namespace sv;

extern "C" sv_status sv_shape_logits(const sv_batch* bt, const void* logits, int32_t logits_type,
                                     int64_t logits_stride, int32_t vocab,
                                     const sv_logit_rules* rules, float* out, int32_t* dev_status,
                                     void* stream) {
  SV_TRACE("sv_shape_logits");
  if (!bt || !rules || bt->n_req < 0 || bt->total_rows < 0 || bt->max_rows_per_req < 1 || vocab < 1)
    return SV_ERR_INVALID_ARGUMENT;
  if (logits_type != SV_LOGITS_F32 && logits_type != SV_LOGITS_BF16)
    return SV_ERR_INVALID_ARGUMENT;
  if (bt->max_rows_per_req > kMaxRows) return SV_ERR_UNSUPPORTED_SHAPE;
  if (bt->total_rows > 1 && logits_stride < vocab) return SV_ERR_INVALID_ARGUMENT;
  const sv_logit_rules& ru = *rules;
  const bool pen = ru.repetition || ru.frequency || ru.presence;
  if (ru.history && (!ru.history_len || ru.max_history < 0)) return SV_ERR_INVALID_ARGUMENT;
  if (ru.bias_begin && (!ru.bias_token || !ru.bias_value || ru.n_bias < 0))
    return SV_ERR_INVALID_ARGUMENT;
  if (ru.mask && (ru.mask_stride < (vocab + 31) / 32 || ru.n_masks < 0 ||
                  (!ru.mask_row && ru.n_masks < bt->total_rows)))
    return SV_ERR_INVALID_ARGUMENT;
  if (bt->n_req == 0 || bt->total_rows == 0) return SV_OK;
  if (!bt->cu_rows || !logits || !out || (pen && (!bt->parent || !bt->tokens)))
    return SV_ERR_INVALID_ARGUMENT;
  const uintptr_t esz = logits_type == SV_LOGITS_F32 ? 4 : 2;
  const uintptr_t in = (uintptr_t)logits, to = (uintptr_t)out;
  if ((in & (esz - 1)) || (to & 3)) return SV_ERR_INVALID_ARGUMENT;
  // in place or apart: each logit is read by the thread that writes it
  const uintptr_t in_end =
      in + ((uintptr_t)(bt->total_rows - 1) * (uintptr_t)logits_stride + (uintptr_t)vocab) * esz;
  const uintptr_t to_end = to + (uintptr_t)bt->total_rows * (uintptr_t)vocab * 4;
  const bool same = in == to && esz == 4 && (bt->total_rows == 1 || logits_stride == vocab);
  if (!same && in < to_end && to < in_end) return SV_ERR_INVALID_ARGUMENT;
  rul::Args a;
  a.bt = *bt;
  a.logits = logits;
  a.stride = logits_stride;
  a.out = out;
  a.ru = ru;
  if (!pen) a.ru.history = nullptr;
  if (!a.ru.history) a.ru.max_history = 0;
  a.dev_status = dev_status;
  a.V = vocab;
  a.slices = (vocab + rul::kSlice - 1) / rul::kSlice;
  // four entries at a time where every row starts on a multiple of four
  // (16-byte stores; the loads are 16 bytes of fp32 or 8 of bf16)
  const bool vec = vocab % 4 == 0 && (to & 15) == 0 && (in & (4 * esz - 1)) == 0 &&
                   (bt->total_rows == 1 || logits_stride % 4 == 0);
  const long groups = ((long)bt->total_rows + rul::kGroup - 1) / rul::kGroup;
  if (groups * a.slices > 0x7fffffffL) return SV_ERR_UNSUPPORTED_SHAPE;
  const size_t smem = rul::kBiasAt + (ru.bias_begin ? rul::kBiasBytes : 0);
  void (*kernel)(rul::Args) =
      logits_type == SV_LOGITS_F32
          ? (vec ? rul::rules_kernel<float, true> : rul::rules_kernel<float, false>)
          : (vec ? rul::rules_kernel<__nv_bfloat16, true> : rul::rules_kernel<__nv_bfloat16, false>);
  if (sv::launch(kernel, (unsigned)(groups * a.slices), rul::kThreads, smem,
                 static_cast<cudaStream_t>(stream), a) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}
