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
// entries of the vocabulary and some rows of one request, counts the
// request's history into shared memory once (every CTA reads the whole
// history from L2 and keeps what falls in its slice: no workspace, no global
// atomics, no order that could change a result), marks the touched tokens in
// a bit map, and streams the rows: four entries cost one nibble test unless
// one of them is marked.  The drafts of a row's path are added to the counts
// before the row and taken out after it, which needs a barrier only in the
// few slices that hold one.

#include "sv_internal.cuh"

namespace sv {
namespace rul {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlice = 4096;  // vocabulary entries of a CTA
constexpr int kMaxChunk = 32; // rows of a CTA at most
constexpr int kQuads = kSlice / (4 * kThreads);
constexpr int kHistLoads = 16;  // history tokens of a thread in flight

struct Args {
  sv_batch bt;
  const void* logits;
  long stride;
  float* out;
  sv_logit_rules ru;
  int32_t* dev_status;
  int V, slices, chunks, chunk;  // chunks of `chunk` rows per request
};

struct Smem {
  unsigned cnt[kSlice];        // occurrences; the top bit: seen in the prompt
  unsigned bits[kSlice / 32];  // tokens of the slice that a rule touches
  int tok[kMaxRows];
  int8_t par[kMaxRows];
  unsigned mine[kMaxRows / 32];                // nodes whose token is in the slice
  unsigned path[kMaxChunk][kMaxRows / 32];     // of those, the nodes on the row's path
  int masked[kMaxChunk];                       // the row's mask row, -1: none
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
  unsigned* s_first = reinterpret_cast<unsigned*>(s_raw + kBiasAt);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int slice = (int)(blockIdx.x % (unsigned)a.slices);
  const int unit = (int)(blockIdx.x / (unsigned)a.slices);
  const int i = unit / a.chunks, chunk = unit % a.chunks;
  const int lo = slice * kSlice, n = min(kSlice, a.V - lo);
  const sv_logit_rules& ru = a.ru;

  // ---- the request: everything that only its number leads to, at once ----
  const Window w = window_of(a.bt, i);
  Rule rule;
  rule.rho = ru.repetition ? ru.repetition[i] : 1.f;
  rule.freq = ru.frequency ? ru.frequency[i] : 0.f;
  rule.pres = ru.presence ? ru.presence[i] : 0.f;
  const int hlen = ru.history ? ru.history_len[i] : 0;
  const int plen = ru.history && ru.prompt_len ? ru.prompt_len[i] : 0;
  const int b0 = ru.bias_begin ? ru.bias_begin[i] : 0;
  const int b1 = ru.bias_begin ? ru.bias_begin[i + 1] : 0;
  rule.pen = rule.rho != 1.f || rule.freq != 0.f || rule.pres != 0.f;
  rule.bias = ru.bias_value + b0;
  const unsigned* first = b1 > b0 ? s_first : nullptr;
  int finding = 0;
  if (!w.ok)
    finding = SV_DEV_BAD_WINDOW;
  else if (!(rule.rho > 0.f && rule.rho < INFINITY) || !(fabsf(rule.freq) < INFINITY) ||
           !(fabsf(rule.pres) < INFINITY) || b0 < 0 || b1 < b0 || b1 > ru.n_bias)
    finding = SV_DEV_BAD_PARAM;
  else if (hlen < 0 || hlen > ru.max_history || plen < 0 || plen > hlen)
    finding = SV_DEV_BAD_LENGTH;
  if (finding) {  // the request's rows are left as they were
    if (tid == 0) flag(a.dev_status, finding);
    return;
  }
  const int j0 = w.b + chunk * a.chunk, j1 = min(w.e, j0 + a.chunk);  // this CTA's nodes
  if (j0 >= j1) return;
  const int ra = w.cu + j0, rows = j1 - j0;

  // ---- its counts, biases and paths in shared memory ----
  bool bad = false;
  if (tid < kSlice / 32) sm.bits[tid] = 0;
  if (rule.pen) {
    // (one node per thread: a request has at most kMaxRows of them)
    int p = 0, t = -1;
    if (tid < w.rows) {
      p = a.bt.parent[w.cu + tid];
      t = a.bt.tokens[w.cu + tid];
      bad = tid == 0 ? p != -1 : (p < 0 || p >= tid);
    }
    if (tid < kMaxRows) {
      sm.tok[tid] = t;
      sm.par[tid] = (int8_t)(bad ? 0 : p);
      const unsigned m = __ballot_sync(0xffffffffu, tid > 0 && tid < w.rows &&
                                                       (unsigned)(t - lo) < (unsigned)n);
      if (lane == 0) sm.mine[wid] = m;
    }
    for (int o = tid; o < kSlice / 4; o += kThreads)
      reinterpret_cast<uint4*>(sm.cnt)[o] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (first)
    for (int o = tid; o < kSlice / 4; o += kThreads)
      reinterpret_cast<uint4*>(s_first)[o] =
          make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
  if (__syncthreads_or(bad)) {
    if (tid == 0) flag(a.dev_status, SV_DEV_BAD_PARENT);
    return;
  }
  auto touch = [&](unsigned o) { atomicOr(&sm.bits[o >> 5], 1u << (o & 31)); };
  if (rule.pen) {
    const int32_t* h = ru.history + (size_t)i * ru.max_history;
    for (int t0 = 0; t0 < hlen; t0 += kThreads * kHistLoads) {
      int v[kHistLoads];
#pragma unroll
      for (int k = 0; k < kHistLoads; ++k) {
        const int t = t0 + k * kThreads + tid;
        v[k] = t < hlen ? __ldg(h + t) : -1;
      }
#pragma unroll
      for (int k = 0; k < kHistLoads; ++k) {
        const int t = t0 + k * kThreads + tid;
        const unsigned o = (unsigned)(v[k] - lo);
        if (v[k] >= 0 && o < (unsigned)n) {
          if (t < plen) atomicOr(&sm.cnt[o], kSeen);
          else atomicAdd(&sm.cnt[o], 1u);
          touch(o);
        }
      }
    }
    // the path of every row of this CTA, its nodes in the slice only
    if ((sm.mine[0] | sm.mine[1] | sm.mine[2] | sm.mine[3]) != 0) {
      if (tid < kMaxRows && (sm.mine[tid >> 5] >> (tid & 31) & 1u)) touch((unsigned)(sm.tok[tid] - lo));
      if (tid < rows) {
        unsigned m[kMaxRows / 32] = {};
        for (int p = j0 + tid; p > 0; p = sm.par[p]) {  // parents lie before their children
#pragma unroll
          for (int k = 0; k < kMaxRows / 32; ++k)
            if (p >> 5 == k) m[k] |= 1u << (p & 31);
        }
#pragma unroll
        for (int k = 0; k < kMaxRows / 32; ++k) sm.path[tid][k] = m[k] & sm.mine[k];
      }
    }
  }
  for (int t = b0 + tid; t < b1; t += kThreads) {
    const unsigned o = (unsigned)(ru.bias_token[t] - lo);
    if (o < (unsigned)n) {
      atomicMin(&s_first[o], (unsigned)(t - b0));
      touch(o);
    }
  }
  if (ru.mask) {
    for (int k = wid; k < rows; k += kWarps) {  // a warp for each row
      int m = ru.mask_row ? ru.mask_row[ra + k] : ra + k;
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
      if (lane == 0) sm.masked[k] = m;
    }
  }
  __syncthreads();
  const bool paths =
      rule.pen && (sm.mine[0] | sm.mine[1] | sm.mine[2] | sm.mine[3]) != 0;

  // ---- the rows ----
  // Adds d to the count of every node of row k's path in the slice.
  auto add_path = [&](int k, unsigned d) {
    if (tid < kMaxRows && (sm.path[k][tid >> 5] >> (tid & 31) & 1u))
      atomicAdd(&sm.cnt[sm.tok[tid] - lo], d);
  };
  auto on_path = [&](int k) {
    return (sm.path[k][0] | sm.path[k][1] | sm.path[k][2] | sm.path[k][3]) != 0;
  };
  int added = -1;  // the row whose path is in the counts
  for (int k = 0; k < rows; ++k) {
    if (paths) {  // the same for the whole CTA, as what follows
      const bool some = on_path(k);
      if (some || added >= 0) {
        __syncthreads();
        if (added >= 0) add_path(added, 0xffffffffu);
        if (some) add_path(k, 1u);
        added = some ? k : -1;
        __syncthreads();
      }
    }
    const T* src = static_cast<const T*>(a.logits) + (size_t)(ra + k) * a.stride + lo;
    float* dst = a.out + (size_t)(ra + k) * a.V + lo;
    const int m = ru.mask ? sm.masked[k] : -1;
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
  // rows of a CTA: as many of a request's as leave every SM eight CTAs
  const int nsm = num_sms();
  if (nsm < 1) return SV_ERR_CUDA;
  const long fair = (long)bt->total_rows * a.slices / ((long)nsm * 8);
  a.chunk = (int)max(4L, min((long)rul::kMaxChunk, fair));
  a.chunks = (bt->max_rows_per_req + a.chunk - 1) / a.chunk;
  const long ctas = (long)bt->n_req * a.chunks * a.slices;
  if (ctas > 0x7fffffffL) return SV_ERR_UNSUPPORTED_SHAPE;
  const size_t smem = rul::kBiasAt + (ru.bias_begin ? rul::kBiasBytes : 0);
  void (*kernel)(rul::Args) =
      logits_type == SV_LOGITS_F32
          ? (vec ? rul::rules_kernel<float, true> : rul::rules_kernel<float, false>)
          : (vec ? rul::rules_kernel<__nv_bfloat16, true> : rul::rules_kernel<__nv_bfloat16, false>);
  if (sv::launch(kernel, (unsigned)ctas, rul::kThreads, smem,
                 static_cast<cudaStream_t>(stream), a) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}
