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
// Bound: HBM, 4 bytes written and 2 or 4 read per logit; a barred logit need
// not be read, and in place an untouched one need not be moved.  Few tokens of
// a row are touched by a penalty or bias, and they are the same for all rows
// of a request but for their paths.  So a CTA takes kSlice entries of the
// vocabulary and some rows of one request and first boils the request's rules
// down to shared memory: the history is counted (every CTA reads the whole
// history from L2 and keeps what falls in its slice: no workspace, no global
// atomics, no order that could change a result), and counts and biases become
// one addend per entry and one bit, "seen".  The rows then stream through
// registers, four entries at a time; a warp whose 128 entries hold a touched
// one applies factor and addend to all of them without a branch (an untouched
// entry has addend 0), the others only pass theirs on.
// The drafts of a row's path change the addends of their tokens before the
// row, which needs barriers only in the few slices that hold one.

#include "sv_internal.cuh"

namespace sv {
namespace rul {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlice = 4096;    // vocabulary entries of a CTA
constexpr int kWords = kSlice / 32;
constexpr int kQuads = kSlice / (4 * kThreads);
constexpr int kMaxChunk = 32;   // rows of a CTA at most
constexpr int kHistVecs = 2;    // vectors of four history tokens a thread has in flight

struct Args {
  sv_batch bt;
  const void* logits;
  const void* logits_end;
  long stride;
  float* out;
  sv_logit_rules ru;
  int32_t* dev_status;
  int V, units, chunks, chunk;  // units: requests x chunks of `chunk` rows
  int in_place;
  int alike;  // input rows lie in four entries as the output's do
};

struct Smem {
  union {
    unsigned cnt[kSlice];      // first occurrences, kSeen and kDraft,
    float add[kSlice];         // then the addend
  };
  unsigned hit[kWords + 1];    // touched entries, a bit each (and a word for a look past the end)
  unsigned seen[kWords + 1];   // entries that the repetition penalty takes
  int tok[kMaxRows];
  int8_t par[kMaxRows];
  unsigned mine[kMaxRows / 32];             // nodes whose token is in the slice
  unsigned path[kMaxChunk][kMaxRows / 32];  // of those, the nodes on the row's path
  int masked[kMaxChunk];                    // the row's mask row, -1: none
};
// Behind it, with biases: the lowest list position of each token.
constexpr size_t kBiasAt = (sizeof(Smem) + 15) / 16 * 16;
constexpr size_t kBiasBytes = kSlice * sizeof(unsigned);

constexpr unsigned kSeen = 0x80000000u;   // the token is in the prompt
constexpr unsigned kDraft = 0x40000000u;  // the token is some draft's

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Four neighbours of a row as loaded, and as fp32.
struct Quad32 {
  float4 x;
  // alike: they lie together in 16 bytes
  __device__ __forceinline__ void load(const float* p, bool alike, const void*) {
    if (alike) x = *reinterpret_cast<const float4*>(p);
    else x = make_float4(p[0], p[1], p[2], p[3]);
  }
  __device__ __forceinline__ float4 get() const { return x; }
};
struct Quad16 {
  uint32_t w0, w1;
  // alike: they lie together in 8 bytes; else the aligned words around them
  // are shifted into place (entry by entry where those reach past the input)
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool alike, const void* end) {
    if (alike) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w0 = u.x;
      w1 = u.y;
      return;
    }
    const uintptr_t at = (uintptr_t)p, lo = at & ~(uintptr_t)3;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(lo);
    w0 = w[0];
    w1 = w[1];
    if (at == lo) return;
    const uint32_t w2 = lo + 12 <= (uintptr_t)end ? w[2] : *reinterpret_cast<const uint16_t*>(w + 2);
    w0 = __funnelshift_r(w0, w1, 16);
    w1 = __funnelshift_r(w1, w2, 16);
  }
  __device__ __forceinline__ float4 get() const {
    return make_float4(__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u),
                       __uint_as_float(w1 << 16), __uint_as_float(w1 & 0xffff0000u));
  }
};
template <typename T>
struct QuadOf { using type = Quad32; };
template <>
struct QuadOf<__nv_bfloat16> { using type = Quad16; };

// Does mask row m permit any of the entries [lo, lo + n)?  By one warp; bits
// past the vocabulary do not count.
__device__ __forceinline__ bool any_permitted(const int32_t* m, int lo, int n, int V) {
  const int lane = threadIdx.x & 31;
  const int w1 = (lo + n + 31) >> 5, last = (V - 1) >> 5;
  for (int w = lo >> 5; w < w1; w += 32 * 8) {
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

// Four bits of a bit map from entry o on.
__device__ __forceinline__ unsigned nibble(const unsigned* bits, int o) {
  unsigned b = bits[o >> 5] >> (o & 31);
  if ((o & 31) > 28) b |= bits[(o >> 5) + 1] << (32 - (o & 31));
  return b & 15u;
}

// EVEN: every row of the output starts on 16 bytes.
template <typename T, bool EVEN>
__global__ void __launch_bounds__(kThreads, 4) rules_kernel(Args a) {
  griddep_entry();
  extern __shared__ __align__(16) uint8_t s_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(s_raw);
  unsigned* s_first = reinterpret_cast<unsigned*>(s_raw + kBiasAt);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  // slices in order: the lowest token ids are the most frequent ones, and
  // counting them takes longest: their slices start first
  const int slice = (int)(blockIdx.x / (unsigned)a.units);
  const int unit = (int)(blockIdx.x % (unsigned)a.units);
  const int i = unit / a.chunks, chunk = unit % a.chunks;
  const int lo = slice * kSlice, n = min(kSlice, a.V - lo);
  const sv_logit_rules& ru = a.ru;

  // ---- the request: everything that only its number leads to, at once ----
  const Window w = window_of(a.bt, i);
  const float rho = ru.repetition ? ru.repetition[i] : 1.f;
  const float freq = ru.frequency ? ru.frequency[i] : 0.f;
  const float pres = ru.presence ? ru.presence[i] : 0.f;
  const int hlen = ru.history ? ru.history_len[i] : 0;
  const int plen = ru.history && ru.prompt_len ? ru.prompt_len[i] : 0;
  const int b0 = ru.bias_begin ? ru.bias_begin[i] : 0;
  const int b1 = ru.bias_begin ? ru.bias_begin[i + 1] : 0;
  const bool pen = rho != 1.f || freq != 0.f || pres != 0.f;
  int finding = 0;
  if (!w.ok)
    finding = SV_DEV_BAD_WINDOW;
  else if (!(rho > 0.f && rho < INFINITY) || !(fabsf(freq) < INFINITY) ||
           !(fabsf(pres) < INFINITY) || b0 < 0 || b1 < b0 || b1 > ru.n_bias)
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
  const bool rules = pen || b1 > b0;
  const T* src = static_cast<const T*>(a.logits) + (size_t)ra * a.stride + lo;
  float* dst = a.out + (size_t)ra * a.V + lo;

  // ---- its rules in shared memory ----
  // What these need is loaded before the first barrier: the tree (one node a
  // thread), the rows' mask numbers, the head of the history.
  const int32_t* h = ru.history + (size_t)i * ru.max_history;
  int hhead = 0, hvecs = 0;  // tokens before the aligned vectors, vectors
  int4 hv[kHistVecs];
  bool bad = false;
  int node_p = 0, node_t = -1;
  if (pen) {
    if (tid < w.rows) {
      node_p = a.bt.parent[w.cu + tid];
      node_t = a.bt.tokens[w.cu + tid];
      bad = tid == 0 ? node_p != -1 : (node_p < 0 || node_p >= tid);
    }
    if (hlen > 0) {
      hhead = min(hlen, (int)((0u - (unsigned)((uintptr_t)h >> 2)) & 3u));
      hvecs = (hlen - hhead) >> 2;
    }
#pragma unroll
    for (int q = 0; q < kHistVecs; ++q) {
      const int t = q * kThreads + tid;
      if (t < hvecs) hv[q] = __ldg(reinterpret_cast<const int4*>(h + hhead) + t);
    }
  }
  int btok = -1;
  float bval = 0.f;
  if (b0 + tid < b1) {
    btok = ru.bias_token[b0 + tid];
    bval = ru.bias_value[b0 + tid];
  }
  if (ru.mask && tid < rows) {
    int m = ru.mask_row ? ru.mask_row[ra + tid] : ra + tid;
    if (m < -1 || m >= ru.n_masks) {
      flag(a.dev_status, SV_DEV_BAD_PARAM);
      m = -1;
    }
    sm.masked[tid] = m;
  }
  auto mine = [&](int v) { return v >= 0 && (unsigned)(v - lo) < (unsigned)n; };
  if (rules) {
    for (int o = tid; o < kSlice / 4; o += kThreads)
      reinterpret_cast<uint4*>(sm.cnt)[o] = make_uint4(0u, 0u, 0u, 0u);
    if (b1 > b0)
      for (int o = tid; o < kSlice / 4; o += kThreads)
        reinterpret_cast<uint4*>(s_first)[o] =
            make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
    if (tid < kMaxRows) {
      sm.tok[tid] = node_t;
      sm.par[tid] = (int8_t)(bad ? 0 : node_p);
      const unsigned m = __ballot_sync(0xffffffffu, tid > 0 && mine(node_t));
      if (lane == 0) sm.mine[wid] = m;
    }
  }
  if (__syncthreads_or(bad)) {  // the request's rows are left as they were
    if (tid == 0) flag(a.dev_status, SV_DEV_BAD_PARENT);
    return;
  }
  if (ru.mask) {
    // a warp for each row: a mask that lets nothing through would leave no
    // distribution
    for (int k = wid; k < rows; k += kWarps) {
      const int m = sm.masked[k];
      if (m < 0) continue;
      const int32_t* words = ru.mask + (size_t)m * ru.mask_stride;
      if (!any_permitted(words, lo, n, a.V) && !any_permitted(words, 0, a.V, a.V) && lane == 0) {
        flag(a.dev_status, SV_DEV_EMPTY_MASK);
        sm.masked[k] = -1;
      }
    }
  }
  bool paths = false;
  int node_n = 0;         // the node's token: occurrences without the path,
  bool node_seen = false;
  float node_bias = 0.f;  // bias
  if (rules) {
    if (pen) {
      auto take = [&](int t, int v) {
        if (mine(v)) {
          if (t < plen) atomicOr(&sm.cnt[v - lo], kSeen);
          else atomicAdd(&sm.cnt[v - lo], 1u);
        }
      };
      for (int t0 = 0; t0 < hvecs; t0 += kThreads * kHistVecs) {
        int4 next[kHistVecs];
#pragma unroll
        for (int q = 0; q < kHistVecs; ++q) {  // the following round's loads
          const int t = t0 + (kHistVecs + q) * kThreads + tid;
          if (t < hvecs) next[q] = __ldg(reinterpret_cast<const int4*>(h + hhead) + t);
        }
#pragma unroll
        for (int q = 0; q < kHistVecs; ++q) {
          const int t = t0 + q * kThreads + tid;
          if (t < hvecs) {
            take(hhead + 4 * t, hv[q].x);
            take(hhead + 4 * t + 1, hv[q].y);
            take(hhead + 4 * t + 2, hv[q].z);
            take(hhead + 4 * t + 3, hv[q].w);
          }
          hv[q] = next[q];
        }
      }
      if (tid < hlen - 4 * hvecs) {  // what no whole vector holds
        const int t = tid < hhead ? tid : 4 * hvecs + tid;
        take(t, h[t]);
      }
      // the path of every row of this CTA, its nodes in the slice only
      paths = (sm.mine[0] | sm.mine[1] | sm.mine[2] | sm.mine[3]) != 0;
      if (paths) {
        if (tid > 0 && mine(node_t)) atomicOr(&sm.cnt[node_t - lo], kDraft);
        if (tid < rows) {
          unsigned m[kMaxRows / 32] = {};
          for (int p = j0 + tid; p > 0; p = sm.par[p]) {  // parents lie before their children
#pragma unroll
            for (int q = 0; q < kMaxRows / 32; ++q)
              if (p >> 5 == q) m[q] |= 1u << (p & 31);
          }
#pragma unroll
          for (int q = 0; q < kMaxRows / 32; ++q) sm.path[tid][q] = m[q] & sm.mine[q];
        }
      }
    }
    if (mine(btok)) atomicMin(&s_first[btok - lo], (unsigned)tid);
    for (int t = b0 + kThreads + tid; t < b1; t += kThreads) {
      const int v = ru.bias_token[t];
      if (mine(v)) atomicMin(&s_first[v - lo], (unsigned)(t - b0));
    }
    __syncthreads();
    if (paths) {
      if (tid > 0 && mine(node_t)) {
        const unsigned c = sm.cnt[node_t - lo];
        node_n = (int)(c & ~(kSeen | kDraft));
        node_seen = node_n > 0 || (c & kSeen);
        const unsigned f = b1 > b0 ? s_first[node_t - lo] : 0xffffffffu;
        if (f != 0xffffffffu) node_bias = ru.bias_value[b0 + (int)f];
      }
      __syncthreads();  // the counts become addends
    }
#pragma unroll
    for (int q = 0; q < kSlice / kThreads; ++q) {
      const int o = q * kThreads + tid;
      const unsigned c = sm.cnt[o];
      const int m = (int)(c & ~(kSeen | kDraft));
      const bool biased = b1 > b0 && s_first[o] != 0xffffffffu;
      sm.add[o] = m ? -(freq * (float)m + pres) : 0.f;
      const unsigned seen = __ballot_sync(0xffffffffu, m > 0 || (c & kSeen));
      const unsigned hit = __ballot_sync(0xffffffffu, c != 0u || biased);
      if (lane == 0) {
        sm.seen[o >> 5] = seen;
        sm.hit[o >> 5] = hit;
      }
    }
    if (tid == 0) sm.hit[kWords] = sm.seen[kWords] = 0;
    if (b1 > b0) {
      __syncthreads();
      // of a token's entries the first adds its value
      if (mine(btok) && s_first[btok - lo] == (unsigned)tid) sm.add[btok - lo] += bval;
      for (int t = b0 + kThreads + tid; t < b1; t += kThreads) {
        const int v = ru.bias_token[t];
        if (mine(v) && s_first[v - lo] == (unsigned)(t - b0)) sm.add[v - lo] += ru.bias_value[t];
      }
    }
  }
  __syncthreads();
  auto on_path = [&](int k) {
    return (sm.path[k][0] | sm.path[k][1] | sm.path[k][2] | sm.path[k][3]) != 0;
  };
  const float inv = 1.f / rho;
  // y of touched entry o with value x
  auto shaped = [&](float x, float add, bool seen) {
    const float y = x * (x > 0.f ? inv : rho);
    return (seen ? y : x) + add;
  };
  unsigned hits[kQuads] = {};  // EVEN: this thread's touched entries, the same in every row
  if (EVEN && rules) {
#pragma unroll
    for (int q = 0; q < kQuads; ++q) hits[q] = nibble(sm.hit, 4 * (q * kThreads + tid));
  }

  // ---- the rows ----
  // Each row is loaded (its mask's bits first) before the row before it is
  // worked on.
  using Quad = typename QuadOf<T>::type;
  struct Row {
    Quad x[kQuads];
    unsigned let;  // permitted entries, four bits a quad
  };
  auto words_of = [&](int k) {
    const int m = ru.mask ? sm.masked[k] : -1;
    return m >= 0 ? ru.mask + (size_t)m * ru.mask_stride + (lo >> 5) : nullptr;
  };
  // entries [head, head + mid) of the row at d start on 16 bytes of the output
  auto head_of = [&](const float* d) {
    return EVEN ? 0 : min(n, (int)((0u - (unsigned)((uintptr_t)d >> 2)) & 3u));
  };
  auto fetch = [&](int k, const T* s, const float* d, Row& row) {
    const int32_t* words = words_of(k);
    const int head = head_of(d), end = EVEN ? n : head + ((n - head) & ~3);
    row.let = 0xffffffffu;
    if (words) {
      row.let = 0;
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        const int o = head + 4 * (q * kThreads + tid);
        if (o < end) {
          const int wd = o >> 5;
          unsigned b = (unsigned)__ldg(words + wd) >> (o & 31);
          if (!EVEN && (o & 31) > 28) b |= (unsigned)__ldg(words + wd + 1) << (32 - (o & 31));
          row.let |= (b & 15u) << (4 * q);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const int o = head + 4 * (q * kThreads + tid);
      bool want = o < end && (row.let >> (4 * q) & 15u);
      if (a.in_place && !words) want = want && rules && (EVEN ? hits[q] : nibble(sm.hit, o));
      if (want) row.x[q].load(s + o, a.alike, a.logits_end);
    }
  };
  bool added = false;  // some row's path is in the addends
  Row next;
  fetch(0, src, dst, next);
  for (int k = 0; k < rows; ++k, src += a.stride, dst += a.V) {
    Row row = next;
    if (k + 1 < rows) fetch(k + 1, src + a.stride, dst + a.V, next);
    const int32_t* words = words_of(k);
    const bool sparse = a.in_place && !words;  // only touched entries change
    const int head = head_of(dst), end = EVEN ? n : head + ((n - head) & ~3);
    if (paths) {
      const bool some = on_path(k);
      if (some || added) {  // the same for the whole CTA
        __syncthreads();
        if (tid > 0 && mine(node_t)) {
          // (nodes with the same token write the same)
          int c = node_n;
          for (int q = 0; q < kMaxRows / 32; ++q)
            for (unsigned b = sm.path[k][q]; b; b &= b - 1)
              c += sm.tok[32 * q + __ffs(b) - 1] == node_t;
          const int o = node_t - lo;
          sm.add[o] = node_bias - (c ? freq * (float)c + pres : 0.f);
          if (node_seen || c) atomicOr(&sm.seen[o >> 5], 1u << (o & 31));
          else atomicAnd(&sm.seen[o >> 5], ~(1u << (o & 31)));
        }
        added = some;
        __syncthreads();
      }
    }
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const int o = head + 4 * (q * kThreads + tid);
      const unsigned let = row.let >> (4 * q) & 15u;
      const unsigned hit = !rules ? 0u : EVEN ? hits[q] : o < end ? nibble(sm.hit, o) : 0u;
      float4 x = row.x[q].get();
      if (__any_sync(0xffffffffu, hit & let)) {
        if (o < end) {
          const unsigned seen = nibble(sm.seen, o);
          float4 d;
          if (EVEN) d = *reinterpret_cast<const float4*>(sm.add + o);
          else d = make_float4(sm.add[o], sm.add[o + 1], sm.add[o + 2], sm.add[o + 3]);
          x.x = shaped(x.x, d.x, seen & 1u);
          x.y = shaped(x.y, d.y, seen & 2u);
          x.z = shaped(x.z, d.z, seen & 4u);
          x.w = shaped(x.w, d.w, seen & 8u);
        }
      }
      if (!(let & 1u)) x.x = -INFINITY;
      if (!(let & 2u)) x.y = -INFINITY;
      if (!(let & 4u)) x.z = -INFINITY;
      if (!(let & 8u)) x.w = -INFINITY;
      if (o < end && !(sparse && !hit)) *reinterpret_cast<float4*>(dst + o) = x;
    }
    const int rest = n - (end - head);
    if (!EVEN && tid < rest) {  // what no 16 bytes of the output hold
      const int o = tid < head ? tid : end - head + tid;
      const bool may = !words || ((unsigned)__ldg(words + (o >> 5)) >> (o & 31) & 1u);
      float y = -INFINITY;
      if (may) {
        y = load1(src + o);
        if (rules) y = shaped(y, sm.add[o], sm.seen[o >> 5] >> (o & 31) & 1u);
      }
      dst[o] = y;
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
  a.in_place = same ? 1 : 0;
  a.logits_end = reinterpret_cast<const void*>(in_end);
  a.alike = ((in / esz - to / 4) & 3) == 0 &&
            (bt->total_rows == 1 || (logits_stride - vocab) % 4 == 0);
  const bool even = (to & 15) == 0 && vocab % 4 == 0;
  const int nsm = num_sms();
  if (nsm < 1) return SV_ERR_CUDA;
  const int slices = (vocab + rul::kSlice - 1) / rul::kSlice;
  // rows of a CTA: all of a request's, unless that leaves room for more CTAs
  const long fair = (long)bt->total_rows * slices / ((long)nsm * 6);
  a.chunk = (int)max(1L, min((long)rul::kMaxChunk, fair));
  a.chunks = (bt->max_rows_per_req + a.chunk - 1) / a.chunk;
  const long units = (long)bt->n_req * a.chunks, ctas = units * slices;
  if (ctas > 0x7fffffffL) return SV_ERR_UNSUPPORTED_SHAPE;
  a.units = (int)units;
  const size_t smem = rul::kBiasAt + (ru.bias_begin ? rul::kBiasBytes : 0);
  void (*const kernel)(rul::Args) =
      esz == 4 ? (even ? rul::rules_kernel<float, true> : rul::rules_kernel<float, false>)
               : (even ? rul::rules_kernel<__nv_bfloat16, true>
                       : rul::rules_kernel<__nv_bfloat16, false>);
  if (sv::launch(kernel, (unsigned)ctas, rul::kThreads, smem, static_cast<cudaStream_t>(stream),
                 a) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}
