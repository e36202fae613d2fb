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
// of a request but for their paths.  So a CTA takes a slice of the
// vocabulary and some rows of one request and first boils the request's rules
// down to shared memory: the history is counted (every CTA reads the whole
// history from L2 and keeps what falls in its slice: no workspace, no global
// atomics, no order that could change a result), and counts and biases become
// one addend per entry and one bit, "seen".  The rows then stream through
// registers, four entries at a time, each row loaded before the one before it
// is worked on; a warp whose 128 entries hold a touched one applies factor and
// addend to all of them without a branch (an untouched entry has addend 0),
// the others only pass theirs on.  The drafts of a row's path change the
// addends of their tokens before the row, which needs barriers only in the few
// slices that hold one.
//
// Measured (1280 rows of 151936, histories of 3450 tokens on average, 300
// biases, masks; floor 232 us at the copy rate): 270 us, 230 us without rules;
// 256 single rows of 128256 with 7750 tokens of history 78 us (floor 39).
// The same work with rules applied to touched entries alone under branches:
// 341; touched entries written over the copied rows: 439; rows passing through
// a shared-memory ring of bulk copies: 437 to 528, with warps specialised: 416;
// the history counted by eight CTAs through distributed shared memory: 360
// (the slice of the most frequent tokens takes 42 % of the remote updates).
// 783 rows of 50257 in bf16 under masks that permit 48 tokens: 58.9 us; barred
// entries written before the rules are prepared: 68.2; vectors that begin on
// 128 instead of 16 bytes of the output: 63.5.

#include "sv_internal.cuh"

namespace sv {
namespace rul {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4, kWideCtasPerSm = 3;
constexpr int kWarps = kThreads / 32;
// Vocabulary entries of a CTA: four quads a thread, or eight where requests
// have single rows.  Those need no registers for a next row, and half as many
// CTAs read each history (256 rows of 128256, 7750 tokens: fp32 78 us against
// 89, bf16 69 against 96; without a history bf16 35 against 41, fp32 with
// biases alone 55 against 53).  With more rows the next one's loads are worth
// more: 256 chains of five in bf16, each row loaded when its turn comes, 276 us
// against 183.
constexpr int kRowQuads = 4, kSingleQuads = 8;
template <int kQuads>
constexpr int kSliceOf = 4 * kThreads * kQuads;
constexpr int kMaxChunk = 9;    // rows of a CTA at most: a root and eight drafts
constexpr int kHistVecs = 3;    // vectors of four history tokens a thread has in flight (two: 272 us, four:
                                // 269 us but 256 single rows 97 instead of 89)

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

template <int kQuads>
struct Smem {
  static constexpr int kSlice = kSliceOf<kQuads>, kWords = kSlice / 32;
  union {
    unsigned cnt[kSlice];      // first occurrences and kDraft,
    float add[kSlice];         // then the addend
  };
  uint8_t asked[kSlice];       // 1: the token is in the prompt
  unsigned hit[kWords + 1];    // touched entries, a bit each (and a word for a look past the end)
  unsigned seen[kWords + 1];   // entries that the repetition penalty takes
  int tok[kMaxRows];
  int8_t par[kMaxRows];
  unsigned mine[kMaxRows / 32];             // nodes whose token is in the slice
  unsigned path[kMaxChunk][kMaxRows / 32];  // of those, the nodes on the row's path
  int masked[kMaxChunk];                    // the row's mask row, -1: none
  unsigned words[kQuads > kRowQuads ? 1 : kMaxChunk][kWords + 1];  // that mask's bits of the slice
};
// Behind it, with biases: the lowest list position of each token (in 16 bits
// for wide slices: 32 would leave room for two CTAs instead of three, 94 us
// instead of 78).
template <int kQuads>
struct FirstOf {
  using type = unsigned;
};
template <>
struct FirstOf<kSingleQuads> {
  using type = unsigned short;
};
__device__ __forceinline__ void first_min(unsigned* at, unsigned v) { atomicMin(at, v); }
__device__ __forceinline__ void first_min(unsigned short* at, unsigned v) {
  unsigned short old = *at;
  while (v < old) {  // *at falls with every turn but the last
    const unsigned short was = atomicCAS(at, old, (unsigned short)v);
    if (was == old) break;
    old = was;
  }
}
__device__ __forceinline__ void first_load(const unsigned* at, unsigned (&f)[4]) {
  const uint4 v = *reinterpret_cast<const uint4*>(at);
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
__device__ __forceinline__ void first_load(const unsigned short* at, unsigned (&f)[4]) {
  const ushort4 v = *reinterpret_cast<const ushort4*>(at);
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
template <int kQuads>
constexpr size_t kBiasAt = (sizeof(Smem<kQuads>) + 15) / 16 * 16;

constexpr unsigned kDraft = 0x80000000u;  // the token is some draft's

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
  __device__ __forceinline__ float4 get(bool) const { return x; }
};
struct Quad16 {
  uint32_t w[3];
  // alike: they lie together in 8 bytes; else the aligned words around them,
  // shifted into place when they are used (a shift here would wait for them).
  // A first half word before the input lies in the same four bytes as its
  // first entry; a last one behind it is not read.
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool alike, const void* end) {
    if (alike) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x;
      w[1] = u.y;
      return;
    }
    const uintptr_t lo = (uintptr_t)p & ~(uintptr_t)3;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(lo);
    w[0] = q[0];
    w[1] = q[1];
    if ((uintptr_t)p & 2) w[2] = lo + 12 <= (uintptr_t)end ? q[2] : *reinterpret_cast<const uint16_t*>(q + 2);
  }
  // odd: they start in the upper half of a word
  __device__ __forceinline__ float4 get(bool odd) const {
    const uint32_t w0 = odd ? __funnelshift_r(w[0], w[1], 16) : w[0];
    const uint32_t w1 = odd ? __funnelshift_r(w[1], w[2], 16) : w[1];
    return make_float4(__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u),
                       __uint_as_float(w1 << 16), __uint_as_float(w1 & 0xffff0000u));
  }
};
template <typename T>
struct QuadOf { using type = Quad32; };
template <>
struct QuadOf<__nv_bfloat16> { using type = Quad16; };

// Does mask row m permit anything?  By one warp; bits past the vocabulary do
// not count.
__device__ __forceinline__ bool any_permitted(const int32_t* m, int V) {
  const int lane = threadIdx.x & 31;
  const int words = (V + 31) >> 5;
  for (int w = 0; w < words; w += 32 * 8) {
    unsigned x = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int at = w + 32 * k + lane;
      if (at < words) {
        unsigned b = (unsigned)__ldg(m + at);
        if (at == words - 1 && (V & 31)) b &= (1u << (V & 31)) - 1u;
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

// EVEN: every row of the output starts on 16 bytes.  kQuads: kSingleQuads where
// each request has one row at most, else kRowQuads.
template <typename T, bool EVEN, int kQuads>
__global__ void __launch_bounds__(kThreads, kQuads > kRowQuads ? kWideCtasPerSm : kCtasPerSm)
    rules_kernel(Args a) {
  griddep_entry();
  constexpr int kSlice = kSliceOf<kQuads>, kWords = kSlice / 32;
  constexpr bool kSingle = kQuads > kRowQuads;
  extern __shared__ __align__(16) uint8_t s_raw[];
  Smem<kQuads>& sm = *reinterpret_cast<Smem<kQuads>*>(s_raw);
  using First = typename FirstOf<kQuads>::type;
  constexpr unsigned kNone = (First)~0u;
  First* s_first = reinterpret_cast<First*>(s_raw + kBiasAt<kQuads>);
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
  else if (!(rho >= 0x1p-126f && rho <= 0x1p126f) || !(fabsf(freq) < INFINITY) ||
           !(fabsf(pres) < INFINITY) || b0 < 0 || b1 < b0 || b1 > ru.n_bias)
    finding = SV_DEV_BAD_PARAM;
  else if (hlen < 0 || hlen > ru.max_history || plen < 0 || plen > hlen)
    finding = SV_DEV_BAD_LENGTH;
  // The request's rows are left as they were, and it is told apart from the
  // others (every CTA of it comes to the same end).
  auto refuse = [&](int why) {
    if (tid != 0) return;
    flag(a.dev_status, why);
    if (ru.row_end) ru.row_end[i] = 0;
  };
  if (finding) {
    refuse(finding);
    return;
  }
  const int j0 = w.b + chunk * a.chunk, j1 = min(w.e, j0 + a.chunk);  // this CTA's nodes
  if (j0 >= j1) return;
  const int ra = w.cu + j0, rows = j1 - j0;
  const bool rules = pen || b1 > b0;
  // In place, an unmasked row's untouched entries stay where they are, unless it
  // is the only one: loading it before it is known which they are is faster then
  // (256 single rows of 4096 entries a CTA: 90 us against 103).
  const bool lean = a.in_place && rows > 1;
  const T* src = static_cast<const T*>(a.logits) + (size_t)ra * a.stride + lo;
  float* dst = a.out + (size_t)ra * a.V + lo;

  // This thread's touched entries, four bits a quad: sixteen bits for each
  // place that a row can start at, or those of the one row.
  constexpr bool kOne = EVEN || kSingle;
  static_assert(4 * kQuads * (kOne ? 1 : 4) <= (kOne ? 32 : 64), "");
  uint64_t hits4 = 0;
  unsigned seen_own = 0;  // EVEN: its entries that the repetition penalty takes, paths apart
  auto hits_at = [&](int head) {
    return kOne ? (unsigned)hits4 : (unsigned)(hits4 >> (16 * head)) & 0xffffu;
  };
  // Each row is loaded (its mask's bits first) before the row before it is
  // worked on.
  using Quad = typename QuadOf<T>::type;
  struct Row {
    Quad x[kQuads];
    unsigned let;  // permitted entries, four bits a quad
    float edge;    // !EVEN: one of the entries that no 16 bytes of the output hold
    bool open;     // it is permitted
  };
  auto words_of = [&](int k) -> const unsigned* {
    return ru.mask && sm.masked[k] >= 0 ? sm.words[k] : nullptr;
  };
  // entries [head, head + mid) of the row at d start on 16 bytes of the output
  auto head_of = [&](const float* d) {
    return EVEN ? 0 : min(n, (int)((0u - (unsigned)((uintptr_t)d >> 2)) & 3u));
  };
  auto fetch = [&](int k, const T* s, const float* d, Row& row) {
    const unsigned* words = words_of(k);
    const int head = head_of(d), end = EVEN ? n : head + ((n - head) & ~3);
    row.let = 0xffffffffu;
    row.open = true;
    if (words) {
      row.let = 0u;
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        const int o = head + 4 * (q * kThreads + tid);
        if (o < end) row.let |= nibble(words, o) << (4 * q);
      }
    }
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const int o = head + 4 * (q * kThreads + tid);
      bool want = o < end && (row.let >> (4 * q) & 15u);
      if (lean && !words) want = want && (hits_at(head) >> (4 * q) & 15u);
      if (want) row.x[q].load(s + o, a.alike, a.logits_end);
    }
    if (!EVEN && tid < n - (end - head)) {
      const int o = tid < head ? tid : end - head + tid;
      const bool may = !words || (words[o >> 5] >> (o & 31) & 1u);
      if (may) row.edge = load1(s + o);
      else row.open = false;
    }
  };
  Row next;

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
  // (a negative token is a large offset)
  auto mine = [&](int v) { return (unsigned)v - (unsigned)lo < (unsigned)n; };
  if (rules) {
    for (int o = tid; o < kSlice / 4; o += kThreads) {
      reinterpret_cast<uint4*>(sm.cnt)[o] = make_uint4(0u, 0u, 0u, 0u);
      reinterpret_cast<uint32_t*>(sm.asked)[o] = 0u;
    }
    if (b1 > b0)
      for (int o = tid; o < kSlice * (int)sizeof(First) / 16; o += kThreads)
        reinterpret_cast<uint4*>(s_first)[o] =
            make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
    if (tid < kMaxRows) {
      sm.tok[tid] = node_t;
      sm.par[tid] = (int8_t)(bad ? 0 : node_p);
      const unsigned m = __ballot_sync(0xffffffffu, tid > 0 && tid < w.rows && mine(node_t));
      if (lane == 0) sm.mine[wid] = m;
    }
  }
  if (__syncthreads_or(bad)) {
    refuse(SV_DEV_BAD_PARENT);
    return;
  }
  if (ru.mask) {
    for (int k = wid; k < rows; k += kWarps) {  // a warp for each row
      const int m = sm.masked[k];
      if (m < 0) continue;
      const int32_t* mask = ru.mask + (size_t)m * ru.mask_stride;
      unsigned any = 0;
#pragma unroll
      for (int q = 0; q < kWords / 32; ++q) {
        const int at = 32 * q + lane;
        unsigned b = 32 * at < n ? (unsigned)__ldg(mask + (lo >> 5) + at) : 0u;
        if (n - 32 * at < 32 && 32 * at < n) b &= (1u << (n & 31)) - 1u;
        sm.words[k][at] = b;
        any |= b;
      }
      if (lane == 0) sm.words[k][kWords] = 0;
      // a mask that lets nothing through would leave no distribution
      if (!__any_sync(0xffffffffu, any != 0) && !any_permitted(mask, a.V) && lane == 0) {
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
      // a prompt's token leaves a mark (a plain store: all write the same),
      // an output's is counted
      auto mark = [&](int v) { if (mine(v)) sm.asked[v - lo] = 1; };
      auto count = [&](int v) { if (mine(v)) atomicAdd(&sm.cnt[v - lo], 1u); };
      auto take = [&](int t, int v) {
        if (t < plen) mark(v);
        else count(v);
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
          const int at = hhead + 4 * t;
          if (t >= hvecs) {
          } else if (at >= plen) {
            count(hv[q].x);
            count(hv[q].y);
            count(hv[q].z);
            count(hv[q].w);
          } else if (at + 4 <= plen) {
            mark(hv[q].x);
            mark(hv[q].y);
            mark(hv[q].z);
            mark(hv[q].w);
          } else {
            take(at, hv[q].x);
            take(at + 1, hv[q].y);
            take(at + 2, hv[q].z);
            take(at + 3, hv[q].w);
          }
          hv[q] = next[q];
        }
      }
      if (tid < hlen - 4 * hvecs) {  // what no whole vector holds
        const int t = tid < hhead ? tid : 4 * hvecs + tid;
        take(t, h[t]);
      }
      // the path of every row of this CTA, its nodes in the slice only
      paths = !kSingle && (sm.mine[0] | sm.mine[1] | sm.mine[2] | sm.mine[3]) != 0;
      if (paths) {
        if (tid > 0 && tid < w.rows && mine(node_t)) atomicOr(&sm.cnt[node_t - lo], kDraft);
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
    if (mine(btok)) first_min(&s_first[btok - lo], (unsigned)tid);
    for (int t = b0 + kThreads + tid; t < b1; t += kThreads) {
      const int v = ru.bias_token[t];
      if (mine(v)) first_min(&s_first[v - lo], (unsigned)(t - b0));
    }
  }
  __syncthreads();  // counts and mask bits are there
  // The first row's loads go out under what is left to do for the rules, unless
  // the rules say which entries to load.
  const bool early = !lean || words_of(0);
  if (early) fetch(0, src, dst, next);
  if (rules) {
    if (paths) {
      if (tid > 0 && tid < w.rows && mine(node_t)) {
        node_n = (int)(sm.cnt[node_t - lo] & ~kDraft);
        node_seen = node_n > 0 || sm.asked[node_t - lo];
        const unsigned f = b1 > b0 ? s_first[node_t - lo] : kNone;
        if (f != kNone) node_bias = ru.bias_value[b0 + (int)f];
      }
      __syncthreads();  // the counts become addends
    }
    const bool maps = !EVEN || paths;  // bit maps for all to read, or only this thread's own bits
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const int o = 4 * (q * kThreads + tid);
      const uint4 c = *reinterpret_cast<const uint4*>(sm.cnt + o);
      const uint32_t asked = *reinterpret_cast<const uint32_t*>(sm.asked + o);
      unsigned seen = 0, hit = 0;
      if (c.x | c.y | c.z | c.w) {
        const auto addend = [&](unsigned v) {
          const unsigned m = v & ~kDraft;
          return m ? -(freq * (float)m + pres) : 0.f;
        };
        *reinterpret_cast<float4*>(sm.add + o) =
            make_float4(addend(c.x), addend(c.y), addend(c.z), addend(c.w));
        seen = (c.x & ~kDraft ? 1u : 0u) | (c.y & ~kDraft ? 2u : 0u) | (c.z & ~kDraft ? 4u : 0u) |
               (c.w & ~kDraft ? 8u : 0u);
        hit = (c.x ? 1u : 0u) | (c.y ? 2u : 0u) | (c.z ? 4u : 0u) | (c.w ? 8u : 0u);
      }
      // the four bytes' marks as four bits
      const unsigned marks = (asked * 0x10204080u) >> 28;
      seen |= marks;
      hit |= marks;
      if (b1 > b0) {
        unsigned f[4];
        first_load(s_first + o, f);
        if ((f[0] & f[1] & f[2] & f[3]) != kNone)
          hit |= (f[0] != kNone ? 1u : 0u) | (f[1] != kNone ? 2u : 0u) | (f[2] != kNone ? 4u : 0u) |
                 (f[3] != kNone ? 8u : 0u);
      }
      if (EVEN) {
        hits4 |= (uint64_t)hit << (4 * q);
        seen_own |= seen << (4 * q);
      }
      if (maps) {
        // eight lanes' nibbles make a word
        seen <<= 4 * (lane & 7);
        hit <<= 4 * (lane & 7);
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
          seen |= __shfl_xor_sync(0xffffffffu, seen, d);
          hit |= __shfl_xor_sync(0xffffffffu, hit, d);
        }
        if ((lane & 7) == 0) {
          sm.seen[o >> 5] = seen;
          sm.hit[o >> 5] = hit;
        }
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
  if (rules) __syncthreads();
  auto on_path = [&](int k) {
    return (sm.path[k][0] | sm.path[k][1] | sm.path[k][2] | sm.path[k][3]) != 0;
  };
  const float inv = 1.f / rho;
  // y of touched entry o with value x
  auto shaped = [&](float x, float add, bool seen) {
    const float f = x > 0.f ? inv : rho;
    return fmaf(x, seen ? f : 1.f, add);
  };
  if (!EVEN && rules) {
    const int e0 = kSingle ? head_of(dst) : 0;
#pragma unroll
    for (int e = 0; e < (kSingle ? 1 : 4); ++e)
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        const int o = e0 + e + 4 * (q * kThreads + tid);
        if (o < n) hits4 |= (uint64_t)nibble(sm.hit, o) << (16 * e + 4 * q);
      }
  }

  // ---- the rows ----
  bool added = false;  // some row's path is in the addends
  if (!early) fetch(0, src, dst, next);
  for (int k = 0; k < rows; ++k, src += a.stride, dst += a.V) {
    Row row = next;
    if (!kSingle && k + 1 < rows) fetch(k + 1, src + a.stride, dst + a.V, next);
    const unsigned* words = words_of(k);
    const bool sparse = lean && !words;  // only touched entries change
    const int head = head_of(dst), end = EVEN ? n : head + ((n - head) & ~3);
    const bool odd = sizeof(T) == 2 && !a.alike && ((uintptr_t)(src + head) & 2);
    if (paths) {
      const bool some = on_path(k);
      if (some || added) {  // the same for the whole CTA
        __syncthreads();
        if (tid > 0 && tid < w.rows && mine(node_t)) {
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
    const unsigned hits = hits_at(head);
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const int o = head + 4 * (q * kThreads + tid);
      const unsigned let = row.let >> (4 * q) & 15u;
      const unsigned hit = hits >> (4 * q) & 15u;
      float4 x = row.x[q].get(odd);
      if (__any_sync(0xffffffffu, hit & let)) {
        if (o < end) {
          const unsigned seen = EVEN && !paths ? seen_own >> (4 * q) : nibble(sm.seen, o);
          float4 d;
          if (EVEN) d = *reinterpret_cast<const float4*>(sm.add + o);
          else d = make_float4(sm.add[o], sm.add[o + 1], sm.add[o + 2], sm.add[o + 3]);
          x.x = shaped(x.x, d.x, seen & 1u);
          x.y = shaped(x.y, d.y, seen & 2u);
          x.z = shaped(x.z, d.z, seen & 4u);
          x.w = shaped(x.w, d.w, seen & 8u);
        }
      }
      if (words) {
        if (!(let & 1u)) x.x = -INFINITY;
        if (!(let & 2u)) x.y = -INFINITY;
        if (!(let & 4u)) x.z = -INFINITY;
        if (!(let & 8u)) x.w = -INFINITY;
      }
      if (o < end && !(sparse && !hit)) *reinterpret_cast<float4*>(dst + o) = x;
    }
    const int rest = n - (end - head);
    if (!EVEN && tid < rest) {  // what no 16 bytes of the output hold
      const int o = tid < head ? tid : end - head + tid;
      float y = row.edge;
      if (rules) y = shaped(y, sm.add[o], sm.seen[o >> 5] >> (o & 31) & 1u);
      if (!row.open) y = -INFINITY;
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
  if (bt->max_rows_per_req > kMaxRows || vocab > 1 << 30) return SV_ERR_UNSUPPORTED_SHAPE;
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
  const long room = (long)nsm * rul::kCtasPerSm;
  const int wide = rul::kSliceOf<rul::kSingleQuads>;
  // Wide slices where they leave no place for a CTA empty.
  const bool single = ((pen && a.ru.max_history > 0) || esz == 2) && bt->max_rows_per_req == 1 &&
                      (!ru.bias_begin || ru.n_bias < 0xffff) &&
                      (long)bt->n_req * ((vocab + wide - 1) / wide) >= room;
  const int slice = single ? wide : rul::kSliceOf<rul::kRowQuads>;
  const int slices = (vocab + slice - 1) / slice;
  // Rows of a CTA: all of a request's up to kMaxChunk, unless that leaves places
  // for CTAs empty: a CTA's rows follow one another, its rules cost a few rows'
  // time.  (Eight chains with histories of 8000: one row a CTA 24 us, three 15;
  // sixteen trees of 33 to 65 rows: seventeen a CTA 71 us, nine 60.)
  const long fair = ((long)bt->total_rows * slices + room - 1) / room;
  const int most = (int)max(1L, min((long)rul::kMaxChunk, fair));
  a.chunks = (bt->max_rows_per_req + most - 1) / most;
  a.chunk = (bt->max_rows_per_req + a.chunks - 1) / a.chunks;
  const long units = (long)bt->n_req * a.chunks, ctas = units * slices;
  if (ctas > 0x7fffffffL) return SV_ERR_UNSUPPORTED_SHAPE;
  a.units = (int)units;
  const auto pick = [&](auto t) -> void (*)(rul::Args) {
    using T = decltype(t);
    if (single)
      return even ? rul::rules_kernel<T, true, rul::kSingleQuads>
                  : rul::rules_kernel<T, false, rul::kSingleQuads>;
    return even ? rul::rules_kernel<T, true, rul::kRowQuads>
                : rul::rules_kernel<T, false, rul::kRowQuads>;
  };
  const auto kernel = esz == 4 ? pick(0.f) : pick(__nv_bfloat16());
  size_t smem = single ? rul::kBiasAt<rul::kSingleQuads> : rul::kBiasAt<rul::kRowQuads>;
  if (ru.bias_begin) smem += slice * (single ? sizeof(unsigned short) : sizeof(unsigned));
  if (single) {
    static PerDevice limit[4];
    if (smem_limit_once(limit[2 * (esz == 4) + even], kernel,
                        rul::kBiasAt<rul::kSingleQuads> + wide * sizeof(unsigned short)) !=
        cudaSuccess)
      return SV_ERR_CUDA;
  }
  if (sv::launch(kernel, (unsigned)ctas, rul::kThreads, smem, static_cast<cudaStream_t>(stream),
                 a) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}
