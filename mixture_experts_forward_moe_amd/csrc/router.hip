// router.hip -- the router of an MoE layer: the choice of top_k experts per
// token with their routing weights, the load-balancing loss of a routing, and
// the gradient of the logits from both.
//
// Score s of logit l: exp(l) / sum exp(l), or 1 / (1 + exp(-l)).  The choice
// goes by the logit, or by score + select_bias in fp64 (so that it does not
// hang on how an fp32 score rounds).  Loss, over T tokens:
//   coef E sum_e f_e P_e,  f_e = n_e / (T k),  P_e = sum_t p_te / T
//   d logit_e = p_e (u_e - sum u p) [(1 - s_e) for sigmoid],  u_e = coef E / T (f_e - 1 / E)
//
// One DPP row of 16 lanes owns a token: lane j holds the logits 64 c + 4 j ..
// + 3 (16-byte loads, 256 bytes a row of lanes; up to 64 experts one logit in
// 16 instead), so a maximum or a sum over the experts is a loop over a lane's
// registers and four DPP steps, and a wavefront serves four tokens with each
// instruction.
//
// The choice: the k-th largest of the (half) lanes' maxima bounds the k-th key
// from below, and only keys above the bound (about nine of 256 for k = 8) go
// on, one to a lane, where each lane counts the ones before its own.  The
// k rounds of maximum and removal that this replaces cost five instructions a
// register and round; they stay for k > 16 and for rows where more than 32
// keys pass (many equal ones).  score + bias is compared in fp32 first, and in
// fp64 for a token any two of whose candidates are closer than the error of
// that.
//
// Bound: up to some thousand tokens by latency (8 tokens of 256 experts: 4.7 us,
// a kernel of that length has a launch, one trip to memory and the chain of
// the choice).  From there on the choice without a bias by instructions, 640 a
// wavefront of four tokens (65536 x 256: 22.3 us fp32, 71 MB, 3.2 TB/s; 21 - 22
// bf16).  The others wait for memory as well:
// - with a bias (38 - 41 us; 8 tokens 6.4 - 6.7) a lane's biases are asked for
//   once the logits have come, and the chosen logits are read again;
// - with the loss (39 us; 16384 x 256: 19.6, of which the join is 7) the join
//   takes 16 bytes of each line, and reads every line eight times;
// - the gradient (39 us fp32, 138 MB, 3.5 TB/s; 32 bf16; 16384 x 256: 14.2, of the
//   weights alone 8.8) loads a lane's values of prob_grad one after another
//   before its first token, and its ids before their logits;
// - bf16 rows, and rows that are not whole groups of four, wait for each group
//   of 64 logits before they ask for the next.
// Equal logits, of which every one is a candidate, go by rounds: 111 us.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "device_common.h"
#include "internal.h"

namespace moe {

namespace {

// Threads, and tokens at a time.  With statistics 512 threads: a workgroup's
// partial sums are joined later, so there are at most 512 workgroups, and 256
// threads each would leave two wavefronts a SIMD.
constexpr int threads_of(bool stats) { return stats ? 512 : 256; }
constexpr int RT = 256, TOKENS = RT / 16;  // of the backward pass
constexpr int STAT_TOKENS = threads_of(true) / 16, STAT_BLOCKS = 512;  // of the statistics

template <int CTRL>
DEV int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
DEV float dpp(float v) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, v)));
}
template <int CTRL>
DEV double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)dpp<CTRL>((int)(uint32_t)b), hi = (uint32_t)dpp<CTRL>((int)(uint32_t)(b >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// the value d lanes before in the row (0x110 + d), 0 in front of the first
template <int CTRL>
DEV int dpp_zero(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, false);
}

// a reduction over the 16 lanes of a token
template <typename T, typename F>
DEV T row_reduce(T v, F f) {
  v = f(v, dpp<DPP_XOR1>(v));
  v = f(v, dpp<DPP_XOR2>(v));
  v = f(v, dpp<DPP_HALF_MIRROR>(v));
  return f(v, dpp<DPP_MIRROR>(v));
}
template <typename T>
DEV T row_max(T v) {
  return row_reduce(v, [](T a, T b) { return a > b ? a : b; });
}
template <typename T>
DEV T row_min(T v) {
  return row_reduce(v, [](T a, T b) { return a < b ? a : b; });
}
template <typename T>
DEV T row_add(T v) {
  return row_reduce(v, [](T a, T b) { return a + b; });
}

// A copy of v that the compiler cannot see through: what a token's work derives
// from the lane's number is made anew for each token instead of being kept in
// registers over all of them (which cost a third of the wavefronts).
DEV int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// NaN and -inf: not choosable; +inf counts as FLT_MAX
DEV float clean(float l) { return l == l ? fminf(l, FLT_MAX) : -INFINITY; }

// expert of register i of lane j, of V
template <int V>
DEV int expert_of(int i, int j) {
  return V == 4 ? 16 * i + j : (i >> 2) * 64 + 4 * j + (i & 3);
}

// e^x for x <= 0 to about one step: the product with log2(e) is carried in two
// parts into the hardware's exp2; below the normal range, and for the NaN of
// -inf - -inf, 0
DEV float exp_neg(float x) {
  x = fmaxf(x, -200.0f);
  const float t = x * 1.44269502f;
  const float e = fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269502f, -t));
  const float p = __builtin_amdgcn_exp2f(t);
  return fmaf(p, e * 0.693147182f, p);
}

// logits of a row; -inf past E.  vec: rows of whole, aligned groups of four.
// Groups of 64 experts that the row fills are loaded without a test; in the
// last one a lane past the end reads the row's last ones again.
template <int V, bool F32>
DEV void load_row_as(const void* logits, int64_t at, int E, int j, bool vec, float (&l)[V]) {
  constexpr int G = V == 4 ? 1 : V / 4;  // groups of 64
  const float* f = reinterpret_cast<const float*>(logits) + (F32 ? at : 0);
  const uint16_t* h = reinterpret_cast<const uint16_t*>(logits) + (F32 ? 0 : at);
  auto one = [&](int e) {
    if constexpr (F32) return f[e];
    else return bf16_to_f32(h[e]);
  };
#pragma unroll
  for (int c = 0; c < G; c++) {
    const bool full = 64 * (c + 1) <= E;
    if (V > 4 && vec) {
      const int e = full ? expert_of<V>(4 * c, j) : min(expert_of<V>(4 * c, j), E - 4);
      if constexpr (F32) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(f + e);
#pragma unroll
        for (int i = 0; i < 4; i++) l[4 * c + i] = v[i];
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(h + e);
        l[4 * c] = __uint_as_float(v.x << 16);
        l[4 * c + 1] = __uint_as_float(v.x & 0xffff0000u);
        l[4 * c + 2] = __uint_as_float(v.y << 16);
        l[4 * c + 3] = __uint_as_float(v.y & 0xffff0000u);
      }
    } else if (full) {
#pragma unroll
      for (int i = 0; i < 4; i++) l[4 * c + i] = one(expert_of<V>(4 * c + i, j));
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) l[4 * c + i] = one(min(expert_of<V>(4 * c + i, j), E - 1));
    }
  }
#pragma unroll
  for (int c = 0; c < G; c++) {
#pragma unroll
    for (int i = 0; i < 4; i++) l[4 * c + i] = clean(l[4 * c + i]);
    if (64 * (c + 1) > E) {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (expert_of<V>(4 * c + i, j) >= E) l[4 * c + i] = -INFINITY;
    }
  }
}
template <int V>
DEV void load_row(const void* logits, int f32, int64_t at, int E, int j, bool vec, float (&l)[V]) {
  if (f32) load_row_as<V, true>(logits, at, E, j, vec, l);
  else load_row_as<V, false>(logits, at, E, j, vec, l);
}

// sigmoid and 1 - sigmoid: with z = e^-|l|, 1 / (1 + z) and z / (1 + z)
DEV float sigmoid_f32(float l) {
  const float z = exp_neg(-fabsf(l));
  return (l < 0.0f ? z : 1.0f) * __builtin_amdgcn_rcpf(1.0f + z);
}

// Probabilities of a row: the softmax, or the sigmoid scores over their sum.
// Both are taken relative to the largest logit, so that a row of very
// negative logits does not become 0 / 0: s = exp(min(l, 0)) / (1 + exp(-|l|)),
// and the factor exp(-min(max, 0)) cancels in the quotient (it is 1 unless
// every logit of the row is negative).  Returns the reciprocal of the sum, the
// softmax's largest probability.
template <int V>
DEV float probabilities(const float (&l)[V], float top, int sigmoid, float (&p)[V]) {
  float sum = 0.0f;
  if (!sigmoid) {
#pragma unroll
    for (int i = 0; i < V; i++) p[i] = exp_neg(l[i] - top);
  } else if (__all(top >= 0.0f)) {
#pragma unroll
    for (int i = 0; i < V; i++) p[i] = sigmoid_f32(l[i]);
  } else {
    const float ref = fminf(top, 0.0f);
#pragma unroll
    for (int i = 0; i < V; i++) {
      const float e = exp_neg(fminf(l[i], 0.0f) - ref) * __builtin_amdgcn_rcpf(1.0f + exp_neg(-fabsf(l[i])));
      p[i] = l[i] == -INFINITY ? 0.0f : e;
    }
  }
#pragma unroll
  for (int i = 0; i < V; i++) sum += p[i];
  sum = row_add(sum);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < V; i++) p[i] *= inv;
  return inv;
}

// Score of a chosen logit before the division by the sum over the chosen
// (renormalize), relative to the largest chosen one as in probabilities()
DEV float chosen_score(float l, float top, int sigmoid) {
  if (l == -INFINITY) return 0.0f;
  if (!sigmoid) return exp_neg(l - top);
  return exp_neg(fminf(l, 0.0f) - fminf(top, 0.0f)) / (1.0f + exp_neg(-fabsf(l)));
}

constexpr int SLOTS = ROUTER_MAX_TOP_K / 16;  // chosen places a lane holds: j, j + 16, ...

// A key as an integer of the same order (no NaN, -0 as 0).
DEV uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// What a lane holds of a choice: expert and logit of places place[q]
struct Chosen {
  int id[SLOTS], place[SLOTS];
  float l[SLOTS];
};

// A logit of the row that starts at element `at`.
DEV float logit(const RouterParams& a, int64_t at, int e) {
  return clean(a.logits_f32 ? reinterpret_cast<const float*>(a.logits)[at + e]
                            : bf16_to_f32(reinterpret_cast<const uint16_t*>(a.logits)[at + e]));
}

// The key in fp64 of expert e with logit l: score + bias.  sum: sum_f64 of the
// row (SOFTMAX).
DEV double key_f64(const RouterParams& a, float l, int e, float top, double sum) {
  const double d = (double)l;
  return (a.sigmoid ? 1.0 / (1.0 + exp(-d)) : exp(d - (double)top) / sum) + (double)a.select_bias[e];
}
DEV double sum_f64(const RouterParams& a, int64_t at, float top, int j) {
  if (a.sigmoid) return 1.0;
  double sum = 0.0;
#pragma unroll 1
  for (int e = j; e < a.E; e += 16) {
    const float l = logit(a, at, e);
    if (l != -INFINITY) sum += exp((double)l - (double)top);
  }
  return row_add(sum);
}

// The choice by candidates (see above) of the wavefront's four tokens, up to 16
// experts each: the number of slots used, one candidate a lane or two (17 to 32
// of them).  key: the logits, or with BIAS fp32 forms of the keys, each off by
// at most err + 2^-23 |key|; where two candidates are closer than that the
// candidates' keys are compared in fp64.  rounds: in, the token counts (nothing
// is chosen for one that does not); out, it has more candidates and goes the
// other way.  Each token by itself, so that what it gets does not hang on its
// neighbours.
template <int V, bool BIAS>
DEV int choose_candidates(const RouterParams& a, int64_t at_row, float top, const float (&key)[V], float err, int j,
                           uint2* cand, Chosen& c, bool& rounds) {
  const int k = a.top_k;
  // A lower bound of the k-th key: the k-th largest of the maxima of half lanes
  // (the least of those with fewer than k above them; of 256 random keys 9 pass
  // for k = 8), or of whole lanes, for which a third of the instructions do, where
  // k is below 8: 8.7 keys pass for k = 7, more than 16 for 0.05% of the rows,
  // but 10.4 and 0.9% for k = 8, a quarter of the rows for k = 10 (65536 x 60, k
  // = 4: 11.4 us against 14.0 with half lanes; 4096 x 256, k = 8: 6.4 against
  // 5.1).  Up to 128 experts only: with both in one kernel the larger ones lose 4%
  // for k = 8 (65536 x 256: 23.7 us against 22.6).
  float ma = key[0], mb = key[V / 2];
#pragma unroll
  for (int i = 1; i < V / 2; i++) {
    ma = fmaxf(ma, key[i]);
    mb = fmaxf(mb, key[V / 2 + i]);
  }
  float bound;
  if (V <= 8 && k <= 7) {
    ma = fmaxf(ma, mb);
    int na = 0;
#define ROTATE(R) na += dpp<0x120 + R>(ma) > ma;
    ROTATE(1) ROTATE(2) ROTATE(3) ROTATE(4) ROTATE(5) ROTATE(6) ROTATE(7) ROTATE(8) ROTATE(9) ROTATE(10) ROTATE(11)
    ROTATE(12) ROTATE(13) ROTATE(14) ROTATE(15)
#undef ROTATE
    bound = na < k ? ma : INFINITY;
  } else {
    int na = mb > ma, nb = ma > mb;
#define ROTATE(R)                                                     \
  {                                                                   \
    const float oa = dpp<0x120 + R>(ma), ob = dpp<0x120 + R>(mb);     \
    na += (oa > ma) + (ob > ma);                                      \
    nb += (oa > mb) + (ob > mb);                                      \
  }
    ROTATE(1) ROTATE(2) ROTATE(3) ROTATE(4) ROTATE(5) ROTATE(6) ROTATE(7) ROTATE(8) ROTATE(9) ROTATE(10) ROTATE(11)
    ROTATE(12) ROTATE(13) ROTATE(14) ROTATE(15)
#undef ROTATE
    bound = fminf(na < k ? ma : INFINITY, nb < k ? mb : INFINITY);
  }
  // What the errors can hide below it: k keys are at least `bound`, so the k-th
  // true one is at least bound - err - 2^-24 |bound| (the error that the addition
  // makes, half of what is allowed for), and a key that reaches that is at least
  // bound - 2 err - 2^-22 |bound|.  Keys far below, such as those of a bias that
  // takes an expert out, have no part in it, whatever their own error.
  bound = row_min(bound);
  if (BIAS) bound -= 2.0f * (err + 0x1p-23f * fabsf(bound));
  bound = fmaxf(bound, -FLT_MAX);  // (-inf is no candidate)
  // candidates of this lane, and of the lanes before it
  int n = 0;
#pragma unroll
  for (int i = 0; i < V; i++) n += key[i] >= bound;
  int at = n;
  at += dpp_zero<0x111>(at);
  at += dpp_zero<0x112>(at);
  at += dpp_zero<0x114>(at);
  at += dpp_zero<0x118>(at);
  int total = __shfl(at, 15, 16);
  const bool counts = rounds;
  rounds = counts && total > 32;
  if (!counts || rounds) {  // (nothing is >= NaN: no key passes, not +inf either)
    total = 0;
    bound = __builtin_nanf("");
  }
  at -= n;
#pragma unroll
  for (int i = 0; i < V; i++) {
    if (key[i] >= bound) {
      cand[at] = make_uint2(__float_as_uint(key[i]), (uint32_t)expert_of<V>(i, j));
      at++;
    }
  }
  wave_fence();
  const bool two = __any(total > 16);
  const bool have = j < total, have2 = j + 16 < total;
  const uint2 own = have ? cand[j] : make_uint2(0u, 0u), own2 = have2 ? cand[j + 16] : make_uint2(0u, 0u);
  wave_fence();
  const float v = __uint_as_float(own.x), v2 = __uint_as_float(own2.x);
  const int e = have ? (int)own.y : INT32_MAX, e2 = have2 ? (int)own2.y : INT32_MAX;
  // places by descending key, then ascending expert
  int rank = 0, rank2 = 0;
  bool exactly = BIAS && two;
  if (!two) {
    const uint32_t hi = have ? ordered(v) : 0u, lo = ~(uint32_t)e;
    // (all lanes take part in each rotation: one that a condition had switched
    // off would be read as 0)
    bool close = false;
    const float apart = 2.0f * (err + 0x1p-23f * fabsf(v));  // (each of a pair looks: the larger error counts)
#define ROTATE(R)                                                                                        \
  {                                                                                                      \
    const uint32_t h2 = (uint32_t)dpp<0x120 + R>((int)hi), l2 = (uint32_t)dpp<0x120 + R>((int)lo);        \
    rank += (((uint64_t)h2 << 32) | l2) > (((uint64_t)hi << 32) | lo);                                   \
    if (BIAS) {                                                                                          \
      const float o = dpp<0x120 + R>(v);                                                                 \
      close |= have && h2 != 0u && fabsf(o - v) <= apart;                                                \
    }                                                                                                    \
  }
    ROTATE(1) ROTATE(2) ROTATE(3) ROTATE(4) ROTATE(5) ROTATE(6) ROTATE(7) ROTATE(8) ROTATE(9) ROTATE(10) ROTATE(11)
    ROTATE(12) ROTATE(13) ROTATE(14) ROTATE(15)
#undef ROTATE
    if (BIAS) exactly = __any(close);
  }
  if (two || exactly) {
    typedef typename std::conditional<BIAS, double, float>::type K;
    K x = -INFINITY, y = -INFINITY;
    if constexpr (BIAS) {
      const double sum = sum_f64(a, at_row, top, j);
      if (have) x = key_f64(a, logit(a, at_row, e), e, top, sum);
      if (have2) y = key_f64(a, logit(a, at_row, e2), e2, top, sum);
    } else {
      if (have) x = v;
      if (have2) y = v2;
    }
    auto before = [](K a, int ea, K b, int eb) { return (int)(a > b || (a == b && ea < eb)); };
    rank = before(y, e2, x, e);
    rank2 = before(x, e, y, e2);
#pragma unroll 1
    for (int s = 1; s < 16; s++) {
      // (lane j + s of the row; rarely taken, so small rather than fast)
      const int from = (j + s) & 15;
      const K ox = __shfl(x, from, 16), oy = __shfl(y, from, 16);
      const int ex = __shfl(e, from, 16), ey = __shfl(e2, from, 16);
      rank += before(ox, ex, x, e) + before(oy, ey, x, e);
      rank2 += before(ox, ex, y, e2) + before(oy, ey, y, e2);
    }
  }
  c.id[0] = have ? e : -1;
  c.place[0] = have ? rank : j;
  c.l[0] = have ? v : -INFINITY;  // (without a bias, the logit)
  c.id[1] = have2 ? e2 : -1;
  c.place[1] = have2 ? rank2 : j + 16;
  c.l[1] = have2 ? v2 : -INFINITY;
  return two ? 2 : 1;
}

// The choice by k rounds of maximum and removal, the row read again in each
// (it is in the first-level cache; registers for it would halve the wavefronts
// of the other way).  Lane j looks at the experts j, j + 16, .. and gets places
// j, j + 16, .., which c holds with no expert before.
template <bool BIAS>
DEV void choose_rounds(const RouterParams& a, int64_t at_row, float top, int j, Chosen& c) {
  uint64_t taken = 0;
  const double sum = BIAS ? sum_f64(a, at_row, top, j) : 1.0;
#pragma unroll 1
  for (int s = 0; s < a.top_k; s++) {
    // the largest key; of equal ones the lowest expert
    typename std::conditional<BIAS, double, float>::type best = -INFINITY;
    int e = INT32_MAX;
#pragma unroll 2
    for (int x = j; x < a.E; x += 16) {
      const float l = logit(a, at_row, x);
      if (l == -INFINITY || (taken >> (x >> 4) & 1)) continue;
      decltype(best) v;
      if constexpr (BIAS) v = key_f64(a, l, x, top, sum);
      else v = l;
      if (v > best) {  // (not for NaN)
        best = v;
        e = x;
      }
    }
    const auto win = row_max(best);
    e = row_min(best == win ? e : INT32_MAX);
    const bool any = win > -INFINITY;
    if (any && (e & 15) == j) taken |= (uint64_t)1 << (e >> 4);
    if (any && (s & 15) == j) {
#pragma unroll
      for (int q = 0; q < SLOTS; q++)
        if (q == s >> 4) c.id[q] = e;
    }
  }
}

template <int V, bool SELECT, bool BIAS, bool STATS>
__global__ __launch_bounds__(threads_of(STATS)) void router_kernel(const RouterParams a, bool vec) {
  constexpr int RT = threads_of(STATS), TOKENS = RT / 16;
  __shared__ int counts[STATS ? 16 * V : 1];
  __shared__ float psums[STATS ? RT / 64 : 1][STATS ? 16 * V : 1];
  __shared__ int tokens;
  __shared__ uint2 cand[SELECT ? TOKENS : 1][32];
  float psum[STATS ? V : 1];
  int seen = 0;
  if constexpr (STATS) {
    for (int e = threadIdx.x; e < 16 * V; e += RT) counts[e] = 0;
    if (threadIdx.x == 0) tokens = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
#pragma unroll
    for (int i = 0; i < V; i++) psum[i] = 0.0f;
    __syncthreads();
  }
  for (int64_t t0 = (int64_t)blockIdx.x * TOKENS; t0 < a.M; t0 += (int64_t)gridDim.x * TOKENS) {
    const int j = opaque(threadIdx.x & 15);
    const int64_t t = t0 + (threadIdx.x >> 4);
    const bool in = t < a.M;
    const bool on = in && (!a.token_mask || a.token_mask[t] != 0);
    const int64_t row = in ? t : a.M - 1;  // (lanes past the end stay: they take part in nothing but DPP)
    float l[V];
    load_row<V>(a.logits, a.logits_f32, row * a.row_stride, a.E, j, vec, l);
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; i++) top = fmaxf(top, l[i]);
    top = row_max(top);

    float p[STATS ? V : 1], most = 0.0f;  // (the softmax's largest probability)
    if constexpr (STATS) {
      most = probabilities<V>(l, top, a.sigmoid, p);
      if (on) {
#pragma unroll
        for (int i = 0; i < V; i++) psum[i] += p[i];
        seen += j == 0;
      }
    }

    Chosen c;
    if constexpr (SELECT) {
      const int64_t at_row = row * a.row_stride;
      float sum = 0.0f;  // of the scores' numerators: over all experts, or over the chosen ones
      if (!a.renormalize && !a.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; i++) sum += exp_neg(l[i] - top);
      }
      int used = (a.top_k + 15) / 16;
      bool rounds = on;  // this token's choice goes by rounds
#pragma unroll
      for (int q = 0; q < SLOTS; q++) {
        c.id[q] = -1;
        c.place[q] = j + 16 * q;
      }
      uint2* own_cand = cand[threadIdx.x >> 4];
      if constexpr (BIAS) {
        // Scores are off by, in steps of 2^-24: a sigmoid, 8 of the row's largest
        // (exp2 and rcp one of 2^-23 each, 1 + z and the product a half).  A softmax
        // V + 24 of its largest: V + 4 additions, 4 for exp, quotient and
        // product, and what the rounding of d = l - top does to the exp, |d| each,
        // of which a probability's |d| e^d is less than one and the sum's mean
        // at most ln E < 7.  The addition rounds relative to the key.  Scores below
        // fp32's normal range are 0: 2^-126 more.
        if (!a.sigmoid) {
          if constexpr (STATS) {
#pragma unroll
            for (int i = 0; i < V; i++) p[i] = l[i] == -INFINITY ? -INFINITY : p[i];
#pragma unroll
            for (int i = 0; i < V; i++) l[i] = p[i];
          } else {
            float q[V];
            most = probabilities<V>(l, top, 0, q);
#pragma unroll
            for (int i = 0; i < V; i++) l[i] = l[i] == -INFINITY ? -INFINITY : q[i];
          }
        }
#pragma unroll
        for (int i = 0; i < V; i++) {
          const int e = expert_of<V>(i, j);
          const float v = (a.sigmoid ? sigmoid_f32(l[i]) : l[i]) + a.select_bias[min(e, a.E - 1)];
          l[i] = l[i] != -INFINITY && v == v ? v : -INFINITY;
        }
        const float err = (a.sigmoid ? 8.0f * sigmoid_f32(top) : (V + 24) * most) * 0x1p-24f + 0x1p-125f;
        if (a.top_k <= 16) used = choose_candidates<V, true>(a, at_row, top, l, err, j, own_cand, c, rounds);
      } else {
        if (a.top_k <= 16) used = choose_candidates<V, false>(a, at_row, top, l, 0.0f, j, own_cand, c, rounds);
      }
      if (rounds) choose_rounds<BIAS>(a, at_row, top, j, c);
      const bool read_logits = BIAS || rounds;
#pragma unroll
      for (int q = 0; q < SLOTS; q++) {
        if (q >= used) c.id[q] = -1;
        if (c.id[q] < 0 || c.place[q] >= a.top_k) c.l[q] = -INFINITY;
        else if (read_logits) c.l[q] = logit(a, at_row, c.id[q]);
      }
      // weights
      float ctop = -INFINITY, w[SLOTS];
#pragma unroll
      for (int q = 0; q < SLOTS; q++) ctop = fmaxf(ctop, c.l[q]);
      ctop = a.renormalize || a.sigmoid ? row_max(ctop) : top;
#pragma unroll
      for (int q = 0; q < SLOTS; q++) {
        w[q] = 0.0f;
        if (q >= used) continue;
        if (a.sigmoid && !a.renormalize) w[q] = c.l[q] == -INFINITY ? 0.0f : sigmoid_f32(c.l[q]);
        else w[q] = chosen_score(c.l[q], ctop, a.sigmoid);
        if (a.renormalize) sum += w[q];
      }
      if (a.renormalize || !a.sigmoid) {
        sum = row_add(sum);
#pragma unroll
        for (int q = 0; q < SLOTS; q++)
          if (q < used) w[q] = sum > 0.0f ? w[q] / sum : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < SLOTS; q++) {
        if (q < used && in && c.place[q] < a.top_k) {
          a.ids[t * a.top_k + c.place[q]] = on ? c.id[q] : -1;
          a.weights[t * a.top_k + c.place[q]] = on ? w[q] : 0.0f;
          if constexpr (STATS) {
            if (on && c.id[q] >= 0) atomicAdd(&counts[c.id[q]], 1);
          }
        }
      }
    } else if constexpr (STATS) {
      for (int s = j; s < a.top_k; s += 16) {
        const int id = on ? a.ids[t * a.top_k + s] : -1;
        if (id >= 0 && id < a.E) atomicAdd(&counts[id], 1);
      }
    }
  }
  if constexpr (STATS) {
    const int j = threadIdx.x & 15;
    // this workgroup's sums: four tokens' rows of a wavefront, then its wavefronts
#pragma unroll
    for (int i = 0; i < V; i++) {
      float v = psum[i];
      v += __shfl_xor(v, 16);
      v += __shfl_xor(v, 32);
      if ((threadIdx.x & 63) < 16) psums[threadIdx.x >> 6][expert_of<V>(i, j)] = v;
    }
    if (seen) atomicAdd(&tokens, seen);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += RT) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < RT / 64; w++) v += psums[w][e];
      a.prob_partial[(int64_t)blockIdx.x * a.E + e] = v;
      a.count_partial[(int64_t)blockIdx.x * a.E + e] = counts[e];
    }
    if (threadIdx.x == 0) a.token_partial[blockIdx.x] = tokens;
  }
}

// Outputs of expert e, whose probabilities sum to s and whose routes are n, of
// T tokens; returns its term of the loss, f P.
DEV double balance_expert(const BalanceParams& a, int e, double s, int n, int tokens) {
  const double T = (double)tokens;
  const double f = tokens > 0 ? (double)n / (T * a.top_k) : 0.0;
  const double mean = tokens > 0 ? s / T : 0.0;
  a.counts[e] = n;
  a.mean_probs[e] = (float)mean;
  a.prob_grad[e] = tokens > 0 ? (float)((double)a.coef * a.E / T * (f - 1.0 / a.E)) : 0.0f;
  return f * mean;
}

// The partials r, r + STEP, .. of expert e, eight of them loaded at a time
// (past the last one: that one again, which does not count).
template <int STEP>
DEV void add_partials(const BalanceParams& a, int r, int e, double& s, int& n) {
#pragma unroll 1
  for (int p = r; p < a.partials; p += 8 * STEP) {
    float f[8];
    int c[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int at = min(p + i * STEP, a.partials - 1) * a.E + e;
      f[i] = a.prob_partial[at];
      c[i] = a.count_partial[at];
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const bool in = p + i * STEP < a.partials;
      s += in ? (double)f[i] : 0.0;
      n += in ? c[i] : 0;
    }
  }
}

// Joins the workgroups' statistics, 4 experts a workgroup, 64 rows of lanes
// over the partials, joined in a fixed order in fp64; the last workgroup to
// arrive adds the loss terms of all of them, in a fixed order.
constexpr int FT = 256;
constexpr int FE = 4;

__global__ __launch_bounds__(FT) void balance_finish_kernel(const BalanceParams a) {
  __shared__ double psum[FT / FE][FE];
  __shared__ int count[FT / FE][FE];
  __shared__ int total;
  const int c = threadIdx.x % FE, r = threadIdx.x / FE;
  const int e = blockIdx.x * FE + c;
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  double s = 0.0;
  int n = 0, t = 0;
  static_assert(STAT_BLOCKS <= 2 * FT, "two token counts a thread");
  const int q = threadIdx.x;
  const int t0 = a.token_partial[min(q, a.partials - 1)], t1 = a.token_partial[min(q + FT, a.partials - 1)];
  if (e < a.E) add_partials<FT / FE>(a, r, e, s, n);
  t = (q < a.partials ? t0 : 0) + (q + FT < a.partials ? t1 : 0);
  psum[r][c] = s;
  count[r][c] = n;
  if (t) atomicAdd(&total, t);
  __syncthreads();
  if (threadIdx.x >= 64) return;
  // one wavefront: lane l takes rows l / 4, l / 4 + 16, .. of expert l % 4
  s = 0.0;
  n = 0;
#pragma unroll
  for (int i = 0; i < FT / FE; i += 64 / FE) {
    s += psum[i + r][c];
    n += count[i + r][c];
  }
#pragma unroll
  for (int d = FE; d < 64; d <<= 1) {
    s += __shfl_xor(s, d);
    n += __shfl_xor(n, d);
  }
  double term = 0.0;
  if (threadIdx.x < FE && e < a.E) term = balance_expert(a, e, s, n, total);
#pragma unroll
  for (int d = 1; d < FE; d <<= 1) term += __shfl_xor(term, d);
  // The term goes to memory (agent scope) and is there (vmcnt 0) before the
  // ticket is taken; the terms are read the same way.  No release or acquire
  // of that scope, which would write back and drop this XCD's L2.
  unsigned before = 0;
  if (threadIdx.x == 0) __hip_atomic_store(a.loss_partial + blockIdx.x, term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");  // keeps the store above the wait
  __builtin_amdgcn_s_waitcnt(0x0F70);                      // vmcnt(0): expcnt and lgkmcnt not waited
  if (threadIdx.x == 0) before = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  before = __builtin_amdgcn_readfirstlane(before);
  if (before == gridDim.x - 1) {
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");  // keeps the loads below the ticket
    double sum = 0.0;
    for (unsigned b = threadIdx.x; b < gridDim.x; b += 64)
      sum += __hip_atomic_load(a.loss_partial + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    if (threadIdx.x == 0) *a.loss = (float)((double)a.coef * a.E * sum);
  }
}

// The same of few partials in one workgroup, without the round of atomics:
// OT / C rows of C lanes over the partials (C >= E, a power of two), joined in
// a fixed order.
constexpr int OT = 1024;

template <int C>
__global__ __launch_bounds__(OT) void balance_small_kernel(const BalanceParams a) {
  constexpr int R = OT / C;
  __shared__ double psum[R][C];
  __shared__ int count[R][C];
  __shared__ double terms[C / 64];
  __shared__ int total;
  const int c = threadIdx.x % C, r = threadIdx.x / C;
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  double s = 0.0;
  int n = 0;
  static_assert(STAT_BLOCKS <= OT, "a token count a thread");
  int t = a.token_partial[min((int)threadIdx.x, a.partials - 1)];
  if (c < a.E) add_partials<R>(a, r, c, s, n);
  t = (int)threadIdx.x < a.partials ? t : 0;
  psum[r][c] = s;
  count[r][c] = n;
  if (t) atomicAdd(&total, t);
  __syncthreads();
  double term = 0.0;
  if (r == 0 && c < a.E) {
#pragma unroll
    for (int i = 1; i < R; i++) {
      s += psum[i][c];
      n += count[i][c];
    }
    term = balance_expert(a, c, s, n, total);
  }
  if (r == 0) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) term += __shfl_xor(term, d);
    if (C > 64 && (threadIdx.x & 63) == 0) terms[threadIdx.x >> 6] = term;
  }
  if constexpr (C > 64) {
    __syncthreads();
    term = 0.0;
#pragma unroll
    for (int i = 0; i < C / 64; i++) term += terms[i];
  }
  if (threadIdx.x == 0) *a.loss = (float)((double)a.coef * a.E * term);
}

template <int V>
DEV void store_row(void* out, int f32, int64_t at, int E, int j, bool vec, const float (&d)[V]) {
  if (V > 4 && vec) {
#pragma unroll
    for (int c = 0; c < V / 4; c++) {
      const int e = expert_of<V>(4 * c, j);
      if (e >= E) continue;
      if (f32) {
        *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(out) + at + e) =
            f32x4_t{d[4 * c], d[4 * c + 1], d[4 * c + 2], d[4 * c + 3]};
      } else {
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(out) + at + e) =
            make_uint2(pack_bf16x2(d[4 * c], d[4 * c + 1]), pack_bf16x2(d[4 * c + 2], d[4 * c + 3]));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) {
      const int e = expert_of<V>(i, j);
      if (e >= E) continue;
      if (f32) reinterpret_cast<float*>(out)[at + e] = d[i];
      else reinterpret_cast<uint16_t*>(out)[at + e] = f32_to_bf16(d[i]);
    }
  }
}

// The chosen experts' own terms are scattered through an LDS row of the token.
template <int V>
__global__ __launch_bounds__(RT) void router_backward_kernel(const RouterBackwardParams a, bool vec, bool vec_out) {
  __shared__ __attribute__((aligned(16))) float scatter[TOKENS][16 * V];
  float* row_of = scatter[threadIdx.x >> 4];
  const float dl = a.prob_grad ? (a.d_loss ? *a.d_loss : 1.0f) : 0.0f;
  const bool need_p = a.prob_grad || (!a.sigmoid && !a.renormalize);
  float u[V];  // the loss's gradient in the probabilities, the same for all tokens
#pragma unroll
  for (int i = 0; i < V; i++) {
    const int e = expert_of<V>(i, threadIdx.x & 15);
    u[i] = a.prob_grad ? a.prob_grad[min(e, a.E - 1)] * dl : 0.0f;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * TOKENS; t0 < a.M; t0 += (int64_t)gridDim.x * TOKENS) {
    const int j = opaque(threadIdx.x & 15);
    const int64_t t = t0 + (threadIdx.x >> 4);
    const bool in = t < a.M;
    const bool on = in && (!a.token_mask || a.token_mask[t] != 0);
    const int64_t row = in ? t : a.M - 1;
    float l[V], d[V];
    load_row<V>(a.logits, a.logits_f32, row * a.row_stride, a.E, j, vec, l);
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; i++) {
      top = fmaxf(top, l[i]);
      d[i] = 0.0f;
    }
    top = row_max(top);

    float all = 0.0f;  // sum of dw w, subtracted from every expert (softmax without renormalisation)
    if (a.d_weights) {
      f32x4_t* mine = reinterpret_cast<f32x4_t*>(row_of + 4 * j);  // (all lanes clear the row)
#pragma unroll
      for (int i = 0; i < V / 4; i++) mine[16 * i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      // places j, j + 16, .. of which the first `slots` can be taken
      const int slots = (a.top_k + 15) / 16;
      int id[SLOTS];
      float w[SLOTS], dw[SLOTS], ctop = -INFINITY, sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int q = 0; q < SLOTS; q++) {
        id[q] = -1;
        w[q] = -INFINITY;
        dw[q] = 0.0f;
        if (q >= slots) continue;
        const int s = j + 16 * q;
        if (on && s < a.top_k) id[q] = a.ids[t * a.top_k + s];
        if (id[q] >= a.E) id[q] = -1;
        if (id[q] >= 0) {
          const int64_t at = row * a.row_stride + id[q];
          w[q] = clean(a.logits_f32 ? reinterpret_cast<const float*>(a.logits)[at]
                                    : bf16_to_f32(reinterpret_cast<const uint16_t*>(a.logits)[at]));
          dw[q] = a.d_weights[t * a.top_k + s];
        }
        ctop = fmaxf(ctop, w[q]);
      }
      ctop = row_max(ctop);
      if (!a.renormalize && !a.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; i++) sum += exp_neg(l[i] - top);
        ctop = top;
      }
      float keep[SLOTS];
#pragma unroll
      for (int q = 0; q < SLOTS; q++) {
        keep[q] = 1.0f;
        if (q >= slots) continue;
        if (a.sigmoid) keep[q] = sigmoid_f32(-w[q]);  // 1 - s
        if (a.sigmoid && !a.renormalize) w[q] = w[q] == -INFINITY ? 0.0f : sigmoid_f32(w[q]);
        else w[q] = chosen_score(w[q], ctop, a.sigmoid);
        if (a.renormalize) sum += w[q];
      }
      if (a.renormalize || !a.sigmoid) {
        sum = row_add(sum);
#pragma unroll
        for (int q = 0; q < SLOTS; q++)
          if (q < slots) w[q] = sum > 0.0f ? w[q] / sum : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < SLOTS; q++)
        if (q < slots) dot += dw[q] * w[q];
      dot = row_add(dot);
      if (!a.renormalize) {
        if (!a.sigmoid) all = dot;
        dot = 0.0f;
      }
      wave_fence();
#pragma unroll
      for (int q = 0; q < SLOTS; q++)
        if (id[q] >= 0) atomicAdd(&row_of[id[q]], w[q] * (dw[q] - dot) * keep[q]);
      wave_fence();
      if constexpr (V == 4) {
#pragma unroll
        for (int i = 0; i < V; i++) d[i] = row_of[expert_of<V>(i, j)];
      } else {
#pragma unroll
        for (int i = 0; i < V / 4; i++) {
          const f32x4_t v = mine[16 * i];
#pragma unroll
          for (int x = 0; x < 4; x++) d[4 * i + x] = v[x];
        }
      }
      wave_fence();
    }
    if (need_p) {
      float p[V], dot = 0.0f;
      probabilities<V>(l, top, a.sigmoid, p);
#pragma unroll
      for (int i = 0; i < V; i++) dot = fmaf(u[i], p[i], dot);  // (p is 0 past the last expert)
      dot = row_add(dot);
      if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; i++) d[i] += p[i] * (u[i] - dot) * sigmoid_f32(-l[i]);
      } else {
        dot += all;
#pragma unroll
        for (int i = 0; i < V; i++) d[i] = fmaf(p[i], u[i] - dot, d[i]);
      }
    }
    if (a.token_mask) {
#pragma unroll
      for (int i = 0; i < V; i++) d[i] = on ? d[i] : 0.0f;
    }
    if (in) {
      store_row<V>(a.d_logits, a.logits_f32, t * a.E, a.E, j, vec_out, d);
    }
  }
}

unsigned token_blocks(int64_t M) {
  const int64_t b = (M + TOKENS - 1) / TOKENS;
  return (unsigned)(b < 1 ? 1 : b > (1 << 20) ? 1 << 20 : b);
}

// whole groups of four logits on their own alignment (16 bytes fp32, 8 bf16)
bool whole_groups(const void* p, int f32, int64_t stride, int E) {
  return E % 4 == 0 && stride % 4 == 0 && ((uintptr_t)p & (f32 ? 15 : 7)) == 0;
}

template <int V>
hipError_t launch_v(const RouterParams& p, hipStream_t s) {
  const bool vec = whole_groups(p.logits, p.logits_f32, p.row_stride, p.E);
  const bool stats = p.prob_partial != nullptr;
  const unsigned grid = stats ? (unsigned)router_partials(p.M) : token_blocks(p.M);
  const int threads = threads_of(stats);
  if (p.select && stats) {
    if constexpr (V == 64) {  // (both at once do not fit the registers: one after the other)
      RouterParams q = p;
      q.prob_partial = nullptr;
      const hipError_t e = launch_v<V>(q, s);
      if (e != hipSuccess) return e;
      q = p;
      q.select = 0;
      return launch_v<V>(q, s);
    } else if (p.select_bias) {
      router_kernel<V, true, true, true><<<grid, threads, 0, s>>>(p, vec);
    } else {
      router_kernel<V, true, false, true><<<grid, threads, 0, s>>>(p, vec);
    }
  } else if (stats) {
    router_kernel<V, false, false, true><<<grid, threads, 0, s>>>(p, vec);
  } else if (p.select_bias) {
    router_kernel<V, true, true, false><<<grid, threads, 0, s>>>(p, vec);
  } else {
    router_kernel<V, true, false, false><<<grid, threads, 0, s>>>(p, vec);
  }
  return hipGetLastError();
}

template <int V>
hipError_t launch_back(const RouterBackwardParams& p, hipStream_t s) {
  // (2048 workgroups fill the CUs, and walk the rest of the tokens)
  router_backward_kernel<V><<<std::min(2048u, token_blocks(p.M)), RT, 0, s>>>(
      p, whole_groups(p.logits, p.logits_f32, p.row_stride, p.E), whole_groups(p.d_logits, p.logits_f32, p.E, p.E));
  return hipGetLastError();
}

}  // namespace

int router_partials(int64_t M) {
  const int64_t b = (M + STAT_TOKENS - 1) / STAT_TOKENS;
  return (int)(b < 1 ? 1 : b > STAT_BLOCKS ? STAT_BLOCKS : b);
}

int balance_finish_blocks(int E) { return (E + FE - 1) / FE; }

hipError_t launch_router(const RouterParams& p, hipStream_t s) {
  if (p.E <= 64) return launch_v<4>(p, s);
  if (p.E <= 128) return launch_v<8>(p, s);
  if (p.E <= 256) return launch_v<16>(p, s);
  if (p.E <= 512) return launch_v<32>(p, s);
  return launch_v<64>(p, s);
}

hipError_t launch_balance_finish(const BalanceParams& p, hipStream_t s) {
  // up to 32 Ki sums one workgroup adds them sooner than several and their
  // round of atomics (the loss of 3001 tokens to 60 experts, both kernels: 8.4
  // us against 9.6; 4000 to 256: 11.6 against 12.1; 16384 to 256: 25 against 17)
  if (p.E <= 256 && p.partials * p.E <= 1 << 15) {
    if (p.E <= 64) balance_small_kernel<64><<<1, OT, 0, s>>>(p);
    else if (p.E <= 128) balance_small_kernel<128><<<1, OT, 0, s>>>(p);
    else balance_small_kernel<256><<<1, OT, 0, s>>>(p);
    return hipGetLastError();
  }
  balance_finish_kernel<<<balance_finish_blocks(p.E), FT, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_router_backward(const RouterBackwardParams& p, hipStream_t s) {
  if (p.E <= 64) return launch_back<4>(p, s);
  if (p.E <= 128) return launch_back<8>(p, s);
  if (p.E <= 256) return launch_back<16>(p, s);
  if (p.E <= 512) return launch_back<32>(p, s);
  return launch_back<64>(p, s);
}

}  // namespace moe
