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
// + 3 (16-byte loads, 256 bytes a row of lanes), so a maximum or a sum over
// the experts is a loop over a lane's registers and four DPP steps, and a
// wavefront serves four tokens with each instruction.
#include <cfloat>

#include "device_common.h"
#include "internal.h"

namespace moe {

namespace {

constexpr int RT = 256;        // threads: 16 tokens at a time
constexpr int TOKENS = RT / 16;

constexpr int QUAD_XOR1 = 0xB1, QUAD_XOR2 = 0x4E, ROW_HALF_MIRROR = 0x141, ROW_MIRROR = 0x140;

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

// a reduction over the 16 lanes of a token
template <typename T, typename F>
DEV T row_reduce(T v, F f) {
  v = f(v, dpp<QUAD_XOR1>(v));
  v = f(v, dpp<QUAD_XOR2>(v));
  v = f(v, dpp<ROW_HALF_MIRROR>(v));
  return f(v, dpp<ROW_MIRROR>(v));
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

// NaN and -inf: not choosable; +inf counts as FLT_MAX
DEV float clean(float l) { return l == l ? fminf(l, FLT_MAX) : -INFINITY; }

// expert of register i of lane j
DEV int expert_of(int i, int j) { return (i >> 2) * 64 + 4 * j + (i & 3); }

// logits of a row; -inf past E.  vec: rows of whole, aligned groups of four
template <int V>
DEV void load_row(const void* logits, int f32, int64_t at, int E, int j, bool vec, float (&l)[V]) {
  if (vec) {
#pragma unroll
    for (int c = 0; c < V / 4; c++) {
      const int e = expert_of(4 * c, j);
      f32x4_t v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (e < E) {
        if (f32) {
          v = *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(logits) + at + e);
        } else {
          const uint2 b = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(logits) + at + e);
          v = f32x4_t{__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u), __uint_as_float(b.y << 16),
                      __uint_as_float(b.y & 0xffff0000u)};
        }
      }
#pragma unroll
      for (int i = 0; i < 4; i++) l[4 * c + i] = clean(v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) {
      const int e = expert_of(i, j);
      float v = -INFINITY;
      if (e < E)
        v = f32 ? reinterpret_cast<const float*>(logits)[at + e]
                : bf16_to_f32(reinterpret_cast<const uint16_t*>(logits)[at + e]);
      l[i] = clean(v);
    }
  }
}

// Probabilities of a row: the softmax, or the sigmoid scores over their sum.
// Both are taken relative to the largest logit, so that a row of very
// negative logits does not become 0 / 0: s = exp(min(l, 0)) / (1 + exp(-|l|)),
// and the factor exp(-min(max, 0)) cancels in the quotient.
template <int V>
DEV void probabilities(const float (&l)[V], float top, int sigmoid, float (&p)[V]) {
  float sum = 0.0f;
  const float ref = sigmoid ? fminf(top, 0.0f) : top;
#pragma unroll
  for (int i = 0; i < V; i++) {
    float e = expf((sigmoid ? fminf(l[i], 0.0f) : l[i]) - ref);
    if (sigmoid) e = e / (1.0f + expf(-fabsf(l[i])));
    p[i] = l[i] == -INFINITY ? 0.0f : e;
    sum += p[i];
  }
  sum = row_add(sum);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < V; i++) p[i] *= inv;
}

DEV float sigmoid_f32(float l) { return 1.0f / (1.0f + expf(-l)); }

// Score of a chosen logit before the division by the sum over the chosen
// (renormalize), relative to the largest chosen one as in probabilities()
DEV float chosen_score(float l, float top, int sigmoid) {
  if (l == -INFINITY) return 0.0f;
  if (!sigmoid) return expf(l - top);
  return expf(fminf(l, 0.0f) - fminf(top, 0.0f)) / (1.0f + expf(-fabsf(l)));
}

constexpr int SLOTS = ROUTER_MAX_TOP_K / 16;  // chosen places a lane holds: j, j + 16, ...

// The key of the choice: the logit, or score + bias in fp64.
template <int V, bool BIAS>
struct Keys;
template <int V>
struct Keys<V, false> {
  typedef float type;
  static DEV void make(const float (&l)[V], float, int, const float*, int, int, float (&k)[V]) {
#pragma unroll
    for (int i = 0; i < V; i++) k[i] = l[i];
  }
};
template <int V>
struct Keys<V, true> {
  typedef double type;
  static DEV void make(const float (&l)[V], float top, int sigmoid, const float* bias, int E, int j, double (&k)[V]) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; i++) {
      const double d = (double)l[i];
      k[i] = sigmoid ? 1.0 / (1.0 + exp(-d)) : exp(d - (double)top);
      if (!sigmoid && l[i] != -INFINITY) sum += k[i];
    }
    if (!sigmoid) sum = row_add(sum);
#pragma unroll
    for (int i = 0; i < V; i++) {
      const int e = expert_of(i, j);
      const double b = e < E ? (double)bias[e] : 0.0;
      const double v = (sigmoid ? k[i] : k[i] / sum) + b;
      k[i] = l[i] != -INFINITY && v == v ? v : -INFINITY;
    }
  }
};

template <int V, bool SELECT, bool BIAS, bool STATS>
__global__ __launch_bounds__(RT) void router_kernel(const RouterParams a, bool vec) {
  __shared__ int counts[STATS ? 16 * V : 1];
  __shared__ float psums[STATS ? RT / 64 : 1][STATS ? 16 * V : 1];
  __shared__ int tokens;
  const int j = threadIdx.x & 15;
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

    float p[STATS ? V : 1];
    if constexpr (STATS) {
      probabilities<V>(l, top, a.sigmoid, p);
      if (on) {
#pragma unroll
        for (int i = 0; i < V; i++) psum[i] += p[i];
        seen += j == 0;
      }
    }

    int id[SLOTS];
    if constexpr (SELECT) {
      typename Keys<V, BIAS>::type key[V];
      Keys<V, BIAS>::make(l, top, a.sigmoid, a.select_bias, a.E, j, key);
      float cl[SLOTS];
#pragma unroll
      for (int q = 0; q < SLOTS; q++) {
        id[q] = -1;
        cl[q] = -INFINITY;
      }
      for (int s = 0; s < a.top_k; s++) {
        // the largest key; of equal ones the lowest expert
        auto best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < V; i++) {
          if (key[i] > best) {
            best = key[i];
            at = i;
          }
        }
        const auto win = row_max(best);
        const bool any = win > -INFINITY;
        const int e = row_min(best == win ? expert_of(at, j) : INT32_MAX);
        float wl = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; i++) {
          const bool mine = any && expert_of(i, j) == e;
          if (mine) {
            wl = l[i];
            key[i] = -INFINITY;
          }
        }
        wl = row_max(wl);
        if (any && (s & 15) == j) {
#pragma unroll
          for (int q = 0; q < SLOTS; q++)
            if (q == s >> 4) {
              id[q] = e;
              cl[q] = wl;
            }
        }
      }
      // weights
      float ctop = -INFINITY, sum = 0.0f, w[SLOTS];
#pragma unroll
      for (int q = 0; q < SLOTS; q++) ctop = fmaxf(ctop, cl[q]);
      ctop = row_max(ctop);
      if (a.renormalize) {
#pragma unroll
        for (int q = 0; q < SLOTS; q++) {
          w[q] = chosen_score(cl[q], ctop, a.sigmoid);
          sum += w[q];
        }
        sum = row_add(sum);
#pragma unroll
        for (int q = 0; q < SLOTS; q++) w[q] = sum > 0.0f ? w[q] / sum : 0.0f;
      } else if (a.sigmoid) {
#pragma unroll
        for (int q = 0; q < SLOTS; q++) w[q] = cl[q] == -INFINITY ? 0.0f : sigmoid_f32(cl[q]);
      } else {
#pragma unroll
        for (int i = 0; i < V; i++) sum += l[i] == -INFINITY ? 0.0f : expf(l[i] - top);
        sum = row_add(sum);
#pragma unroll
        for (int q = 0; q < SLOTS; q++) w[q] = cl[q] == -INFINITY ? 0.0f : expf(cl[q] - top) / sum;
      }
      if (in) {
#pragma unroll
        for (int q = 0; q < SLOTS; q++) {
          const int s = j + 16 * q;
          if (s < a.top_k) {
            if (!on) id[q] = -1;
            a.ids[t * a.top_k + s] = id[q];
            a.weights[t * a.top_k + s] = on ? w[q] : 0.0f;
          }
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < SLOTS; q++) {
        const int s = j + 16 * q;
        id[q] = on && s < a.top_k ? a.ids[t * a.top_k + s] : -1;
      }
    }
    if constexpr (STATS) {
      if (on) {
#pragma unroll
        for (int q = 0; q < SLOTS; q++)
          if (j + 16 * q < a.top_k && id[q] >= 0 && id[q] < a.E) atomicAdd(&counts[id[q]], 1);
      }
    }
  }
  if constexpr (STATS) {
    // this workgroup's sums: four tokens' rows of a wavefront, then its wavefronts
#pragma unroll
    for (int i = 0; i < V; i++) {
      float v = psum[i];
      v += __shfl_xor(v, 16);
      v += __shfl_xor(v, 32);
      if ((threadIdx.x & 63) < 16) psums[threadIdx.x >> 6][expert_of(i, j)] = v;
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

// Joins the workgroups' statistics, 32 experts a workgroup (32 lanes wide, 32
// rows of lanes over the partials, joined in a fixed order in fp64); the last
// workgroup to arrive adds the loss terms of all of them, in their order.
constexpr int FT = 1024;
constexpr int FE = 32;

__global__ __launch_bounds__(FT) void balance_finish_kernel(const BalanceParams a) {
  __shared__ double psum[FT / FE][FE + 1];
  __shared__ int count[FT / FE][FE + 1];
  __shared__ int total;
  const int c = threadIdx.x % FE, r = threadIdx.x / FE;
  const int e = blockIdx.x * FE + c;
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  double s = 0.0;
  int n = 0, t = 0;
  if (e < a.E) {
    for (int p = r; p < a.partials; p += FT / FE) {
      s += (double)a.prob_partial[(int64_t)p * a.E + e];
      n += a.count_partial[(int64_t)p * a.E + e];
    }
  }
  for (int p = threadIdx.x; p < a.partials; p += FT) t += a.token_partial[p];
  psum[r][c] = s;
  count[r][c] = n;
  if (t) atomicAdd(&total, t);
  __syncthreads();
  if (threadIdx.x >= 64) return;
  double term = 0.0;
  if (threadIdx.x < FE && e < a.E) {
    s = 0.0;
    n = 0;
    for (int k = 0; k < FT / FE; k++) {
      s += psum[k][c];
      n += count[k][c];
    }
    const double T = (double)total;
    const double f = total > 0 ? (double)n / (T * a.top_k) : 0.0;
    const double mean = total > 0 ? s / T : 0.0;
    a.counts[e] = n;
    a.mean_probs[e] = (float)mean;
    a.prob_grad[e] = total > 0 ? (float)((double)a.coef * a.E / T * (f - 1.0 / a.E)) : 0.0f;
    term = f * mean;
  }
  for (int d = 1; d < 64; d <<= 1) term += __shfl_xor(term, d);
  if (threadIdx.x == 0) {
    __hip_atomic_store(a.loss_partial + blockIdx.x, term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const unsigned before = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    if (before == gridDim.x - 1) {
      double sum = 0.0;
      for (unsigned b = 0; b < gridDim.x; b++)
        sum += __hip_atomic_load(a.loss_partial + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      *a.loss = (float)((double)a.coef * a.E * sum);
    }
  }
}

template <int V>
DEV void store_row(void* out, int f32, int64_t at, int E, int j, bool vec, const float (&d)[V]) {
  if (vec) {
#pragma unroll
    for (int c = 0; c < V / 4; c++) {
      const int e = expert_of(4 * c, j);
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
      const int e = expert_of(i, j);
      if (e >= E) continue;
      if (f32) reinterpret_cast<float*>(out)[at + e] = d[i];
      else reinterpret_cast<uint16_t*>(out)[at + e] = f32_to_bf16(d[i]);
    }
  }
}

DEV void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// The chosen experts' own terms are scattered through an LDS row of the token.
template <int V>
__global__ __launch_bounds__(RT) void router_backward_kernel(const RouterBackwardParams a, bool vec, bool vec_out) {
  __shared__ float scatter[TOKENS][16 * V];
  const int j = threadIdx.x & 15;
  float* row_of = scatter[threadIdx.x >> 4];
  const float dl = a.prob_grad ? (a.d_loss ? *a.d_loss : 1.0f) : 0.0f;
  const bool need_p = a.prob_grad || (!a.sigmoid && !a.renormalize);
  for (int64_t t0 = (int64_t)blockIdx.x * TOKENS; t0 < a.M; t0 += (int64_t)gridDim.x * TOKENS) {
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
#pragma unroll
      for (int i = 0; i < V; i++) row_of[expert_of(i, j)] = 0.0f;
      int id[SLOTS];
      float w[SLOTS], dw[SLOTS], keep[SLOTS], ctop = -INFINITY, sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int q = 0; q < SLOTS; q++) {
        const int s = j + 16 * q;
        id[q] = on && s < a.top_k ? a.ids[t * a.top_k + s] : -1;
        if (id[q] >= a.E) id[q] = -1;
        w[q] = -INFINITY;
        dw[q] = 0.0f;
        if (id[q] >= 0) {
          const int64_t at = row * a.row_stride + id[q];
          w[q] = clean(a.logits_f32 ? reinterpret_cast<const float*>(a.logits)[at]
                                    : bf16_to_f32(reinterpret_cast<const uint16_t*>(a.logits)[at]));
          dw[q] = a.d_weights[t * a.top_k + s];
        }
        ctop = fmaxf(ctop, w[q]);
        keep[q] = a.sigmoid ? 1.0f / (1.0f + expf(w[q])) : 1.0f;  // 1 - s
      }
      ctop = row_max(ctop);
      if (!a.renormalize && !a.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; i++) sum += l[i] == -INFINITY ? 0.0f : expf(l[i] - top);
        ctop = top;
      }
#pragma unroll
      for (int q = 0; q < SLOTS; q++) {
        if (a.sigmoid && !a.renormalize) w[q] = w[q] == -INFINITY ? 0.0f : sigmoid_f32(w[q]);
        else w[q] = chosen_score(w[q], ctop, a.sigmoid);
        if (a.renormalize) sum += w[q];
      }
      if (a.renormalize || !a.sigmoid) {
        sum = row_add(sum);
#pragma unroll
        for (int q = 0; q < SLOTS; q++) w[q] = sum > 0.0f ? w[q] / sum : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < SLOTS; q++) dot += dw[q] * w[q];
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
#pragma unroll
      for (int i = 0; i < V; i++) d[i] = row_of[expert_of(i, j)];
      wave_fence();
    }
    if (need_p) {
      float p[V], u[V], dot = 0.0f;
      probabilities<V>(l, top, a.sigmoid, p);
#pragma unroll
      for (int i = 0; i < V; i++) {
        const int e = expert_of(i, j);
        u[i] = a.prob_grad && e < a.E ? a.prob_grad[e] * dl : 0.0f;
        dot = fmaf(u[i], p[i], dot);
      }
      dot = row_add(dot);
#pragma unroll
      for (int i = 0; i < V; i++) {
        float g = p[i] * (u[i] - dot);
        if (a.sigmoid) g = g / (1.0f + expf(l[i]));
        else g -= p[i] * all;
        d[i] += g;
      }
    }
    if (in) {
#pragma unroll
      for (int i = 0; i < V; i++) d[i] = on ? d[i] : 0.0f;
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
  const unsigned grid = stats ? (unsigned)router_partials(p.M, p.E) : token_blocks(p.M);
  if (!p.select) router_kernel<V, false, false, true><<<grid, RT, 0, s>>>(p, vec);
  else if (p.select_bias && stats) router_kernel<V, true, true, true><<<grid, RT, 0, s>>>(p, vec);
  else if (p.select_bias) router_kernel<V, true, true, false><<<grid, RT, 0, s>>>(p, vec);
  else if (stats) router_kernel<V, true, false, true><<<grid, RT, 0, s>>>(p, vec);
  else router_kernel<V, true, false, false><<<grid, RT, 0, s>>>(p, vec);
  return hipGetLastError();
}

template <int V>
hipError_t launch_back(const RouterBackwardParams& p, hipStream_t s) {
  router_backward_kernel<V><<<token_blocks(p.M), RT, 0, s>>>(
      p, whole_groups(p.logits, p.logits_f32, p.row_stride, p.E), whole_groups(p.d_logits, p.logits_f32, p.E, p.E));
  return hipGetLastError();
}

}  // namespace

int router_partials(int64_t M, int) {
  const int64_t b = (M + TOKENS - 1) / TOKENS;
  return (int)(b < 1 ? 1 : b > 512 ? 512 : b);
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
