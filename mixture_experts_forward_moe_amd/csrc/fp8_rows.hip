// fp8_rows.hip -- rows in 8 bits: quantisers, the experts' rows sorted and
// back, and gated activations whose inputs are kept in 8 bits.
//
// A row is held as E4M3 codes with one E8M0 byte for each 128 values, the least
// power of two that brings the block's largest value to 448 or less.  So the
// codes of a block never overflow, decoding is exact in bf16 (a code times a
// power of two; under the least scales bf16's own steps keep the codes to multiples
// of 2^-133), and the matrix instruction takes the bytes as they are.  An
// infinity or a NaN has no part in the scale and becomes a NaN code: what
// overflowed stays visible.
//
// Every kernel here is bound by HBM: a wavefront takes pieces of 512 values
// of a row (16 bytes a lane, a block of 128 in 16 lanes) and reads each input
// once; the scale is an integer maximum over those lanes.
#include "device_common.h"
#include "internal.h"

namespace moe {

namespace {

constexpr int BLOCK = 128;
constexpr int PIECE = 512;  // values of a row that a wavefront takes at once

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// the largest |v| of eight bf16 (as bits); those that are not finite count as 0
DEV uint32_t amax8(const u32x4_t& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t lo = v[i] & 0x7fffu, hi = (v[i] >> 16) & 0x7fffu;
    m = max(m, lo < 0x7f80u ? lo : 0u);
    m = max(m, hi < 0x7f80u ? hi : 0u);
  }
  return m;
}

template <int CTRL>
DEV uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true));
}

// E8M0 code of a block whose largest magnitude has the bf16 bits m: 448 is
// 1.75 * 2^8, so its exponent less 8, one more past a mantissa of 1.75
DEV uint32_t scale_code(uint32_t m) {
  const int c = (int)(m >> 7) - 8 + ((m & 127u) > 96u ? 1 : 0);
  return (uint32_t)max(c, 1);
}

// The codes of eight bf16 values of a block that 16 lanes hold, and its E8M0 code
DEV u32x2_t quantize8(const u32x4_t& v, uint32_t& code) {
  uint32_t m = amax8(v);
  m = dpp_max<DPP_XOR1>(m);
  m = dpp_max<DPP_XOR2>(m);
  m = dpp_max<DPP_HALF_MIRROR>(m);
  m = dpp_max<DPP_MIRROR>(m);
  code = scale_code(m);
  const float s = __uint_as_float(code << 23);
  u32x2_t o;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const uint32_t lo = v[2 * i], hi = v[2 * i + 1];
    i16x2_t r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, lo), s, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, hi), s, true);
    o[i] = __builtin_bit_cast(uint32_t, r);
  }
  return o;
}

// the eight values of codes under their E8M0 code, in fp32, finite but for NaN codes
DEV void decode8(const u32x2_t& q, uint32_t code, float (&v)[8]) {
  const float s = e8m0_scale_operand(code);
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const f32x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[i], s, false);
    const f32x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[i], s, true);
    v[4 * i] = lo[0];
    v[4 * i + 1] = lo[1];
    v[4 * i + 2] = hi[0];
    v[4 * i + 3] = hi[1];
  }
  if (code >= 247u) {  // 256 times 2^120, what the largest finite bf16 are rounded to, is past fp32: the end of its range
    constexpr float TOP = 0x1.fffffep127f;
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = v[i] > TOP ? TOP : v[i] < -TOP ? -TOP : v[i];
  }
}

DEV void unpack8(const u32x4_t& p, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[2 * i] = __uint_as_float(p[i] << 16);
    v[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
  }
}

DEV u32x4_t pack8(const float (&v)[8]) {
  u32x4_t p;
#pragma unroll
  for (int i = 0; i < 4; i++) p[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  return p;
}

DEV u32x4_t ld8(const uint16_t* p) { return *reinterpret_cast<const u32x4_t*>(p); }
DEV void st8(uint16_t* p, const u32x4_t& v) { *reinterpret_cast<u32x4_t*>(p) = v; }
DEV void st8(uint8_t* p, const u32x2_t& v) { *reinterpret_cast<u32x2_t*>(p) = v; }

// This wavefront's number in a grid_of: workgroups past ROW_OF_GRID go on in the
// grid's next row, so that its threads stay below 2^32 in each dimension
constexpr int64_t ROW_OF_GRID = 1 << 23;
DEV int64_t wave_number() {
  return ((int64_t)blockIdx.y * ROW_OF_GRID + blockIdx.x) * (blockDim.x >> 6) +
         __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// ------------------------------------------------------------- rows

template <int U>
__global__ __launch_bounds__(256) void fp8_rows_kernel(const uint16_t* x, int64_t stride, int64_t rows, int cols,
                                                       int parts, uint8_t* q, uint8_t* sf) {
  const int64_t w = wave_number(), row = w / parts;
  if (row >= rows) return;
  const int lane = threadIdx.x & 63, c0 = (int)(w - row * parts) * (PIECE * U) + 8 * lane;
  const int nb = (cols + BLOCK - 1) / BLOCK;
  u32x4_t v[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int c = c0 + PIECE * u;
    v[u] = u32x4_t{0u, 0u, 0u, 0u};
    if (c < cols) v[u] = ld8(x + row * stride + c);
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int c = c0 + PIECE * u;
    uint32_t code;
    const u32x2_t o = quantize8(v[u], code);
    if (c < cols) {
      st8(q + row * cols + c, o);
      if ((lane & 15) == 0) sf[row * nb + (c >> 7)] = (uint8_t)code;
    }
  }
}

// ------------------------------------------------------------- dispatch

// A wavefront reads its part of a token's row once, and writes it at the
// slots of the token's routes; a token without a local route is not read.
// 65536 tokens of 6144, 65000 routes, codes: 174 us, 6.9 TB/s.
template <int U>
__global__ __launch_bounds__(256) void dispatch_kernel(const DispatchParams a, int parts) {
  const int64_t w = wave_number(), t = w / parts;
  if (t >= a.M) return;
  const int lane = threadIdx.x & 63, c0 = (int)(w - t * parts) * (PIECE * U) + 8 * lane;
  const int nb = (a.H + BLOCK - 1) / BLOCK;
  const int slot = lane < a.top_k ? a.slots[t * a.top_k + lane] : -1;
  uint64_t routes = __ballot(slot >= 0);
  if (routes == 0) return;
  u32x4_t v[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int c = c0 + PIECE * u;
    v[u] = u32x4_t{0u, 0u, 0u, 0u};
    if (c < a.H) v[u] = ld8(a.x + t * a.x_row_stride + c);
  }
  u32x2_t o[U];
  uint32_t code[U];
  if (a.q) {
#pragma unroll
    for (int u = 0; u < U; u++) o[u] = quantize8(v[u], code[u]);
  }
  while (routes) {
    const int j = __builtin_ctzll(routes);
    routes &= routes - 1;
    const int64_t s = __builtin_amdgcn_readlane(slot, j);
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int c = c0 + PIECE * u;
      if (c >= a.H) continue;
      if (a.rows) st8(a.rows + s * a.H + c, v[u]);
      if (a.q) {
        st8(a.q + s * a.H + c, o[u]);
        if ((lane & 15) == 0) a.q_sf[s * nb + (c >> 7)] = (uint8_t)code[u];
      }
    }
  }
}

// dx[t] = the sum over the token's routes, in their order, in fp32.  (A piece a
// wavefront: four of them at once are no faster, 16384 tokens of 8 routes of 4096
// 239 us and 241, 8192 of 2 of 8192 74 and 81.)
__global__ __launch_bounds__(256) void dispatch_backward_kernel(const uint16_t* dxp, const int32_t* slots, int64_t M,
                                                                int top_k, int H, int accumulate, int parts,
                                                                uint16_t* dx) {
  const int64_t w = wave_number(), t = w / parts;
  if (t >= M) return;
  const int lane = threadIdx.x & 63, c = (int)(w - t * parts) * PIECE + 8 * lane;
  const int slot = lane < top_k ? slots[t * top_k + lane] : -1;
  uint64_t routes = __ballot(slot >= 0);
  float acc[8];
  u32x4_t old = {0u, 0u, 0u, 0u};
  if (accumulate && c < H) old = ld8(dx + t * H + c);
  unpack8(old, acc);
  while (routes) {
    const int j = __builtin_ctzll(routes);
    routes &= routes - 1;
    const int64_t s = __builtin_amdgcn_readlane(slot, j);
    if (c < H) {
      float v[8];
      unpack8(ld8(dxp + s * H + c), v);
#pragma unroll
      for (int i = 0; i < 8; i++) acc[i] += v[i];
    }
  }
  if (c < H) st8(dx + t * H + c, pack8(acc));
}

// ------------------------------------------------------------- gradients of the finalize

// A workgroup takes a token: its dout row stays in registers (NI pieces of
// 2048 values), each of its routes' y2 rows passes once.  The dot products are
// sums of fp32 products within a lane, then over the lanes and the wavefronts
// in a fixed order.  16384 tokens of 8 routes of 4096 (y2 read, gradients written in
// bf16 and in codes): 550 us, 5.1 TB/s.
template <int NI>
__global__ __launch_bounds__(256) void finalize_backward_kernel(const FinalizeBackwardParams a) {
  __shared__ float part[4][64];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nb = (a.H + BLOCK - 1) / BLOCK;
  const int64_t r0 = t * a.top_k;
  const int slot = lane < a.top_k ? a.slots[r0 + lane] : -1;
  const float weight = lane < a.top_k ? a.weights[r0 + lane] * a.rsf : 0.0f;
  uint64_t routes = __ballot(slot >= 0);
  if (routes == 0) {
    if (a.dw && tid < a.top_k) a.dw[r0 + tid] = 0.0f;
    return;
  }
  u32x4_t d[NI];
#pragma unroll
  for (int i = 0; i < NI; i++) {
    const int c = 8 * tid + 2048 * i;
    d[i] = u32x4_t{0u, 0u, 0u, 0u};
    if (c < a.H) d[i] = ld8(a.dout + t * a.H + c);
  }
  while (routes) {
    const int j = __builtin_ctzll(routes);
    routes &= routes - 1;
    const int64_t s = __builtin_amdgcn_readlane(slot, j);
    const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), j));
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; i++) {
      const int c = 8 * tid + 2048 * i;
      float g[8];
      unpack8(d[i], g);
      if (a.dw && c < a.H) {
        float y[8];
        unpack8(ld8(a.y2 + s * a.H + c), y);
#pragma unroll
        for (int e = 0; e < 8; e++) dot = fmaf(g[e], y[e], dot);
      }
      if (a.dy2 || a.q) {
#pragma unroll
        for (int e = 0; e < 8; e++) g[e] *= wj;
        const u32x4_t p = pack8(g);
        if (a.dy2 && c < a.H) st8(a.dy2 + s * a.H + c, p);
        if (a.q) {
          uint32_t code;
          const u32x2_t o = quantize8(p, code);
          if (c < a.H) {
            st8(a.q + s * a.H + c, o);
            if ((lane & 15) == 0) a.q_sf[s * nb + (c >> 7)] = (uint8_t)code;
          }
        }
      }
    }
    if (a.dw) {
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) dot += __shfl_xor(dot, m);
      if (lane == 0) part[wave][j] = dot;
    }
  }
  if (!a.dw) return;
  __syncthreads();
  if (tid < a.top_k)  // (wavefront 0 and its lane's own slot)
    a.dw[r0 + tid] = slot >= 0 ? a.rsf * (((part[0][tid] + part[1][tid]) + part[2][tid]) + part[3][tid]) : 0.0f;
}

// ------------------------------------------------------------- activations

// f(g), f'(g), the up part and whether it follows u.  SwiGLU: min(g, l)
// sigmoid(a min(g, l)) and clamp(u, -l, l) + b; past a limit the derivative is
// 0, at it that of the inside.  Selections, not fminf, so that a NaN stays one.
// Where a sigmoid is 0 its product with what may overflow is 0.
// GeGLU: g (1 + tanh z) / 2 is g sigmoid(2 z); both sigmoid(2 z) and
// sigmoid(-2 z) come from exp(-2 |z|), so that neither is a difference (1 +
// tanh z would be off by 30% at g = -5); the reciprocal of what lies in [1, 2] is the
// instruction's, a step off at most (65536 x 2048: 195 us, with a division 214).
struct GatePart {
  float f, df, up, dup;
};
template <int AK>
DEV GatePart gate_part(float g, float u, const GateAct& p) {
  if constexpr (AK == ACT_GEGLU_TANH) {
    const float c = 0.7978845608028654f;
    const float z = c * (g + 0.044715f * g * g * g);
    const float e = expf(-2.0f * fabsf(z)), big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
    const float s = z > 0.0f ? big : small;
    const float slope = small == 0.0f ? 0.0f : 2.0f * g * big * small * (c * (1.0f + 3.0f * 0.044715f * g * g));
    return {g * s, s + slope, u, 1.0f};
  } else {
    const float gc = g > p.limit ? p.limit : g;
    const float uc = u > p.limit ? p.limit : u < -p.limit ? -p.limit : u;
    const float s = 1.0f / (1.0f + expf(-p.alpha * gc));
    // (a g may overflow where 1 - s is 0, which it is from 128 on; a NaN is one by s)
    const float df = s == 0.0f ? 0.0f : s * (1.0f + fminf(p.alpha * gc, 128.0f) * (1.0f - s));
    return {gc * s, g > p.limit ? 0.0f : df, uc + p.beta, fabsf(u) > p.limit ? 0.0f : 1.0f};
  }
}

// y = f(g) up(u) of eight columns a lane, rounded to bf16 and quantised; g and u
// quantised too where they are kept.  A plan's padding slots are passed over.
// 65536 x 2048: 216 us, 4.4 TB/s (GeGLU 195), its gradient 255, 5.3 TB/s (244): HBM, and
// the few rows' 3.3 to 3.7 us are a launch's and one trip to memory.
template <int AK, int U>
__global__ __launch_bounds__(256) void act_kernel(const ActParams a, int parts) {
  const int64_t w = wave_number(), row = w / parts;
  if (row >= a.rows) return;
  if (a.routes && ld_uniform(a.routes + row) < 0) return;
  const int lane = threadIdx.x & 63, c0 = (int)(w - row * parts) * (PIECE * U) + 8 * lane;
  const int nb = (a.I + BLOCK - 1) / BLOCK;
  u32x4_t g[U], u[U];
#pragma unroll
  for (int i = 0; i < U; i++) {
    const int c = c0 + PIECE * i;
    g[i] = u[i] = u32x4_t{0u, 0u, 0u, 0u};
    if (c < a.I) {
      g[i] = ld8(a.h + row * 2 * a.I + c);
      u[i] = ld8(a.h + row * 2 * a.I + a.I + c);
    }
  }
#pragma unroll
  for (int i = 0; i < U; i++) {
    const int c = c0 + PIECE * i;
    float gv[8], uv[8], y[8];
    unpack8(g[i], gv);
    unpack8(u[i], uv);
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const GatePart p = gate_part<AK>(gv[e], uv[e], a.act);
      y[e] = p.f * p.up;
    }
    uint32_t code;
    const u32x2_t o = quantize8(pack8(y), code);
    if (c < a.I) {
      st8(a.y + row * a.I + c, o);
      if ((lane & 15) == 0) a.y_sf[row * nb + (c >> 7)] = (uint8_t)code;
    }
    if (a.hq) {
      uint32_t cg, cu;
      const u32x2_t og = quantize8(g[i], cg), ou = quantize8(u[i], cu);
      if (c < a.I) {
        st8(a.hq + row * 2 * a.I + c, og);
        st8(a.hq + row * 2 * a.I + a.I + c, ou);
        if ((lane & 15) == 0) {
          a.hq_sf[row * 2 * nb + (c >> 7)] = (uint8_t)cg;
          a.hq_sf[row * 2 * nb + nb + (c >> 7)] = (uint8_t)cu;
        }
      }
    }
  }
}

template <int AK, int U>
__global__ __launch_bounds__(256) void act_backward_kernel(const ActBackwardParams a, int parts) {
  const int64_t w = wave_number(), row = w / parts;
  if (row >= a.rows) return;
  if (a.routes && ld_uniform(a.routes + row) < 0) return;
  const int lane = threadIdx.x & 63, c0 = (int)(w - row * parts) * (PIECE * U) + 8 * lane;
  const int nb = (a.I + BLOCK - 1) / BLOCK;
  u32x2_t g[U], u[U];
  u32x4_t d[U];
  uint32_t gs[U], us[U];
#pragma unroll
  for (int i = 0; i < U; i++) {
    const int c = c0 + PIECE * i;
    g[i] = u[i] = u32x2_t{0u, 0u};
    d[i] = u32x4_t{0u, 0u, 0u, 0u};
    gs[i] = us[i] = 1u;
    if (c < a.I) {
      g[i] = *reinterpret_cast<const u32x2_t*>(a.hq + row * 2 * a.I + c);
      u[i] = *reinterpret_cast<const u32x2_t*>(a.hq + row * 2 * a.I + a.I + c);
      gs[i] = a.hq_sf[row * 2 * nb + (c >> 7)];
      us[i] = a.hq_sf[row * 2 * nb + nb + (c >> 7)];
      d[i] = ld8(a.dy + row * a.I + c);
    }
  }
#pragma unroll
  for (int i = 0; i < U; i++) {
    const int c = c0 + PIECE * i;
    float gv[8], uv[8], dv[8], dg[8], du[8];
    decode8(g[i], gs[i], gv);
    decode8(u[i], us[i], uv);
    unpack8(d[i], dv);
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const GatePart p = gate_part<AK>(gv[e], uv[e], a.act);
      dg[e] = dv[e] * p.df * p.up;
      du[e] = dv[e] * p.f * p.dup;
    }
    const u32x4_t pg = pack8(dg), pu = pack8(du);
    if (a.dh && c < a.I) {
      st8(a.dh + row * 2 * a.I + c, pg);
      st8(a.dh + row * 2 * a.I + a.I + c, pu);
    }
    if (a.dq) {
      uint32_t cg, cu;
      const u32x2_t og = quantize8(pg, cg), ou = quantize8(pu, cu);
      if (c < a.I) {
        st8(a.dq + row * 2 * a.I + c, og);
        st8(a.dq + row * 2 * a.I + a.I + c, ou);
        if ((lane & 15) == 0) {
          a.dq_sf[row * 2 * nb + (c >> 7)] = (uint8_t)cg;
          a.dq_sf[row * 2 * nb + nb + (c >> 7)] = (uint8_t)cu;
        }
      }
    }
  }
}

// ------------------------------------------------------------- weights

// A workgroup takes a block of 128 x 128: scale = amax / 448 (2^-126 at least),
// codes of w / scale, stored in w's order and, through LDS, transposed.  32 x 4096 x
// 6144: 450 us, with the transposed codes 604, both 5.3 TB/s.
__global__ __launch_bounds__(256) void fp8_weight_kernel(const uint16_t* w, int N, int K, uint8_t* q, float* sf,
                                                         uint8_t* qt, float* sft) {
  constexpr int PITCH = BLOCK + 4;
  __shared__ uint8_t tile[BLOCK * PITCH];
  __shared__ uint32_t top[4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int nbn = (N + BLOCK - 1) / BLOCK, nbk = (K + BLOCK - 1) / BLOCK;
  const int64_t b = blockIdx.x / ((int64_t)nbn * nbk);
  const int in = (int)(blockIdx.x - b * nbn * nbk), bn = in / nbk, bk = in % nbk;
  const int n0 = bn * BLOCK, k0 = bk * BLOCK;
  w += b * N * K;
  // thread: 8 columns 8 (tid & 15), rows tid / 16 + 16 i
  const int k = k0 + 8 * (tid & 15);
  u32x4_t v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int n = n0 + (tid >> 4) + 16 * i;
    v[i] = u32x4_t{0u, 0u, 0u, 0u};
    if (n < N && k < K) v[i] = ld8(w + (int64_t)n * K + k);
    m = max(m, amax8(v[i]));
  }
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, s));
  if (lane == 0) top[tid >> 6] = m;
  __syncthreads();
  m = max(max(top[0], top[1]), max(top[2], top[3]));
  const float scale = fmaxf(__fdiv_rn(__uint_as_float(m << 16), 448.0f), 0x1p-126f);
  if (tid == 0) {
    sf[b * nbn * nbk + (int64_t)bn * nbk + bk] = scale;
    if (sft) sft[b * nbn * nbk + (int64_t)bk * nbn + bn] = scale;
  }
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int row = (tid >> 4) + 16 * i, n = n0 + row;
    float f[8];
    unpack8(v[i], f);
    u32x2_t o;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      float e[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float x = f[4 * h + j];
        // (the quotient of the largest one may come out above 448)
        e[j] = fabsf(x) < __builtin_inff() ? fminf(fmaxf(__fdiv_rn(x, scale), -448.0f), 448.0f) : x;
      }
      i16x2_t r = {0, 0};
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, e[0], e[1], 1.0f, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, e[2], e[3], 1.0f, true);
      o[h] = __builtin_bit_cast(uint32_t, r);
    }
    if (n < N && k < K) st8(q + b * N * K + (int64_t)n * K + k, o);
    if (qt) {
      *reinterpret_cast<uint32_t*>(tile + PITCH * row + 8 * (tid & 15)) = o[0];
      *reinterpret_cast<uint32_t*>(tile + PITCH * row + 8 * (tid & 15) + 4) = o[1];
    }
  }
  if (!qt) return;
  __syncthreads();
  // thread: 8 rows 8 (tid & 15) of w, columns tid / 16 + 16 i
  const int n = n0 + 8 * (tid & 15);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int col = (tid >> 4) + 16 * i;
    u32x2_t o;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      uint32_t p = 0;
#pragma unroll
      for (int j = 0; j < 4; j++) p |= (uint32_t)tile[PITCH * (8 * (tid & 15) + 4 * h + j) + col] << (8 * j);
      o[h] = p;
    }
    if (k0 + col < K && n < N) st8(qt + b * N * K + (int64_t)(k0 + col) * N + n, o);
  }
}

// Wavefronts of a row of `cols` values and the grid of them, four a workgroup (up to
// 2^22 tokens of 32 pieces: 2^25 workgroups)
int parts_of(int cols, int u) { return (cols + PIECE * u - 1) / (PIECE * u); }
dim3 grid_of(int64_t rows, int parts) {
  const int64_t n = (rows * parts + 3) / 4;
  if (n <= ROW_OF_GRID) return dim3((unsigned)n);
  return dim3((unsigned)ROW_OF_GRID, (unsigned)((n + ROW_OF_GRID - 1) / ROW_OF_GRID));
}

// Few rows: a piece a wavefront, so that all of them are on their way at once; many:
// several, whose loads go out together.  Rows quantised, one piece and four: 8 x 6144
// 2.4 us and 2.7, 2048 x 4096 5.4 and 4.9, 16384 x 4096 33.5 and 30.2 (6.7 TB/s);
// activations, one and two: 301 x 1536 3.4 and 4.3, 65536 x 2048 226 and 207.
bool few(int64_t rows, int cols) { return rows * parts_of(cols, 1) <= 4096; }

}  // namespace

hipError_t launch_quantize_fp8(const uint16_t* x, int64_t stride, int64_t rows, int cols, uint8_t* q, uint8_t* sf,
                               hipStream_t s) {
  if (few(rows, cols)) {
    const int p = parts_of(cols, 1);
    fp8_rows_kernel<1><<<grid_of(rows, p), 256, 0, s>>>(x, stride, rows, cols, p, q, sf);
  } else {
    const int p = parts_of(cols, 4);
    fp8_rows_kernel<4><<<grid_of(rows, p), 256, 0, s>>>(x, stride, rows, cols, p, q, sf);
  }
  return hipGetLastError();
}

hipError_t launch_quantize_fp8_weight(const uint16_t* w, int batches, int N, int K, uint8_t* q, float* sf, uint8_t* qt,
                                      float* sft, hipStream_t s) {
  const int64_t blocks = (int64_t)batches * ((N + BLOCK - 1) / BLOCK) * ((K + BLOCK - 1) / BLOCK);
  fp8_weight_kernel<<<(unsigned)blocks, 256, 0, s>>>(w, N, K, q, sf, qt, sft);
  return hipGetLastError();
}

// (With codes, one piece and two: 512 tokens of 8 routes of 4096 5.7 us and 7.3, 65536
// of about one route of 6144 219 and 174; bf16 alone is no faster in two, those 231 and
// 252.)
hipError_t launch_dispatch(const DispatchParams& a, hipStream_t s) {
  if (few(a.M, a.H) || !a.q) {
    const int p = parts_of(a.H, 1);
    dispatch_kernel<1><<<grid_of(a.M, p), 256, 0, s>>>(a, p);
  } else {
    const int p = parts_of(a.H, 2);
    dispatch_kernel<2><<<grid_of(a.M, p), 256, 0, s>>>(a, p);
  }
  return hipGetLastError();
}

hipError_t launch_dispatch_backward(const uint16_t* dxp, const int32_t* slots, int64_t M, int top_k, int H,
                                    int accumulate, uint16_t* dx, hipStream_t s) {
  const int p = parts_of(H, 1);
  dispatch_backward_kernel<<<grid_of(M, p), 256, 0, s>>>(dxp, slots, M, top_k, H, accumulate, p, dx);
  return hipGetLastError();
}

hipError_t launch_finalize_backward(const FinalizeBackwardParams& a, hipStream_t s) {
  const unsigned grid = (unsigned)a.M;
  switch ((a.H + 2047) / 2048) {
    case 1: finalize_backward_kernel<1><<<grid, 256, 0, s>>>(a); break;
    case 2: finalize_backward_kernel<2><<<grid, 256, 0, s>>>(a); break;
    case 3: finalize_backward_kernel<3><<<grid, 256, 0, s>>>(a); break;
    case 4: finalize_backward_kernel<4><<<grid, 256, 0, s>>>(a); break;
    default: finalize_backward_kernel<8><<<grid, 256, 0, s>>>(a); break;
  }
  return hipGetLastError();
}

template <int AK>
hipError_t act_as(const ActParams& a, hipStream_t s) {
  if (few(a.rows, a.I)) {
    const int p = parts_of(a.I, 1);
    act_kernel<AK, 1><<<grid_of(a.rows, p), 256, 0, s>>>(a, p);
  } else {
    const int p = parts_of(a.I, 2);
    act_kernel<AK, 2><<<grid_of(a.rows, p), 256, 0, s>>>(a, p);
  }
  return hipGetLastError();
}
template <int AK>
hipError_t act_backward_as(const ActBackwardParams& a, hipStream_t s) {
  if (few(a.rows, a.I)) {
    const int p = parts_of(a.I, 1);
    act_backward_kernel<AK, 1><<<grid_of(a.rows, p), 256, 0, s>>>(a, p);
  } else {
    const int p = parts_of(a.I, 2);
    act_backward_kernel<AK, 2><<<grid_of(a.rows, p), 256, 0, s>>>(a, p);
  }
  return hipGetLastError();
}

hipError_t launch_act(const ActParams& a, hipStream_t s) {
  return a.act.kind == ACT_GEGLU_TANH ? act_as<ACT_GEGLU_TANH>(a, s) : act_as<ACT_SWIGLU>(a, s);
}
hipError_t launch_act_backward(const ActBackwardParams& a, hipStream_t s) {
  return a.act.kind == ACT_GEGLU_TANH ? act_backward_as<ACT_GEGLU_TANH>(a, s) : act_backward_as<ACT_SWIGLU>(a, s);
}

}  // namespace moe
