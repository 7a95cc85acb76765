// norm.hip -- the residual addition with the root-mean-square norm that makes
// the experts' input (bf16 and, in the same pass, its MX codes), and the
// norm's gradients.
//
//   h = bf16(x + residual);  r = 1 / sqrt(mean(h^2) + eps);  y = bf16(h r w)
//   dx = bf16(dh + r g - h r^3 mean(g h)),  g = dy w;  dw = sum_rows dy h r
//
// No operand is used more than a few times: both passes are bound by HBM.  A
// row stays in registers between the sum of squares and the output, so every
// byte is moved once.  A thread owns vectors of 8 consecutive values (16
// bytes); a quad of lanes holds a 32-value MX block, whose maximum is two DPP
// steps.
#include "device_common.h"
#include "internal.h"

namespace moe {

namespace {

// values of lanes XOR 1 / 2 of a quad, and of the mirrored half row / row:
// max or sum over 16 lanes in four steps
template <int CTRL>
DEV float dpp(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
constexpr int QUAD_XOR1 = 0xB1, QUAD_XOR2 = 0x4E, ROW_HALF_MIRROR = 0x141, ROW_MIRROR = 0x140;

DEV float wave_sum(float v) {
  v += dpp<QUAD_XOR1>(v);
  v += dpp<QUAD_XOR2>(v);
  v += dpp<ROW_HALF_MIRROR>(v);
  v += dpp<ROW_MIRROR>(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// Sum over the T threads of a row; `red` is this step's LDS scratch (one
// float a wave), not in use by a wave that could still be one step behind.
template <int T>
DEV float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < T / 64; w++) v += red[w];
  }
  return v;
}

DEV void unpack8(const u32x4_t& v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
DEV u32x4_t pack8(const float (&f)[8]) {
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  return v;
}

// eight weights from column c
DEV void load_weight8(const void* w, int f32, int c, float (&f)[8]) {
  if (f32) {
    const f32x4_t* p = reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(w) + c);
    const f32x4_t a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[i] = a[i];
      f[4 + i] = b[i];
    }
  } else {
    unpack8(*reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint16_t*>(w) + c), f);
  }
}

// T threads a row (64: four rows a workgroup), up to VPT vectors a thread.
template <int T, int VPT>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rmsnorm_kernel(const NormParams a) {
  constexpr int ROWS = T < 256 ? 256 / T : 1;
  __shared__ float red[2][T > 64 ? T / 64 : 1];
  const int t = threadIdx.x % T;
  const int nv = a.H / 8;
  int step = 0;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / T; row < a.M;
       row += (int64_t)gridDim.x * ROWS, step ^= 1) {
    const uint16_t* x = a.x + row * a.x_row_stride;
    const uint16_t* res = a.residual ? a.residual + row * a.residual_row_stride : nullptr;
    u32x4_t h[VPT], rv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; i++) {
      const int v = t + T * i;
      h[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (v < nv) h[i] = *reinterpret_cast<const u32x4_t*>(x + 8 * v);
    }
    if (res) {
#pragma unroll
      for (int i = 0; i < VPT; i++) {
        const int v = t + T * i;
        rv[i] = u32x4_t{0u, 0u, 0u, 0u};
        if (v < nv) rv[i] = *reinterpret_cast<const u32x4_t*>(res + 8 * v);
      }
    }
    float s8[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};  // short chains: a closer sum
#pragma unroll
    for (int i = 0; i < VPT; i++) {
      float f[8];
      unpack8(h[i], f);
      if (res) {
        float g[8];
        unpack8(rv[i], g);
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] += g[j];
        h[i] = pack8(f);  // the stream keeps bf16: normalise what is stored
        unpack8(h[i], f);
      }
#pragma unroll
      for (int j = 0; j < 8; j++) s8[j] = fmaf(f[j], f[j], s8[j]);
    }
    const float ss =
        row_sum<T>(((s8[0] + s8[1]) + (s8[2] + s8[3])) + ((s8[4] + s8[5]) + (s8[6] + s8[7])), red[step]);
    // once a row, in fp64: r's own rounding moves every bf16 decision of the row
    const float r = (float)(1.0 / sqrt((double)ss / a.H + (double)a.eps));
    if (a.rstd && t == 0) a.rstd[row] = r;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
      const int v = t + T * i;
      if (v >= nv) continue;
      if (a.residual_out) *reinterpret_cast<u32x4_t*>(a.residual_out + row * a.H + 8 * v) = h[i];
      float f[8], w[8];
      unpack8(h[i], f);
      load_weight8(a.weight, a.weight_f32, 8 * v, w);
#pragma unroll
      for (int j = 0; j < 8; j++) f[j] = f[j] * r * w[j];
      const u32x4_t y = pack8(f);
      if (a.y) *reinterpret_cast<u32x4_t*>(a.y + row * a.H + 8 * v) = y;
      if (a.q) {
        unpack8(y, f);  // quantised from the bf16 value, as a separate pass would
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++) m = fmaxf(m, fabsf(f[j]));
        m = fmaxf(m, dpp<QUAD_XOR1>(m));
        m = fmaxf(m, dpp<QUAD_XOR2>(m));
        uint32_t code;
        const int64_t at = row * a.H + 8 * v;
        if (a.elem == 0) {
          code = mx_scale_code(m, 8);
          uint2 o;
          o.x = f32x2_to_e4m3x2_mx(f[0], f[1], code) | (f32x2_to_e4m3x2_mx(f[2], f[3], code) << 16);
          o.y = f32x2_to_e4m3x2_mx(f[4], f[5], code) | (f32x2_to_e4m3x2_mx(f[6], f[7], code) << 16);
          *reinterpret_cast<uint2*>(a.q + at) = o;
        } else {
          code = mx_scale_code(m, 2);
          const float s = e8m0_scale_operand(code);
          uint32_t o = 0;
#pragma unroll
          for (int j = 0; j < 4; j++) o |= f32x2_to_e2m1x2(f[2 * j], f[2 * j + 1], s) << (8 * j);
          *reinterpret_cast<uint32_t*>(a.q + at / 2) = o;
        }
        if ((t & 3) == 0) a.q_sf[at / 32] = (uint8_t)code;
      }
    }
  }
}

template <int T, int VPT>
hipError_t launch_norm(const NormParams& p, hipStream_t s) {
  constexpr int ROWS = T < 256 ? 256 / T : 1;
  const int64_t blocks = (p.M + ROWS - 1) / ROWS;
  rmsnorm_kernel<T, VPT><<<(unsigned)(blocks < (1 << 20) ? blocks : 1 << 20), T < 256 ? 256 : T, 0, s>>>(p);
  return hipGetLastError();
}

// Rows are walked by a fixed set of workgroups (row b, b + P, ...), each
// keeping its columns' sums of dy h r in registers: the weight gradient costs
// one [P, H] array of partial sums instead of a second pass over the rows.
template <int T, int VPT>
__global__ __launch_bounds__(T) void rmsnorm_backward_kernel(const NormBackwardParams a) {
  __shared__ float red[2][T / 64];
  const int t = threadIdx.x;
  const int nv = a.H / 8;
  float w[VPT][8], acc[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; i++) {
#pragma unroll
    for (int j = 0; j < 8; j++) w[i][j] = acc[i][j] = 0.0f;
    if (t + T * i < nv) load_weight8(a.weight, a.weight_f32, 8 * (t + T * i), w[i]);
  }
  int step = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, step ^= 1) {
    const u32x4_t zero = {0u, 0u, 0u, 0u};
    u32x4_t dy[VPT], h[VPT], dh[VPT];
#pragma unroll
    for (int i = 0; i < VPT; i++) {
      const int v = t + T * i;
      const int64_t at = row * a.H + 8 * v;
      dy[i] = h[i] = dh[i] = zero;
      if (v < nv) {
        dy[i] = *reinterpret_cast<const u32x4_t*>(a.dy + at);
        h[i] = *reinterpret_cast<const u32x4_t*>(a.h + at);
        if (a.dh) dh[i] = *reinterpret_cast<const u32x4_t*>(a.dh + at);
      }
    }
    const float r = a.rstd[row];
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
      float d[8], f[8];
      unpack8(dy[i], d);
      unpack8(h[i], f);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float n = f[j] * r;
        acc[i][j] = fmaf(d[j], n, acc[i][j]);
        c = fmaf(d[j] * w[i][j], n, c);
      }
    }
    c = row_sum<T>(c, red[step]) / (float)a.H;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
      const int v = t + T * i;
      if (v >= nv) continue;
      float d[8], f[8], e[8];
      unpack8(dy[i], d);
      unpack8(h[i], f);
      unpack8(dh[i], e);
#pragma unroll
      for (int j = 0; j < 8; j++) f[j] = e[j] + r * (d[j] * w[i][j] - f[j] * r * c);
      *reinterpret_cast<u32x4_t*>(a.dx + row * a.H + 8 * v) = pack8(f);
    }
  }
  if (a.partial) {
#pragma unroll
    for (int i = 0; i < VPT; i++) {
      const int v = t + T * i;
      if (v >= nv) continue;
      f32x4_t* o = reinterpret_cast<f32x4_t*>(a.partial + (int64_t)blockIdx.x * a.H + 8 * v);
      o[0] = f32x4_t{acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
      o[1] = f32x4_t{acc[i][4], acc[i][5], acc[i][6], acc[i][7]};
    }
  }
}

// dweight[c] = sum over P partial rows, 32 columns a workgroup: 8 lanes of
// four columns, 32 row groups, joined in a fixed order.
__global__ __launch_bounds__(256) void dweight_kernel(const float* __restrict__ partial, int P, int H,
                                                      float* __restrict__ dweight) {
  __shared__ float sum[32][33];
  const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3;
  const int c0 = blockIdx.x * 32 + 4 * cg;
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c0 < H) {
    for (int p = rg; p < P; p += 32) s += *reinterpret_cast<const f32x4_t*>(partial + (int64_t)p * H + c0);
  }
#pragma unroll
  for (int j = 0; j < 4; j++) sum[rg][4 * cg + j] = s[j];
  __syncthreads();
  const int c = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x < 32 && c < H) {
    float v = 0.0f;
    for (int g = 0; g < 32; g++) v += sum[g][threadIdx.x];
    dweight[c] = v;
  }
}

template <int T, int VPT>
hipError_t launch_back(const NormBackwardParams& p, hipStream_t s) {
  rmsnorm_backward_kernel<T, VPT><<<norm_backward_partials(p.M), T, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

int norm_backward_partials(int64_t M) {
  const int64_t p = (M + 15) / 16;
  return (int)(p < 1 ? 1 : p > 512 ? 512 : p);
}

hipError_t launch_rmsnorm(const NormParams& p, hipStream_t s) {
  const int nv = p.H / 8;
  if (p.M >= 2048 && nv <= 64 * 12) {
    if (nv <= 64) return launch_norm<64, 1>(p, s);
    if (nv <= 64 * 2) return launch_norm<64, 2>(p, s);
    if (nv <= 64 * 4) return launch_norm<64, 4>(p, s);
    if (nv <= 64 * 8) return launch_norm<64, 8>(p, s);
    return launch_norm<64, 12>(p, s);
  }
  if (nv <= 256) return launch_norm<256, 1>(p, s);
  if (nv <= 1024) return launch_norm<1024, 1>(p, s);
  if (nv <= 2048) return launch_norm<1024, 2>(p, s);
  return launch_norm<1024, 4>(p, s);
}

hipError_t launch_rmsnorm_backward(const NormBackwardParams& p, float* dweight, hipStream_t s) {
  const int nv = p.H / 8;
  hipError_t e = hipSuccess;
  if (p.M > 0) {
    if (nv <= 256) e = launch_back<256, 1>(p, s);
    else if (nv <= 512) e = launch_back<256, 2>(p, s);
    else if (nv <= 768) e = launch_back<256, 3>(p, s);
    else if (nv <= 1024) e = launch_back<256, 4>(p, s);
    else if (nv <= 2048) e = launch_back<1024, 2>(p, s);
    else e = launch_back<1024, 4>(p, s);
    if (e != hipSuccess) return e;
  }
  if (!dweight) return hipSuccess;
  dweight_kernel<<<(p.H + 31) / 32, 256, 0, s>>>(p.partial, p.M > 0 ? norm_backward_partials(p.M) : 0, p.H, dweight);
  return hipGetLastError();
}

}  // namespace moe
