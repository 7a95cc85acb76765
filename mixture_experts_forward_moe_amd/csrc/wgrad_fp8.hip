// wgrad_fp8.hip -- the gradient of a product's weights, dW = dy^T x, from rows of
// x kept in 8 bits: of one matrix, or of every expert from its rows.
//
// x's codes are decoded to bf16 once, on their way into LDS, where both operands
// lie with the rows (the sum's index) apart; a code times a power of two is exact
// in bf16, so the products are exact and the sums fp32.
#include "device_common.h"
#include "internal.h"

namespace moe {

namespace {

// 16 codes under one E8M0 code as bf16 pairs
DEV void decode16(const u32x4_t& c, uint32_t code, uint32_t (&o)[8]) {
  const float s = e8m0_scale_operand(code);
#pragma unroll
  for (int i = 0; i < 4; i++) {
    o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, false));
    o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, true));
  }
}

constexpr int BN = 128, BK = 128, ST = 32;

__global__ __launch_bounds__(256) void wgrad_simple_kernel(const WgradParams a, int tiles_n, int tiles_k) {
  constexpr int P = ST + 8;
  __shared__ __attribute__((aligned(16))) uint16_t dn[BN * P], xk[BK * P];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = blockIdx.x / (tiles_n * tiles_k), t = blockIdx.x - e * tiles_n * tiles_k;
  const int n0 = t / tiles_k * BN, k0 = t % tiles_k * BK;
  const int64_t first = a.offsets ? ld_uniform(a.offsets + e) : 0;
  const int64_t end = a.offsets ? first + ld_uniform(a.counts + e) : a.M;
  const int nb = (a.K + 127) / 128;
  f32x4_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int wn = 64 * (wave & 1), wk = 64 * (wave >> 1), r = lane & 15, q = lane >> 4;
  for (int64_t m0 = first; m0 < end; m0 += ST) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int m = (tid >> 4) + 16 * i, n = 8 * (tid & 15);
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (m0 + m < end && n0 + n < a.N) v = *reinterpret_cast<const u32x4_t*>(a.dy + (m0 + m) * a.N + n0 + n);
#pragma unroll
      for (int j = 0; j < 8; j++) dn[(n + j) * P + m] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
    }
    {
      const int m = tid >> 3, k = 16 * (tid & 7);
      uint32_t o[8] = {};
      if (m0 + m < end && k0 + k < a.K)
        decode16(*reinterpret_cast<const u32x4_t*>(a.x + (m0 + m) * a.K + k0 + k),
                 a.x_sf[(m0 + m) * nb + (k0 >> 7)], o);
#pragma unroll
      for (int j = 0; j < 16; j++) xk[(k + j) * P + m] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
    }
    __syncthreads();
    bf16x8_t f[4], g[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[i] = *reinterpret_cast<const bf16x8_t*>(dn + (wn + 16 * i + r) * P + 8 * q);
      g[i] = *reinterpret_cast<const bf16x8_t*>(xk + (wk + 16 * i + r) * P + 8 * q);
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[i], g[j], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const int n = n0 + wn + 16 * i + 4 * q + c, k = k0 + wk + 16 * j + r;
        if (n >= a.N || k >= a.K) continue;
        float* p = a.dw + ((int64_t)e * a.N + n) * a.K + k;
        *p = a.accumulate ? *p + acc[i][j][c] : acc[i][j][c];
      }
}

}  // namespace

hipError_t launch_wgrad_fp8(const WgradParams& a, hipStream_t s) {
  const int tn = (a.N + BN - 1) / BN, tk = (a.K + BK - 1) / BK;
  wgrad_simple_kernel<<<(unsigned)((int64_t)a.experts * tn * tk), 256, 0, s>>>(a, tn, tk);
  return hipGetLastError();
}

}  // namespace moe
