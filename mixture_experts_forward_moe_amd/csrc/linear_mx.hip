// linear_mx.hip -- y = alpha * x W^T + bias for MX operands without a routing
// plan: x E4M3 or E2M1, W E2M1, E8M0 scales per 32 values along K.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes both operands as they are stored,
// with their E8M0 bytes, so nothing is decoded.  A wavefront computes a
// 16 x 16 tile: lane (row r = lane & 15, group q = lane >> 4) holds, of each
// 128 values of K, block q of an E2M1 row (16 bytes) or the two halves
// 16 q .. and 64 + 16 q .. of an E4M3 row, and block q's scale.
#include "device_common.h"
#include "internal.h"

namespace moe {

namespace {

constexpr int LT = 256;

DEV u32x4_t ld16(const uint8_t* p) { return *reinterpret_cast<const u32x4_t*>(p); }

template <int XE>
DEV void load_x(const LinearParams& a, int64_t row, int k, int q, i32x8_t& v, int& sc) {
  const u32x4_t z = {0u, 0u, 0u, 0u};
  u32x4_t lo = z, hi = z;
  if (XE == 1) {
    if (k + 32 * q < a.K) lo = ld16(a.x + row * (a.K / 2) + k / 2 + 16 * q);
  } else {
    if (k + 16 * q < a.K) lo = ld16(a.x + row * a.K + k + 16 * q);
    if (k + 64 + 16 * q < a.K) hi = ld16(a.x + row * a.K + k + 64 + 16 * q);
  }
  v = i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  sc = k + 32 * q < a.K ? a.x_sf[row * (a.K / 32) + k / 32 + q] : 0;
}

template <int XE>
__global__ __launch_bounds__(LT) void linear_kernel(const LinearParams a, int n_tiles, int64_t tiles) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int64_t tile = (int64_t)blockIdx.x * (LT / 64) + (threadIdx.x >> 6);
  if (tile >= tiles) return;
  const int64_t m0 = tile / n_tiles * 16;
  const int n0 = (int)(tile % n_tiles) * 16;
  const int64_t xr = min((int64_t)a.M - 1, m0 + r);
  const int64_t wr = min(a.N - 1, n0 + r);
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = 0; k < a.K; k += 128) {
    i32x8_t xv;
    int xs, ws = 0;
    load_x<XE>(a, xr, k, q, xv, xs);
    u32x4_t w = {0u, 0u, 0u, 0u};
    if (k + 32 * q < a.K) {
      w = ld16(a.w + wr * (a.K / 2) + k / 2 + 16 * q);
      ws = a.w_sf[wr * (a.K / 32) + k / 32 + q];
    }
    const i32x8_t wv = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(xv, wv, acc, XE == 1 ? 4 : 0, 4, 0, xs, 0, ws);
  }
  // element i of lane (r, q): row 4 q + i, column r
  const int n = n0 + r;
  if (n >= a.N) return;
  const float alpha = a.alpha ? *a.alpha : 1.0f;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t m = m0 + 4 * q + i;
    if (m >= a.M) continue;
    float v = acc[i] * alpha;
    if (a.bias) v += a.bias[n];
    const int64_t at = m * a.N + n;
    if (a.y_f32) {
      float* y = reinterpret_cast<float*>(a.y) + at;
      *y = a.accumulate ? *y + v : v;
    } else {
      uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + at;
      *y = f32_to_bf16(a.accumulate ? bf16_to_f32(*y) + v : v);
    }
  }
}

}  // namespace

hipError_t launch_linear_mx(const LinearParams& p, hipStream_t s) {
  const int nt = (p.N + 15) / 16;
  const int64_t tiles = (int64_t)((p.M + 15) / 16) * nt;
  const unsigned grid = (unsigned)((tiles + LT / 64 - 1) / (LT / 64));
  if (p.x_elem == 1) linear_kernel<1><<<grid, LT, 0, s>>>(p, nt, tiles);
  else linear_kernel<0><<<grid, LT, 0, s>>>(p, nt, tiles);
  return hipGetLastError();
}

}  // namespace moe
