// linear_fp8.hip -- y = x W^T + bias of rows in 8 bits: x E4M3 with an E8M0
// byte for each 128 values of a row, W E4M3 with an fp32 scale for each block
// of 128 x 128; of one matrix, or of every expert's rows and weights.
//
// The matrix instruction takes x's bytes as its scale operand.  W's scales are
// any fp32 value, which it does not take: the product of each 128 of K is a
// sum of its own, from zero, that one fused multiply-add with W's scale adds to
// the fp32 sum.
#include "device_common.h"
#include "internal.h"

namespace moe {

namespace {

DEV u32x4_t ld16(const uint8_t* p) { return *reinterpret_cast<const u32x4_t*>(p); }

// rows [first, end) of a group of rows, and their matrix
struct Group {
  int64_t first, end;
  const uint8_t* w;
  const float* w_sf;
};

// group g of rows of `height` (with a plan: part of one of its tiles)
DEV bool group_of(const LinearFp8Params& a, int g, int height, Group& o) {
  if (!a.tile_expert) {
    o.first = (int64_t)g * height;
    o.end = min(a.M, o.first + height);
    o.w = a.w;
    o.w_sf = a.w_sf;
    return o.first < o.end;
  }
  const int parts = max(1, a.tile / height), t = g / parts;
  const int e = ld_uniform(a.tile_expert + t);
  if (e < 0) return false;
  o.first = (int64_t)t * a.tile + (g - t * parts) * height;
  o.end = min(o.first + height, (int64_t)ld_uniform(a.tile_limit + t));
  o.w = a.w + (int64_t)e * a.N * a.K;
  o.w_sf = a.w_sf + (int64_t)e * ((a.N + 127) / 128) * ((a.K + 127) / 128);
  return o.first < o.end;
}

constexpr int STREAM_WAVES = 8;

// 16 MT rows of x a workgroup: it streams 16 rows of W once, its wavefronts
// splitting K, straight into registers; their sums meet in LDS in a fixed order.
// v_mfma_scale_f32_16x16x128_f8f6f4: lane (row r = lane & 15, group q = lane
// >> 4) holds 32 values of K of its row; which ones is the same for both
// operands, and the scale is one for all of them.
template <int MT>
__global__ __launch_bounds__(64 * STREAM_WAVES) void fp8_stream_kernel(const LinearFp8Params a, int tiles_n) {
  constexpr int NW = STREAM_WAVES;
  __shared__ f32x4_t part[NW][MT][64];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = blockIdx.x / tiles_n, n0 = (blockIdx.x - g * tiles_n) * 16;
  Group o;
  if (!group_of(a, g, 16 * MT, o)) return;
  const int kb = (a.K + 127) / 128;
  const int per = (kb + NW - 1) / NW, s_first = wave * per, s_end = min(s_first + per, kb);
  const uint8_t* w = o.w + (int64_t)min(a.N - 1, n0 + r) * a.K + 16 * q;
  const float* wsf = o.w_sf + (int64_t)(n0 >> 7) * kb;
  const uint8_t *x[MT], *xsf[MT];
#pragma unroll
  for (int m = 0; m < MT; m++) {
    const int64_t row = min(o.first + 16 * m + r, o.end - 1);
    x[m] = a.x + row * a.K + 16 * q;
    xsf[m] = a.x_sf + row * kb;
  }
  f32x4_t acc[MT];
#pragma unroll
  for (int m = 0; m < MT; m++) acc[m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = s_first; s < s_end; s++) {
    const u32x4_t zero = {0u, 0u, 0u, 0u};
    const bool in0 = 128 * s + 16 * q < a.K, in1 = 128 * s + 64 + 16 * q < a.K;
    const u32x4_t w0 = in0 ? ld16(w + 128 * s) : zero, w1 = in1 ? ld16(w + 128 * s + 64) : zero;
    const float ws = wsf[s];
    const i32x8_t b = {(int)w0[0], (int)w0[1], (int)w0[2], (int)w0[3], (int)w1[0], (int)w1[1], (int)w1[2], (int)w1[3]};
#pragma unroll
    for (int m = 0; m < MT; m++) {
      const u32x4_t x0 = in0 ? ld16(x[m] + 128 * s) : zero, x1 = in1 ? ld16(x[m] + 128 * s + 64) : zero;
      const int xs = xsf[m][s];
      const i32x8_t c = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
      const f32x4_t none = {0.0f, 0.0f, 0.0f, 0.0f};
      const f32x4_t p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(c, b, none, 0, 0, 0, xs, 0, 127);
#pragma unroll
      for (int i = 0; i < 4; i++) acc[m][i] = fmaf(p[i], ws, acc[m][i]);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; m++) part[wave][m][lane] = acc[m];
  __syncthreads();
  // element i of lane (r, q): row 4 q + i, column r
  if (wave >= MT || n0 + r >= a.N) return;
  f32x4_t v = part[0][wave][lane];
#pragma unroll
  for (int k = 1; k < NW; k++) v += part[k][wave][lane];
  const int n = n0 + r;
  const float bias = a.bias ? a.bias[n] : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t row = o.first + 16 * wave + 4 * q + i;
    if (row >= o.end) continue;
    const float out = v[i] + bias;
    const int64_t at = row * a.N + n;
    if (a.y_f32) {
      float* y = reinterpret_cast<float*>(a.y) + at;
      *y = a.accumulate ? *y + out : out;
    } else {
      uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + at;
      *y = f32_to_bf16(a.accumulate ? bf16_to_f32(*y) + out : out);
    }
  }
}

template <int MT>
hipError_t launch_stream(const LinearFp8Params& a, hipStream_t s) {
  const int tn = (a.N + 15) / 16;
  const int64_t groups = a.tile_expert ? (int64_t)a.tiles * (a.tile > 16 * MT ? a.tile / (16 * MT) : 1)
                                       : (a.M + 16 * MT - 1) / (16 * MT);
  fp8_stream_kernel<MT><<<(unsigned)(groups * tn), 64 * STREAM_WAVES, 0, s>>>(a, tn);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_fp8(const LinearFp8Params& a, hipStream_t s) {
  const int64_t height = a.tile_expert ? a.tile : a.M;
  if (height <= 16) return launch_stream<1>(a, s);
  if (height <= 32) return launch_stream<2>(a, s);
  return launch_stream<4>(a, s);
}

}  // namespace moe
