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

DEV float wave_sum(float v) {
  v += dpp_f32<DPP_XOR1>(v);
  v += dpp_f32<DPP_XOR2>(v);
  v += dpp_f32<DPP_HALF_MIRROR>(v);
  v += dpp_f32<DPP_MIRROR>(v);
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

// 16 bytes of a row; PAST: past the caches, where the rows are more than they
// hold (a consumer would find none of them there)
template <bool PAST>
DEV u32x4_t get16(const uint16_t* p) {
  const u32x4_t* q = reinterpret_cast<const u32x4_t*>(p);
  if constexpr (PAST) return __builtin_nontemporal_load(q);
  else return *q;
}
template <bool PAST>
DEV void put16(uint16_t* p, const u32x4_t& v) {
  if constexpr (PAST) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(p));
  else *reinterpret_cast<u32x4_t*>(p) = v;
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
// 65536 x 6144 with the residual and E4M3 codes: 3.64 GB in 594 - 630 us, 5.8 - 6.1
// TB/s (a large copy reaches 4.7).
template <int T, int VPT, bool PAST>
__global__ __launch_bounds__(T < 128 ? 256 : T) void rmsnorm_kernel(const NormParams a) {
  constexpr int ROWS = T < 128 ? 256 / T : 1;
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
      if (v < nv) h[i] = get16<PAST>(x + 8 * v);
    }
    if (res) {
#pragma unroll
      for (int i = 0; i < VPT; i++) {
        const int v = t + T * i;
        rv[i] = u32x4_t{0u, 0u, 0u, 0u};
        if (v < nv) rv[i] = get16<PAST>(res + 8 * v);
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
      if (a.residual_out) put16<PAST>(a.residual_out + row * a.H + 8 * v, h[i]);
      float f[8], w[8];
      unpack8(h[i], f);
      load_weight8(a.weight, a.weight_f32, 8 * v, w);
#pragma unroll
      for (int j = 0; j < 8; j++)
        f[j] = r > 0.0f ? f[j] * w[j] * r : f[j] * r;  // (h w is exact for a bf16 weight, or past fp32 where r is 0)
      const u32x4_t y = pack8(f);
      if (a.y) put16<PAST>(a.y + row * a.H + 8 * v, y);
      if (a.q) {
        unpack8(y, f);  // quantised from the bf16 value, as a separate pass would
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++) m = fmaxf(m, fabsf(f[j]));
        const int64_t at = row * a.H + 8 * v;
        const uint32_t code = mx_store8(f, m, a.elem, a.q, at);
        if ((t & 3) == 0) a.q_sf[at / 32] = (uint8_t)code;
      }
    }
  }
}

// MANY: rows past the caches' size can come here
template <int T, int VPT, bool MANY = true>
hipError_t launch_norm(const NormParams& p, hipStream_t s) {
  constexpr int ROWS = T < 128 ? 256 / T : 1;
  const int64_t blocks = (p.M + ROWS - 1) / ROWS;
  const unsigned grid = (unsigned)(blocks < 1 << 20 ? blocks : 1 << 20);
  if (MANY && p.past_caches) rmsnorm_kernel<T, VPT, MANY><<<grid, T < 128 ? 256 : T, 0, s>>>(p);
  else rmsnorm_kernel<T, VPT, false><<<grid, T < 128 ? 256 : T, 0, s>>>(p);
  return hipGetLastError();
}

// Rows are walked by a fixed set of workgroups (row b, b + P, ...), each
// keeping its columns' sums of dy h r in registers: the weight gradient costs
// one [P, H] array of partial sums instead of a second pass over the rows.
// The next row's loads go out before this row's sum is joined.  8191 x 4128 with
// dh: 270 MB in 53 - 56 us, 4.8 - 5.1 TB/s; the join of the partials takes 4 us, a launch.
template <int T, int VPT, bool PAST>
__global__ __launch_bounds__(T) void rmsnorm_backward_kernel(const NormBackwardParams a) {
  __shared__ float red[2][T > 64 ? T / 64 : 1];
  const int t = threadIdx.x;
  const int nv = a.H / 8;
  float w[VPT][8], acc[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; i++) {
#pragma unroll
    for (int j = 0; j < 8; j++) w[i][j] = acc[i][j] = 0.0f;
    if (t + T * i < nv) load_weight8(a.weight, a.weight_f32, 8 * (t + T * i), w[i]);
  }
  struct Row {
    u32x4_t dy[VPT], h[VPT], dh[VPT];
    float r;
  };
  auto load = [&](int64_t row) {
    const u32x4_t zero = {0u, 0u, 0u, 0u};
    Row x;
    x.r = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; i++) x.dy[i] = x.h[i] = x.dh[i] = zero;
    if (row < a.M) {
      x.r = a.rstd[row];
#pragma unroll
      for (int i = 0; i < VPT; i++) {
        const int v = t + T * i;
        const int64_t at = row * a.H + 8 * v;
        if (v < nv) {
          x.dy[i] = get16<PAST>(a.dy + at);
          x.h[i] = get16<PAST>(a.h + at);
          if (a.dh) x.dh[i] = get16<PAST>(a.dh + at);
        }
      }
    }
    return x;
  };
  int step = 0;
  Row x = load(blockIdx.x);
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, step ^= 1) {
    const Row next = load(row + gridDim.x);
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
      float d[8], f[8];
      unpack8(x.dy[i], d);
      unpack8(x.h[i], f);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float n = f[j] * x.r;
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
      unpack8(x.dy[i], d);
      unpack8(x.h[i], f);
      unpack8(x.dh[i], e);
#pragma unroll
      for (int j = 0; j < 8; j++) f[j] = e[j] + x.r * (d[j] * w[i][j] - f[j] * x.r * c);
      put16<PAST>(a.dx + row * a.H + 8 * v, pack8(f));
    }
    x = next;
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
// four columns, 128 row groups, joined in a fixed order.
__global__ __launch_bounds__(1024) void dweight_kernel(const float* __restrict__ partial, int P, int H,
                                                       float* __restrict__ dweight) {
  __shared__ float sum[128][33];
  const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3;
  const int c0 = blockIdx.x * 32 + 4 * cg;
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c0 < H) {
    for (int p = rg; p < P; p += 128) s += *reinterpret_cast<const f32x4_t*>(partial + (int64_t)p * H + c0);
  }
#pragma unroll
  for (int j = 0; j < 4; j++) sum[rg][4 * cg + j] = s[j];
  __syncthreads();
  const int c = threadIdx.x >> 5, g = threadIdx.x & 31;
  float v = (sum[g][c] + sum[g + 32][c]) + (sum[g + 64][c] + sum[g + 96][c]);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) v += __shfl_xor(v, d);
  if (g == 0 && blockIdx.x * 32 + c < H) dweight[blockIdx.x * 32 + c] = v;
}

template <int T, int VPT>
hipError_t launch_back(const NormBackwardParams& p, hipStream_t s) {
  const int grid = norm_backward_partials(p.M, p.H);
  if (p.past_caches) rmsnorm_backward_kernel<T, VPT, true><<<grid, T, 0, s>>>(p);
  else rmsnorm_backward_kernel<T, VPT, false><<<grid, T, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

// Threads of a row in the backward pass: 16 bytes each up to 256 threads.
static int backward_threads(int H) { return H <= 512 ? 64 : H <= 1024 ? 128 : H <= 8192 ? 256 : 512; }

// Workgroups of the backward pass: two rows each at least, 131072 threads at
// most, which fill the CUs.
int norm_backward_partials(int64_t M, int H) {
  const int64_t p = (M + 1) / 2, most = 131072 / backward_threads(H);
  return (int)(p < 1 ? 1 : p > most ? most : p);
}

hipError_t launch_rmsnorm(const NormParams& p, hipStream_t s) {
  const int nv = p.H / 8;
  // Many rows: 256 threads each, so that a CU has several rows under way; few: as
  // many threads as vectors, for the shortest chain.  (256 threads against 1024,
  // us.  H = 6144: 64 rows 4.5, 3.7; 512 7.9, 7.4; 1024 11.7, 12.5; 4096 47, 46.
  // H = 8192: 512 10.0, 9.0; 1024 15.7, 15.2; 2048 32.5, 33.3.  Shorter rows, which
  // leave half of the 1024 threads without work, meet earlier: H = 4096 256 rows
  // 4.4, 4.2; 512 5.3, 6.4; 1024 9.3, 10.2; H = 2080 256 3.9, 3.9; 512 4.4, 5.6; 1024 6.5,
  // 9.1.  65536 x 6144 in a wavefront a row with 12 vectors: 976, against 637.)
  if (nv <= 64) return launch_norm<64, 1>(p, s);
  if (nv <= 128) return launch_norm<128, 1>(p, s);
  if (nv <= 256) return launch_norm<256, 1>(p, s);
  if (p.M >= 1024) {
    if (nv <= 512) return launch_norm<256, 2>(p, s);
    if (nv <= 768) return launch_norm<256, 3>(p, s);
    if (nv <= 1024) return launch_norm<256, 4>(p, s);
  }
  if (nv <= 1024) return launch_norm<1024, 1, false>(p, s);  // (fewer than 1024 rows of at most 8192 values)
  return launch_norm<1024, 2>(p, s);
}

hipError_t launch_rmsnorm_backward(const NormBackwardParams& p, float* dweight, hipStream_t s) {
  const int nv = p.H / 8;
  hipError_t e = hipSuccess;
  if (p.M > 0) {
    if (nv <= 64) e = launch_back<64, 1>(p, s);
    else if (nv <= 128) e = launch_back<128, 1>(p, s);
    else if (nv <= 256) e = launch_back<256, 1>(p, s);
    else if (nv <= 512) e = launch_back<256, 2>(p, s);
    else if (nv <= 768) e = launch_back<256, 3>(p, s);
    else if (nv <= 1024) e = launch_back<256, 4>(p, s);
    else e = launch_back<512, 4>(p, s);
    if (e != hipSuccess) return e;
  }
  if (!dweight) return hipSuccess;
  dweight_kernel<<<(p.H + 31) / 32, 1024, 0, s>>>(p.partial, p.M > 0 ? norm_backward_partials(p.M, p.H) : 0, p.H, dweight);
  return hipGetLastError();
}

}  // namespace moe
