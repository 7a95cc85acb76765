// linear_fp8.hip -- y = x W^T + bias of rows in 8 bits: x E4M3 with an E8M0
// byte for each 128 values of a row, W E4M3 with an fp32 scale for each block
// of 128 x 128; of one matrix, or of every expert's rows and weights.
//
// The matrix instruction takes x's bytes as its scale operand.  W's scales are
// any fp32 value, which it does not take: the product of each 128 of K is a
// sum of its own, from zero, that one fused multiply-add with W's scale adds to
// the fp32 sum.
#include <type_traits>

#include "device_common.h"
#include "dynamic_lds.h"
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

// group g of 16 rows: a plan's tile, which has as many
DEV bool group_of(const LinearFp8Params& a, int g, Group& o) {
  o.first = (int64_t)g * 16;
  if (!a.tile_expert) {
    o.end = min(a.M, o.first + 16);
    o.w = a.w;
    o.w_sf = a.w_sf;
    return true;
  }
  const int e = ld_uniform(a.tile_expert + g);
  if (e < 0) return false;
  o.end = ld_uniform(a.tile_limit + g);
  o.w = a.w + (int64_t)e * a.N * a.K;
  o.w_sf = a.w_sf + (int64_t)e * ((a.N + 127) / 128) * ((a.K + 127) / 128);
  return true;
}

// ------------------------------------------------------------- way out

// one value at element `at` of y
DEV void store_one(const LinearFp8Params& a, int64_t at, float v) {
  if (a.y_f32) {
    float* y = reinterpret_cast<float*>(a.y) + at;
    *y = a.accumulate ? *y + v : v;
  } else {
    uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + at;
    *y = f32_to_bf16(a.accumulate ? bf16_to_f32(*y) + v : v);
  }
}

// A wavefront's 16 TM x 16 TN results, rows m0 .. end, columns from n0.  WIDE:
// bf16 that is overwritten, its rows aligned to 16 bytes, leaves through the
// wavefront's own part of LDS, 16 rows at a time (chunks swizzled by the row), in whole
// lines.  Rows of odd sizes do value by value, from neighbouring lanes (16384 x 6147 x
// 4096: 533 us, 854 from the lanes that hold them), but in the kernels that split K,
// which have a tile each and wait for it, from the lanes that hold them (512 x 724 x
// 1024: 6.7 us, 8.0 through LDS).
template <typename S, bool WIDE>
DEV void store_tile(const LinearFp8Params& a, const f32x4_t (&acc)[S::TN][S::TM], int64_t m0, int64_t end, int n0,
                    uint8_t* out, int lane) {
  // (what follows from the lane is computed here, not held over the main loop, where
  // it would be spilled, and read back behind the stores)
  asm volatile("" : "+v"(lane));
  constexpr int TM = S::TM, TN = S::TN, W = 4 * TN;  // columns of a lane
  constexpr int C = 2 * TN;                          // chunks of 16 bytes in a row
  const int r = lane & 15, q = lane >> 4, n = n0 + W * q;
#pragma unroll
  for (int m = 0; m < TM; m++) {
    const int64_t row0 = m0 + 16 * m;
    if constexpr (WIDE) {
      if (row0 >= end) break;
#pragma unroll
      for (int c = 0; c < TN / 2; c++) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = acc[2 * c + (i >> 2)][m][i & 3];
        u32x4_t o;
#pragma unroll
        for (int i = 0; i < 4; i++) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<u32x4_t*>(out + 16 * (C * r + ((TN / 2 * q + c) ^ (r & (C - 1))))) = o;
      }
      wave_fence();  // the rows are read by other lanes
      constexpr int ROWS = 64 / C;  // rows a store
      const int c = lane % C;
      u32x4_t o[16 / ROWS];
#pragma unroll
      for (int i = 0; i < 16 / ROWS; i++) {
        const int rr = ROWS * i + lane / C;
        o[i] = *reinterpret_cast<const u32x4_t*>(out + 16 * (C * rr + (c ^ (rr & (C - 1)))));
      }
#pragma unroll
      for (int i = 0; i < 16 / ROWS; i++) {
        const int rr = ROWS * i + lane / C;
        if (row0 + rr < end && n0 + 8 * c < a.N)
          *reinterpret_cast<u32x4_t*>(reinterpret_cast<uint16_t*>(a.y) + (row0 + rr) * a.N + n0 + 8 * c) = o[i];
      }
      wave_fence();  // and written again once they have been
    } else {
      if (row0 >= end) break;
      // sixteen bytes at a time where y allows it
      const bool four = a.y_f32 && a.N % 4 == 0 && ((uintptr_t)a.y & 15) == 0;
      const bool eight = !a.y_f32 && a.N % 8 == 0 && ((uintptr_t)a.y & 15) == 0;
      if (!four && !eight) {
        const int64_t at = row0 * a.N + n0;
        const int rows = (int)min((int64_t)16, end - row0), cols = a.N - n0;
        if constexpr (S::KG > 1) {
          if (r < rows) {
#pragma unroll
            for (int i = 0; i < W; i++)
              if (W * q + i < cols) store_one(a, at + (r * a.N + W * q + i), acc[i >> 2][m][i & 3]);
          }
          continue;
        }
        // value by value, eight rows at a time, neighbouring lanes at neighbouring columns
#pragma unroll
        for (int h = 0; h < 2; h++) {
          if ((r >> 3) == h) {
#pragma unroll
            for (int t = 0; t < TN; t++)
              *reinterpret_cast<f32x4_t*>(out + 16 * (4 * TN * (r & 7) + TN * q + t)) = acc[t][m];
          }
          wave_fence();
#pragma unroll 1
          for (int b = 0; b < TN / 2; b++) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] = reinterpret_cast<const float*>(out)[64 * (4 * b + i) + lane];
#pragma unroll
            for (int i = 0; i < 4; i++) {
              const int e = 64 * (4 * b + i) + lane, rr = 8 * h + e / (16 * TN), col = e % (16 * TN);
              if (rr < rows && col < cols) store_one(a, at + (rr * a.N + col), v[i]);
            }
          }
          wave_fence();
        }
        continue;
      }
      if (row0 + r >= end) continue;
      const int64_t at = (row0 + r) * a.N + n;
#pragma unroll
      for (int c = 0; c < TN / 2; c++) {
        const int col = n + 8 * c;
        if (col >= a.N) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = acc[2 * c + (i >> 2)][m][i & 3];
        if (four) {
#pragma unroll
          for (int h = 0; h < 2; h++) {
            f32x4_t* p = reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(a.y) + at + 8 * c + 4 * h);
            if (col + 4 * h >= a.N) continue;
            f32x4_t o = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
            if (a.accumulate) o = *p + o;
            *p = o;
          }
        } else {
          u32x4_t* p = reinterpret_cast<u32x4_t*>(reinterpret_cast<uint16_t*>(a.y) + at + 8 * c);
          const u32x4_t old = a.accumulate ? *p : u32x4_t{0u, 0u, 0u, 0u};
          u32x4_t o;
#pragma unroll
          for (int i = 0; i < 4; i++)
            o[i] = pack_bf16x2(__uint_as_float(old[i] << 16) + v[2 * i],
                               __uint_as_float(old[i] & 0xffff0000u) + v[2 * i + 1]);
          *p = o;
        }
      }
    }
  }
}

// ------------------------------------------------------------- streaming kernel

constexpr int STREAM_WAVES = 8;

// 16 rows of x and 16 TN of W a workgroup: its wavefronts split K and load both
// straight into registers; their sums meet in LDS in a fixed order.
// v_mfma_scale_f32_16x16x128_f8f6f4: lane (row r = lane & 15, group q = lane
// >> 4) holds 32 values of K of its row; which ones is the same for both
// operands, and the scale is one for all of them.
template <int TN>
__global__ __launch_bounds__(64 * STREAM_WAVES) void fp8_stream_kernel(const LinearFp8Params a, int tiles_n) {
  constexpr int NW = STREAM_WAVES;
  __shared__ f32x4_t part[NW][TN][64];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = blockIdx.x / tiles_n, n0 = (blockIdx.x - g * tiles_n) * (16 * TN);
  Group o;
  if (!group_of(a, g, o)) return;
  const int kb = (a.K + 127) / 128;
  const int per = (kb + NW - 1) / NW, s_first = wave * per, s_end = min(s_first + per, kb);
  const uint8_t* w[TN];
#pragma unroll
  for (int t = 0; t < TN; t++) w[t] = o.w + (int64_t)min(a.N - 1, n0 + 16 * t + r) * a.K + 16 * q;
  const float* wsf = o.w_sf + (int64_t)(n0 >> 7) * kb;
  const int64_t xr = min(o.first + r, o.end - 1);
  const uint8_t *x = a.x + xr * a.K + 16 * q, *xsf = a.x_sf + xr * kb;
  f32x4_t acc[TN];
#pragma unroll
  for (int t = 0; t < TN; t++) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  for (int s = s_first; s < s_end; s++) {
    const bool in0 = 128 * s + 16 * q < a.K, in1 = 128 * s + 64 + 16 * q < a.K;
    u32x4_t w0[TN], w1[TN];
#pragma unroll
    for (int t = 0; t < TN; t++) {
      w0[t] = in0 ? ld16(w[t] + 128 * s) : zero;
      w1[t] = in1 ? ld16(w[t] + 128 * s + 64) : zero;
    }
    const u32x4_t x0 = in0 ? ld16(x + 128 * s) : zero, x1 = in1 ? ld16(x + 128 * s + 64) : zero;
    const float ws = wsf[s];
    const int xs = xsf[s];
    const i32x8_t c = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
#pragma unroll
    for (int t = 0; t < TN; t++) {
      const i32x8_t b = {(int)w0[t][0], (int)w0[t][1], (int)w0[t][2], (int)w0[t][3],
                         (int)w1[t][0], (int)w1[t][1], (int)w1[t][2], (int)w1[t][3]};
      const f32x4_t none = {0.0f, 0.0f, 0.0f, 0.0f};
      const f32x4_t p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(c, b, none, 0, 0, 0, xs, 0, 127);
#pragma unroll
      for (int i = 0; i < 4; i++) acc[t][i] = fmaf(p[i], ws, acc[t][i]);
    }
  }
#pragma unroll
  for (int t = 0; t < TN; t++) part[wave][t][lane] = acc[t];
  __syncthreads();
  // element i of lane (r, q): row 4 q + i, column r
  if (wave >= TN || n0 + 16 * wave + r >= a.N) return;
  f32x4_t v = part[0][wave][lane];
#pragma unroll
  for (int k = 1; k < NW; k++) v += part[k][wave][lane];
  const int n = n0 + 16 * wave + r;
  const float bias = a.bias ? a.bias[n] : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t row = o.first + 4 * q + i;
    if (row < o.end) store_one(a, row * a.N + n, v[i] + bias);
  }
}

// 32 columns a workgroup, which read x once for both halves, where that leaves one for
// each CU at least: 8 x 8192 x 8192 14.6 us against 16.9, 4 x 65536 x 2048 23 against 26,
// 32 experts of 555 rows, 4096 x 6144, 228 against 295, of 68 rows 145 against 142; 8 x
// 4096 x 6144, 128 workgroups, 10.1 against 7.3.
hipError_t launch_stream(const LinearFp8Params& a, hipStream_t s) {
  const int64_t groups = a.tile_expert ? a.tiles : (a.M + 15) / 16;
  const int tn = (a.N + 31) / 32;
  if (groups * tn >= 256) {
    fp8_stream_kernel<2><<<(unsigned)(groups * tn), 64 * STREAM_WAVES, 0, s>>>(a, tn);
  } else {
    const int t1 = (a.N + 15) / 16;
    fp8_stream_kernel<1><<<(unsigned)(groups * t1), 64 * STREAM_WAVES, 0, s>>>(a, t1);
  }
  return hipGetLastError();
}

// ------------------------------------------------------------- tiled kernel

typedef __attribute__((address_space(3))) void lds_void_t;

// Workgroup barrier: this wavefront's LDS accesses are done, and its loads but for
// the newest VM (written out: a release fence would wait for all of them).
template <int VM>
DEV void stage_barrier() {
  __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4));  // vmcnt(VM) lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int WM_, int WN_, int TM_, int TN_, int NBUF_, int KG_>
struct Tile {
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;  // wavefronts, 16 x 16 results of each
  static constexpr int NBUF = NBUF_;                            // stages in LDS
  static constexpr int KG = KG_;                                // groups of wavefronts that split K
  static constexpr int NT = 64 * WM * WN;                       // threads of a group
  static constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN;
  static constexpr int X_BYTES = BM * 128;
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int OUT = 16 * 16 * TN * 2;                  // a wavefront's way out: 16 rows
  static constexpr int RING = NBUF * STAGE;
  static constexpr int T_OFF = KG * RING;
  static constexpr int LDS = T_OFF + WM * WN * OUT;
  static constexpr int NX = BM * 8 / NT, NW = BN * 8 / NT;      // LDS-DMA loads a wavefront and stage
};

// One workgroup a tile at a time (a plan's tiles have BM rows), K in stages of 128 in a ring of buffers that
// LDS-DMA fills.  A wavefront computes 16 TM rows by 16 TN columns, W's rows the
// first operand: a lane then has 4 TN consecutive columns of one row of y, if
// row 4 a + b of W's tile t is column 4 TN a + 4 t + b.  The rows' fragments
// stay in registers over a stage, W's pass through four of them; the last two of
// a stage are multiplied row tile by row tile, so that the next stage's rows can
// be read behind them, and the barrier between two stages has multiplications
// on both sides.
template <typename S, bool WIDE>
__global__ __launch_bounds__(S::NT * S::KG, 2) void fp8_tile_kernel(const LinearFp8Params a, int tiles_n) {
  constexpr int TM = S::TM, TN = S::TN, BM = S::BM, BN = S::BN, NX = S::NX, NW = S::NW, NBUF = S::NBUF, KG = S::KG;
  static_assert(TN % 4 == 0 && NX >= 1 && NW >= 1, "four buffers of W; whole loads");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_all[];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % (S::WM * S::WN);
  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / S::NT);
  uint8_t* smem = smem_all + kg * S::RING;
  const int wn = wave % S::WN, wm = wave / S::WN;
  // stages of a K group (some past the end of K, whose values count as 0)
  const int kb = (a.K + 127) / 128, KT = max((kb + KG - 1) / KG, NBUF), first_s = kg * KT;

  // tiles of this workgroup: XCD b & 7 takes a contiguous run of them, its
  // workgroups take them in turn; 8 rows of tiles high, so that what an XCD
  // works on at a time shares its rows in the L2
  const int tiles_m = a.tile_expert ? ld_uniform(a.num_tiles) : (int)((a.M + BM - 1) / BM);
  const int64_t tiles = (int64_t)tiles_m * tiles_n, per = (tiles + 7) / 8;
  const int step = gridDim.x >> 3;
  const int64_t first = (blockIdx.x & 7) * per, last = min(first + per, tiles);
  int64_t t = first + (blockIdx.x >> 3);
  if (t >= last) return;

  struct At {
    int64_t m0, end;
    int n0;
    const uint8_t* w;
    const float* w_sf;
  };
  auto tile_at = [&](int64_t t) {
    constexpr int GM = 8;
    const int group = (int)(t / (GM * tiles_n)), in = (int)(t - (int64_t)group * GM * tiles_n);
    const int rows = min(GM, tiles_m - group * GM), tm = group * GM + in % rows;
    At o;
    o.n0 = in / rows * BN;
    o.m0 = (int64_t)tm * BM;
    if (!a.tile_expert) {
      o.end = min(a.M, o.m0 + BM);
      o.w = a.w;
      o.w_sf = a.w_sf;
    } else {
      const int e = ld_uniform(a.tile_expert + tm);
      o.end = ld_uniform(a.tile_limit + tm);
      o.w = a.w + (int64_t)e * a.N * a.K;
      o.w_sf = a.w_sf + (int64_t)e * ((a.N + 127) / 128) * kb;
    }
    return o;
  };

  // what the loads of the moment read: buffers that end with the tile's last row
  // (rows past it read as 0), this lane's place in them (row lane / 8 of eight, a
  // chunk of 16 bytes swizzled by row / 2, whose bit 2 is the load's parity), and
  // the scales' rows (past the last: that one; such products are not stored)
  __amdgpu_buffer_rsrc_t xb, wb;
  const uint8_t* xsf;
  const float* wsf;
  int last_m;
  const int chunk = 16 * ((lane & 7) ^ (lane >> 4));
  const uint32_t place_x = (uint32_t)(8 * NX * wave + (lane >> 3)) * (uint32_t)a.K;
  // row of W that lane / 8 loads: a load's eight rows of LDS, 8 i + 0 .. 7, are
  // rows 4 c .. 4 c + 3 of W for two c
  const uint32_t place_w = (uint32_t)((lane >> 5) * 4 * TN + ((lane >> 3) & 3)) * (uint32_t)a.K;
  auto aim = [&](const At& o) {
    last_m = max(0, (int)(o.end - o.m0) - 1);
    xb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.x + o.m0 * a.K), 0, (last_m + 1) * a.K, 0x00020000);
    wb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(o.w + (int64_t)o.n0 * a.K), 0,
                                           min(BN, a.N - o.n0) * a.K, 0x00020000);
    xsf = a.x_sf + o.m0 * kb;
    wsf = o.w_sf + (int64_t)(min(o.n0 + 16 * TN * wn, a.N - 1) >> 7) * kb;
  };
  // (a chunk past the end of K: the row's first one)
  auto issue = [&](int s, uint8_t* st) {
    uint32_t k[2];  // of loads of even and odd number
#pragma unroll
    for (int v = 0; v < 2; v++) {
      k[v] = (uint32_t)(128 * (first_s + s) + (chunk ^ (64 * v)));
      k[v] = k[v] < (uint32_t)a.K ? k[v] : 0u;
    }
    const uint32_t kx[2] = {NX % 2 && (wave & 1) ? k[1] : k[0], NX % 2 && (wave & 1) ? k[0] : k[1]};
#pragma unroll
    for (int i = 0; i < NX; i++)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xb, (lds_void_t*)(st + 1024 * (NX * wave + i)), 16,
                                               place_x + kx[i & 1] + (uint32_t)(8 * i * a.K), 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NW; i++) {
      const int j = 8 * (NW * wave + i), in = j % (16 * TN);  // the load's first row of LDS
      const int n = j - in + ((in >> 2) & 3) * (4 * TN) + 4 * (in >> 4);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wb, (lds_void_t*)(st + S::X_BYTES + 1024 * (NW * wave + i)), 16,
                                               place_w + k[i & 1] + (uint32_t)(n * a.K), 0, 0, 0);
    }
  };

  const int swizzle = (r >> 1) & 7;
  const int at0 = 128 * r + 16 * (q ^ swizzle), at1 = 128 * r + 16 * ((q + 4) ^ swizzle);
  struct Frag {
    u32x4_t lo, hi;
  };
  auto read_x = [&](const uint8_t* st, int m) {
    const uint8_t* p = st + 2048 * (TM * wm + m);
    return Frag{ld16(p + at0), ld16(p + at1)};
  };
  auto read_w = [&](const uint8_t* st, int t) {
    const uint8_t* p = st + S::X_BYTES + 2048 * (TN * wn + t);
    return Frag{ld16(p + at0), ld16(p + at1)};
  };
  auto mul = [&](const Frag& w, const Frag& x, int xs) {
    const i32x8_t c = {(int)w.lo[0], (int)w.lo[1], (int)w.lo[2], (int)w.lo[3],
                       (int)w.hi[0], (int)w.hi[1], (int)w.hi[2], (int)w.hi[3]};
    const i32x8_t b = {(int)x.lo[0], (int)x.lo[1], (int)x.lo[2], (int)x.lo[3],
                       (int)x.hi[0], (int)x.hi[1], (int)x.hi[2], (int)x.hi[3]};
    const f32x4_t none = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(c, b, none, 0, 0, 0, 127, 0, xs);
  };

  Frag x[TM], w[4];
  f32x4_t acc[TN][TM], p[TM];
  uint32_t word[TM], later[TM];  // scale bytes of the stages from this one on, and of the next four
  float ws;
  auto load_scales = [&](int g) {
    if (kb >= 4) {  // four bytes; a word that reaches past the row's end: its last four
      const int at = min(first_s + 4 * g, kb - 4);
#pragma unroll
      for (int m = 0; m < TM; m++)
        __builtin_memcpy(&later[m], xsf + min(16 * (TM * wm + m) + r, last_m) * kb + at, 4);
    } else {  // the bytes from the K group's first block on (past the last one: that one, of values that count as 0)
      const int b = KG == 1 ? 0 : min(first_s, kb - 1);
#pragma unroll
      for (int m = 0; m < TM; m++) {
        const uint8_t* row = xsf + min(16 * (TM * wm + m) + r, last_m) * kb;
        later[m] = (uint32_t)row[b] | (uint32_t)row[min(b + 1, kb - 1)] << 8 | (uint32_t)row[kb - 1] << 16;
      }
    }
  };
  auto add = [&](int t, int m, const f32x4_t& v, float s) {
#pragma unroll
    for (int i = 0; i < 4; i++) acc[t][m][i] = fmaf(v[i], s, acc[t][m][i]);
  };
  auto pin_all = [&]() {
#pragma unroll
    for (int i = 0; i < TN; i++)
#pragma unroll
      for (int m = 0; m < TM; m++) asm volatile("" : "+v"(acc[i][m]));
  };
  int buf = 0;
  // One stage; its loads fetch stage `ahead` of what is aimed at (K groups have
  // one tile and fetch nothing in its last stages); `wsn`: W's scale of the next
  // stage.
  auto stage = [&](int ahead, const float* wsn, auto tail_) {
    constexpr bool LOAD = KG == 1 || !decltype(tail_)::value;
    uint8_t* st = smem + buf * S::STAGE;
    buf = buf == NBUF - 1 ? 0 : buf + 1;
    const uint8_t* sn = smem + buf * S::STAGE;
#pragma unroll
    for (int i = 0; i < TN - 2; i++) {
      w[(i + 2) & 3] = read_w(st, i + 2);
#pragma unroll
      for (int m = 0; m < TM; m++) {
        if (i > 0) add(i - 1, m, p[m], ws);
        p[m] = mul(w[i & 3], x[m], (int)word[m]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // every fragment of the stage is in registers, the next stage has landed
    stage_barrier<LOAD ? (NBUF - 2) * (NX + NW) : 0>();
    if constexpr (LOAD) issue(ahead, st);
    const float wl = ws;
    ws = ld_uniform(wsn);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < TM; m++) {
      const f32x4_t u = mul(w[(TN - 2) & 3], x[m], (int)word[m]), v = mul(w[(TN - 1) & 3], x[m], (int)word[m]);
      x[m] = read_x(sn, m);
      if (m < 2) w[m] = read_w(sn, m);
      add(TN - 3, m, p[m], wl);
      add(TN - 2, m, u, wl);
      add(TN - 1, m, v, wl);
      word[m] >>= 8;
      __builtin_amdgcn_sched_barrier(0);
    }
    pin_all();
  };
  // the scales of the four stages from s on, and the loads of those after them
  auto next_scales = [&](int s) {
    if ((s & 3) == 0) {
      const int past = max(0, first_s + s + 4 - kb), shift = kb >= 4 ? 8 * min(past, 3) : 0;
#pragma unroll
      for (int m = 0; m < TM; m++) word[m] = later[m] >> shift;
      if (s + 4 < KT) load_scales((s >> 2) + 1);
    }
  };
  auto mask = [&](int s) {  // values past the end of K
    const int k = 128 * (first_s + s);
    if (k + 128 > a.K) {
      const bool in0 = k + 16 * q < a.K, in1 = k + 64 + 16 * q < a.K;
#pragma unroll
      for (int m = 0; m < TM; m++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          x[m].lo[i] = in0 ? x[m].lo[i] : 0u;
          x[m].hi[i] = in1 ? x[m].hi[i] : 0u;
        }
    }
  };

  At o = tile_at(t);
  aim(o);
  load_scales(0);
#pragma unroll
  for (int i = 0; i < NBUF; i++) issue(i, smem + i * S::STAGE);
  ws = ld_uniform(wsf + min(first_s, kb - 1));
  stage_barrier<(NBUF - 1) * (NX + NW)>();
#pragma unroll
  for (int m = 0; m < TM; m++) x[m] = read_x(smem, m);
  w[0] = read_w(smem, 0);
  w[1] = read_w(smem, 1);

#pragma unroll 1
  for (;;) {
#pragma unroll
    for (int i = 0; i < TN; i++)
#pragma unroll
      for (int m = 0; m < TM; m++) acc[i][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (a.bias && kg == 0) {  // the sums start with it
#pragma unroll
      for (int i = 0; i < TN; i++) {
        f32x4_t b;
#pragma unroll
        for (int c = 0; c < 4; c++) b[c] = a.bias[min(o.n0 + 16 * TN * wn + 4 * TN * q + 4 * i + c, a.N - 1)];
#pragma unroll
        for (int m = 0; m < TM; m++) acc[i][m] = b;
      }
    }
    const int64_t tn = t + step;
    const bool more = tn < last;
    const At next = more ? tile_at(tn) : o;
    int s = 0;
#pragma unroll 1
    for (; s < KT - NBUF; s++) {
      next_scales(s);
      if constexpr (KG > 1) mask(s);
      stage(s + NBUF, wsf + min(first_s + s + 1, kb - 1), std::false_type());
    }
    // the last ones fetch the first ones of the next tile (without one, of this
    // tile again, unread)
    const float* of_this = wsf;
#pragma unroll
    for (int i = 0; i < NBUF; i++, s++) {
      next_scales(s);
      mask(s);
      if (KG == 1 && i == 0) aim(next);
      if (KG == 1 && i == NBUF - 1) load_scales(0);
      stage(i, i == NBUF - 1 ? wsf : of_this + min(first_s + s + 1, kb - 1), std::true_type());
    }
    // the K groups' sums: the upper half hands its own to the lower one, until the
    // first group has all of them
#pragma unroll
    for (int half = KG / 2; half >= 1; half /= 2) {
      f32x4_t* to = reinterpret_cast<f32x4_t*>(smem_all);
      const int at = ((kg & (half - 1)) * S::WM * S::WN + wave) * TN * TM * 64 + lane;
      __syncthreads();  // what was read or handed over before
      if (kg >= half && kg < 2 * half) {
#pragma unroll
        for (int i = 0; i < TN * TM; i++) to[at + 64 * i] = acc[i / TM][i % TM];
      }
      __syncthreads();
      if (kg < half) {
#pragma unroll
        for (int i = 0; i < TN * TM; i++) acc[i / TM][i % TM] += to[at + 64 * i];
      }
    }
    if (kg > 0) return;
    store_tile<S, WIDE>(a, acc, o.m0 + 16 * TM * wm, o.end, o.n0 + 16 * TN * wn, smem_all + S::T_OFF + S::OUT * wave, lane);
    if (!more) break;
    t = tn;
    o = next;
  }
  __builtin_amdgcn_s_waitcnt(0x0070);  // no LDS-DMA load may be in flight when the workgroup ends
}

bool wide_rows(const LinearFp8Params& a) {
  return !a.y_f32 && !a.accumulate && a.N % 8 == 0 && ((uintptr_t)a.y & 15) == 0;
}

template <typename S, bool WIDE>
hipError_t launch_tile_as(const LinearFp8Params& a, hipStream_t s) {
  constexpr int PER_CU = 160 * 1024 / S::LDS;
  static_assert(PER_CU >= 1, "two stages exceed the CU's LDS");
  int cus = 0;
  const hipError_t err = allow_lds<fp8_tile_kernel<S, WIDE>>(S::LDS, &cus);
  if (err != hipSuccess) return err;
  const int tn = (a.N + S::BN - 1) / S::BN;
  const int64_t tm = a.tile_expert ? (int64_t)a.tiles : (a.M + S::BM - 1) / S::BM;
  const int64_t most = (int64_t)(cus >= 8 ? cus / 8 * 8 : 8) * PER_CU, tiles = (tm * tn + 7) / 8 * 8;
  const int64_t grid = S::KG == 1 && tiles > most ? most : tiles;  // (K groups: a tile a workgroup)
  fp8_tile_kernel<S, WIDE><<<(unsigned)grid, S::NT * S::KG, S::LDS, s>>>(a, tn);
  return hipGetLastError();
}
template <typename S>
hipError_t launch_tile(const LinearFp8Params& a, hipStream_t s) {
  return wide_rows(a) ? launch_tile_as<S, true>(a, s) : launch_tile_as<S, false>(a, s);
}

// rows x columns of a tile; wavefronts of 16 TM x 16 TN; stages; K groups
using Big = Tile<4, 2, 4, 8, 2, 1>;     // 256 x 256, eight wavefronts, one workgroup a CU
using Middle = Tile<2, 2, 4, 4, 2, 1>;  // 128 x 128, four, two workgroups a CU
using Small = Tile<2, 2, 2, 4, 3, 1>;   // 64 x 128, four, two
using Low = Tile<1, 4, 2, 4, 2, 1>;     // 32 x 256, four, two
using Split2 = Tile<2, 2, 2, 4, 3, 2>;  // 64 x 128, K in two
using Split4 = Tile<2, 1, 2, 4, 2, 4>;  // 64 x 64, K in four
using Split4Low = Tile<1, 1, 2, 4, 2, 4>;  // 32 x 64, K in four

}  // namespace

hipError_t launch_linear_fp8(const LinearFp8Params& a, hipStream_t s) {
  constexpr int64_t CUS = 256;
  if (a.tile_expert) {
    // a workgroup for each of the plan's tiles (32 experts of 4096 x 6144, in tiles of 32
    // and 64 against streaming the same plan in pieces of 16: 1000 rows 206 us, 396; 2000
    // rows 208, 621)
    switch (a.tile) {
      case 16: return launch_stream(a, s);
      case 32: return launch_tile_as<Low, true>(a, s);  // (a plan's rows always leave in whole lines)
      case 64: return launch_tile<Small>(a, s);
      case 128: return launch_tile<Middle>(a, s);
      default: return launch_tile<Big>(a, s);  // 256
    }
  }
  auto tiles = [&](int m, int n) { return ((a.M + m - 1) / m) * ((a.N + n - 1) / n); };
  // The streaming kernel while its 16 x 16 tiles have little to do together, or are few:
  // it waits for memory once, the others for each stage (128 x 724 x 1024: 4.7 us against
  // 6.4; 32 x 2048 x 2048 4.9, 5.6; 128 x 256 x 8192, 128 tiles, 11.4, 13.2; 256 x 1024 x
  // 1024 5.7, 4.7; 64 x 2048 x 2048 5.9, 5.7; 32 x 4096 x 4096 9.3, 8.2).
  const int64_t pieces = tiles(16, 16);
  if (a.M <= 16 || pieces * ((a.K + 127) / 128) <= 4096 || pieces <= CUS / 2) return launch_stream(a, s);
  // A wavefront alone on a SIMD is bound by its own instructions, about 1000 cycles
  // a stage of 32 x 64 results.  While all tiles have a CU each, K is split over
  // more wavefronts: 64 x 4096 x 6144 11.3 us against 24.9 in 64 x 128 tiles, 128 x 4096
  // x 4096 8.3 against 19.3, 256 x 4096 x 4096 13.1 against 19.7, 512 x 4096 x 4096
  // 16.1 against 22.1.
  if (tiles(32, 64) <= CUS) return launch_tile<Split4Low>(a, s);
  if (tiles(64, 64) <= CUS) return launch_tile<Split4>(a, s);
  if (tiles(64, 128) <= CUS) return launch_tile<Split2>(a, s);
  // 256 x 256 tiles where they fill whole rounds of the CUs, three quarters at
  // least (8000 x 2000 x 2000, one full round: 53.6 us against 49.5 in 128 x 128 tiles;
  // 4096 x 4096 x 4096: 68 against 99)
  const int64_t big = tiles(256, 256), rounds = (big + CUS - 1) / CUS;
  if (4 * big >= 3 * CUS * rounds && a.K >= 1024) return launch_tile<Big>(a, s);
  // (4096 x 724 x 1024, 192 tiles of 128 x 128: 19.2 us in 64 x 128, 20.7; 2048 x 4096 x
  // 2048, 512 of them: 29.9, 22.5)
  if (tiles(128, 128) <= CUS) return launch_tile<Small>(a, s);
  return launch_tile<Middle>(a, s);
}

}  // namespace moe
