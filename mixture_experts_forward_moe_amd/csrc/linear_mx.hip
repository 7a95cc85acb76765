// linear_mx.hip -- y = alpha * x W^T + bias for MX operands without a routing
// plan: x E4M3 or E2M1, W E2M1, E8M0 scales per 32 values along K.
//
// The scaled MFMA takes both operands as they are stored, with their E8M0
// bytes, so nothing is decoded and no sum needs a correction afterwards.  What
// such an instruction keeps: E2M1 products add exactly to their fp32 sum; with
// an E4M3 operand each group of 8 consecutive k keeps the bits down to 2^-13
// of its largest product's power of two (measured), and sums are fp32.
//
// Rates from registers, on random data: 6.6 PFLOP/s E2M1 x E2M1, 4.1 - 4.6
// E4M3 x E2M1 (8.8 and 4.9 on zeros: the clock falls with the operands'
// toggling).  L2 into LDS: 15 TB/s in rows of 64 bytes, 27 in rows of 128
// that the workgroups of an XCD share.
//
// Three kernels, in order of size: a streaming one (a row of 16 x 16 tiles: it
// is bound by latency and by the bytes of W), a tiled one (one tile a
// workgroup: it is bound by its stages' trips from L2 to LDS, of which one or two
// are under way at a time) and a persistent one (whole
// rounds of large tiles: it is bound by the matrix cores, whose operands'
// reads and loads share the LDS).  Figures stand at launch().
#include <atomic>
#include <type_traits>

#include "device_common.h"
#include "internal.h"

namespace moe {

namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void_t;

DEV u32x4_t ld16(const uint8_t* p) { return *reinterpret_cast<const u32x4_t*>(p); }
// 16 bytes at any alignment
DEV u32x4_t ld16u(const uint8_t* p) {
  u32x4_t v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// s_waitcnt immediates (gfx9 encoding: vmcnt bits 3:0 and 15:14, expcnt 6:4,
// lgkmcnt 11:8); counters not named are not waited for
constexpr int waitcnt_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }

// workgroup barrier over LDS that waits for this wave's LDS accesses only (a
// release fence would also wait for every LDS-DMA load in flight)
DEV void ring_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

DEV void dma16(const uint8_t* g, uint8_t* base) {
  __builtin_amdgcn_global_load_lds(g, (lds_void_t*)base, 16, 0, 0);
}

// Allows a kernel more than the default dynamic LDS, once per device, and
// gives the device's number of compute units.  Calls of several threads may
// come here at once: one word says that it has been done, and is the number.
template <auto KERN>
hipError_t allow_lds(int bytes, int* cus) {
  static std::atomic<int> count[64] = {};  // 0: not yet
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  const bool known = dev >= 0 && dev < 64;
  *cus = known ? count[dev].load(std::memory_order_acquire) : 0;
  if (*cus > 0) return hipSuccess;
  err = hipFuncSetAttribute((const void*)KERN, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err != hipSuccess) return err;
  err = hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (err == hipSuccess && known) count[dev].store(*cus, std::memory_order_release);
  return err;
}

// ------------------------------------------------------------- tiled kernel

// The column (0..31) that MFMA row i of a weight tile stands for: lane half
// h, element j of the 32x32 result holds row 8 (j / 4) + 4 h + j % 4, which
// is column 16 h + j: a lane has 16 consecutive columns of one y row.
DEV int tile_col(int i) { return 16 * ((i >> 2) & 1) + 4 * (i >> 3) + (i & 3); }

// Chunks (16 bytes) of a row in a stage: C = 4, 8 or 16 of them, 1024 / (16 C)
// rows a LDS-DMA load.  A load fills fixed LDS positions (lane i 16 i past the
// base), so the swizzle that spreads the fragment reads over the banks is
// applied to what each lane loads: rows of 4 chunks are swizzled by row / 4, of
// 8 by row / 2, of 16 by the row.  Of that number the low two bits are the
// lane's (lane / 16), the others the load's own.
template <int C>
struct Chunks {
  static constexpr int ROWS = 64 / C;
  static constexpr int KINDS = C / 4;  // kinds of loads: load i is of kind i % KINDS
  static DEV int row(int load, int lane) { return ROWS * load + lane / C; }
  // byte in the row's part of a stage that a lane loads, in loads of kind v
  static DEV int source(int v, int lane) { return 16 * (((lane & (C - 1)) ^ ((lane >> 4) & 3)) ^ (4 * v)); }
  // byte of logical chunk c in row r of a stage
  static DEV int at(int r, int c) {
    return 16 * C * r + 16 * (c ^ (C == 4 ? (r >> 2) & 3 : C == 8 ? (r >> 1) & 7 : r & 15));
  }
};

template <int XE, int TM, int TN, int KS, int NBUF, int KG>
struct Shape {
  static constexpr int BM = 64 * TM, BN = 64 * TN;  // 2 x 2 wavefronts of 32 TM x 32 TN, KG times
  static constexpr int XB = XE == 1 ? KS / 2 : KS;  // bytes of a row in a stage of KS
  static constexpr int WB = KS / 2;
  static constexpr int NX = BM * XB / 4096, NW = BN * WB / 4096;  // LDS-DMA loads a wavefront and stage
  static constexpr int STAGE = BM * XB + BN * WB;
  static constexpr int GS = 512 / KS;               // stages of a scale record (16 E8M0 bytes)
  static constexpr int SC = (BM + BN) * 16;         // the records: x rows, then weight rows
  static constexpr int SC_OFF = NBUF * STAGE;
  static constexpr int RING = SC_OFF + SC;          // a K group's part
  static constexpr int JOIN = KG > 1 ? KG / 2 * BM * BN * 4 : 0;
  static constexpr int LDS = KG * RING > JOIN ? KG * RING : JOIN;
};

// The 16 E8M0 bytes from byte `at` of a row of nb >= 16 bytes; 0 past its end
// (2^-127 twice: such products vanish).  A record that reaches past the end
// is read from the row's last 16 bytes and shifted down, without a branch, so
// that no byte outside the row is touched.
DEV const uint8_t* scale_source(const uint8_t* row, int at, int nb) { return row + min(at, nb - 16); }
DEV u32x4_t scale_shift(const u32x4_t& v, int at, int nb) {
  const int over = max(0, at + 16 - nb);
  const int w = over >> 2, b = 8 * (over & 3);
  u32x4_t o;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int j = i; j < 4; j++) {
      lo = j == i + w ? v[j] : lo;
      hi = j == i + w + 1 ? v[j] : hi;
    }
    o[i] = (uint32_t)((((uint64_t)hi << 32) | lo) >> b);
  }
  return o;
}
// the same of a shorter row
DEV u32x4_t scale_short(const uint8_t* row, int at, int nb) {
  u32x4_t o = {0u, 0u, 0u, 0u};
  for (int i = 0; i < nb - at; i++) {
    const uint32_t c = row[at + i];
#pragma unroll
    for (int j = 0; j < 4; j++) o[j] |= j == i >> 2 ? c << (8 * (i & 3)) : 0u;
  }
  return o;
}

// Accumulators are complete here: keeps MFMAs from being sunk into a later
// block, with their operands live up to it.
template <int N>
DEV void pin(f32x16_t& v) {
  if constexpr (N > 8) asm volatile("" : "+a"(v));
  else asm volatile("" : "+v"(v));
}

template <int XE>
struct XFrag {
  u32x4_t p[XE == 1 ? 1 : 2];
};

template <int XE, int U>
DEV void mfma_one(f32x16_t& acc, const u32x4_t& w, const XFrag<XE>& x, int ws, int xs) {
  const i32x8_t a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  i32x8_t b;
  if constexpr (XE == 1) {
    b = i32x8_t{(int)x.p[0][0], (int)x.p[0][1], (int)x.p[0][2], (int)x.p[0][3], 0, 0, 0, 0};
  } else {
    b = i32x8_t{(int)x.p[0][0], (int)x.p[0][1], (int)x.p[0][2], (int)x.p[0][3],
                (int)x.p[1][0], (int)x.p[1][1], (int)x.p[1][2], (int)x.p[1][3]};
  }
  // byte 2 U of the (half-shifted) scale words: block 2 U + h of the stage
  acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 4, XE == 1 ? 4 : 0, 2 * U, ws, 2 * U, xs);
}

// alpha * sum + bias, one step with one rounding: written out, so that every
// way out makes the same one
DEV float scaled(float sum, float alpha, float bias) { return fmaf(sum, alpha, bias); }

// y[m, n .. n + 15] of a lane: fp32, or onto what y holds
DEV void store16(const LinearParams& a, const f32x16_t& acc, int64_t m, int n, float alpha) {
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; j++) v[j] = scaled(acc[j], alpha, a.bias && n + j < a.N ? a.bias[n + j] : 0.0f);
  const int64_t at = m * a.N + n;
  if (a.y_f32) {
    float* y = reinterpret_cast<float*>(a.y) + at;
    if (n + 16 <= a.N && a.N % 4 == 0 && ((uintptr_t)a.y & 15) == 0) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        f32x4_t o = {v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
        f32x4_t* p = reinterpret_cast<f32x4_t*>(y) + j;
        if (a.accumulate) o = *p + o;
        *p = o;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; j++)
        if (n + j < a.N) y[j] = a.accumulate ? y[j] + v[j] : v[j];
    }
  } else {
    uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + at;
    if (n + 16 <= a.N && a.N % 8 == 0 && ((uintptr_t)a.y & 15) == 0) {
#pragma unroll
      for (int j = 0; j < 2; j++) {
        u32x4_t* p = reinterpret_cast<u32x4_t*>(y) + j;
        const u32x4_t old = *p;
        u32x4_t o;
#pragma unroll
        for (int i = 0; i < 4; i++)
          o[i] = pack_bf16x2(__uint_as_float(old[i] << 16) + v[8 * j + 2 * i],
                             __uint_as_float(old[i] & 0xffff0000u) + v[8 * j + 2 * i + 1]);
        *p = o;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; j++)
        if (n + j < a.N) y[j] = f32_to_bf16(bf16_to_f32(y[j]) + v[j]);
    }
  }
}

// A wavefront's 32 TM x 32 TN results, first row m0, first column n0.  bf16 y
// that is overwritten goes through OUT bytes of the wavefront's own LDS, OUT
// / 64 rows of a 32 x 32 tile at a time (chunks swizzled by row / 4), and
// leaves 64 bytes a row, neighbours in neighbouring lanes, in the widest
// stores that the rows of y are aligned to.  WIDE (wide_rows): 16 bytes; the
// other ways out are left out of that kernel, where they would cost the main
// loop registers.
template <bool WIDE, int TM, int TN, int OUT>
DEV void store_tiles(const LinearParams& a, const f32x16_t (&acc)[TN][TM], int64_t m0, int n0, uint8_t* out, int lane) {
  const int r = lane & 31, h = lane >> 5;
  const float alpha = a.alpha ? *a.alpha : 1.0f;
  if (!WIDE && (a.y_f32 || a.accumulate)) {
#pragma unroll
    for (int n = 0; n < TN; n++) {
      const int col = n0 + 32 * n + 16 * h;
#pragma unroll
      for (int m = 0; m < TM; m++) {
        const int64_t row = m0 + r + 32 * m;
        if (row < a.M && col < a.N) store16(a, acc[n][m], row, col, alpha);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    return;
  }
  // columns of a piece that the rows of y are aligned to, of less than 16 bytes
  const int align = (int)(((uint32_t)a.N * 2u) | (uint32_t)(uintptr_t)a.y);
  const int width = (align & 7) == 0 ? 4 : (align & 3) == 0 ? 2 : 1;
  constexpr int ROWS = OUT / 64;
  uint16_t* y = reinterpret_cast<uint16_t*>(a.y);
#pragma unroll
  for (int n = 0; n < TN; n++) {
    const int c0 = n0 + 32 * n;
    float bias[16];
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < 16; i++) bias[i] = a.bias[min(c0 + 16 * h + i, a.N - 1)];
    }
#pragma unroll
    for (int m = 0; m < TM; m++) {
      u32x4_t o[2];
#pragma unroll
      for (int c = 0; c < 2; c++) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int k = 8 * c + 2 * i;
          float lo = acc[n][m][k] * alpha, hi = acc[n][m][k + 1] * alpha;
          if (a.bias) {
            lo = scaled(acc[n][m][k], alpha, bias[k]);
            hi = scaled(acc[n][m][k + 1], alpha, bias[k + 1]);
          }
          o[c][i] = pack_bf16x2(lo, hi);
        }
      }
#pragma unroll
      for (int part = 0; part < 32 / ROWS; part++) {
        if (r / ROWS == part) {
#pragma unroll
          for (int c = 0; c < 2; c++)
            *reinterpret_cast<u32x4_t*>(out + 64 * (r % ROWS) + 16 * ((2 * h + c) ^ ((r >> 2) & 3))) = o[c];
        }
        wave_fence();  // the rows are read by other lanes
        const int64_t row0 = m0 + 32 * m + ROWS * part;
        auto rows_of = [&](auto w_) {  // in pieces of W columns, 32 / W lanes a row
          constexpr int W = decltype(w_)::value, LR = 32 / W;
          struct Piece {
            uint16_t v[W];
          } __attribute__((aligned(2 * W)));
          const int c = W * (lane % LR), col = c0 + c;
#pragma unroll
          for (int i = 0; i < ROWS / (64 / LR); i++) {
            const int rr = 64 / LR * i + lane / LR;
            const Piece v =
                *reinterpret_cast<const Piece*>(out + 64 * rr + 16 * ((c >> 3) ^ ((rr >> 2) & 3)) + 2 * (c & 7));
            if (row0 + rr < a.M && col < a.N) *reinterpret_cast<Piece*>(y + (row0 + rr) * a.N + col) = v;
          }
        };
        if constexpr (WIDE) rows_of(std::integral_constant<int, 8>{});
        else if (width == 4) rows_of(std::integral_constant<int, 4>{});
        else if (width == 2) rows_of(std::integral_constant<int, 2>{});
        else rows_of(std::integral_constant<int, 1>{});
        wave_fence();  // and written again once they have been
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// One tile a workgroup: 2 x 2 wavefronts of 32 TM x 32 TN results, K in stages of
// KS in a ring of NBUF that LDS-DMA fills, scales in records of 16 bytes (512
// K) beside it.  The last 64-K step of a stage multiplies while the first
// fragments of the next one are read, so a barrier a stage is all that the
// ring costs.  KG groups of four wavefronts split K where there are few tiles,
// each with a ring of its own; their sums meet in LDS in a fixed order.  Bound
// by the stages' trips: with two buffers one stage is on its way while the other
// multiplies.  512 x 4096 x 4096 E4M3 in 14.1 us (1.22 PFLOP/s): eight steps of
// 64 KiB a CU at 1.27 us (the slope up to K = 16384), 13 TB/s of the 27 above,
// where the matrix cores need 0.5, and 4 us of start, join and way out.  E2M1 in
// 11.8 us (1.46): 16 steps of 32 KiB at 0.57, 15 TB/s, and 2.7 us.
template <int XE, bool WIDE, int TM, int TN, int KS, int NBUF, int KG, int PER_CU>
__global__ __launch_bounds__(256 * KG, PER_CU * KG) void linear_tile_kernel(const LinearParams a, int tiles_m,
                                                                            int tiles_n) {
  using S = Shape<XE, TM, TN, KS, NBUF, KG>;
  using X = Chunks<S::XB / 16>;
  using W = Chunks<S::WB / 16>;
  constexpr int XB = S::XB, WB = S::WB, NX = S::NX, NW = S::NW, BM = S::BM, BN = S::BN, GS = S::GS;
  constexpr int ND = NX + NW;
  constexpr int NQ = TN * TM;                          // MFMAs of 64 K
  constexpr int NF = TN + TM * (XE == 1 ? 1 : 2);      // their fragment reads
  constexpr int QS = KS / 64;                          // 64-K steps of a stage
  static_assert(NX % X::KINDS == 0 && NW % W::KINDS == 0, "a load's kind goes by its number");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_all[];
  const int lane = threadIdx.x & 63, tid = threadIdx.x & 255;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3;
  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  uint8_t* smem = smem_all + kg * S::RING;
  const int wn = wave & 1, wm = wave >> 1;
  const int r = lane & 31, h = lane >> 5;
  const int nb = a.K / 32;
  // stages of each K group (past the end of K: scales 0)
  const int KT = ((a.K + KS - 1) / KS + KG - 1) / KG, k_first = kg * KT;
  const int xrb = XE == 1 ? a.K / 2 : a.K, wrb = a.K / 2;

  // tile of this workgroup: the XCDs (workgroups are dealt to them round
  // robin) take contiguous runs of tiles, GM tile rows high, so that an XCD's
  // L2 holds what its concurrent workgroups share
  int64_t m0;
  int n0;
  {
    const int tiles = tiles_m * tiles_n;
    const int per = (tiles + 7) / 8;
    int t = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (t >= tiles || (int)(blockIdx.x >> 3) >= per) return;
    constexpr int GM = 8;
    const int group = t / (GM * tiles_n), in = t % (GM * tiles_n);
    const int rows = min(GM, tiles_m - group * GM);
    m0 = (int64_t)(group * GM + in % rows) * BM;
    n0 = (in / rows) * BN;
  }

  // source rows of this lane's LDS-DMA loads (rows past the end: the last
  // row, whose products are not stored)
  const uint8_t* xb = a.x + m0 * xrb;
  const uint8_t* wb = a.w + (int64_t)n0 * wrb;
  const int last_m = (int)min((int64_t)BM, a.M - m0) - 1, last_n = min(BN, a.N - n0) - 1;
  uint32_t xo[NX], wo[NW];
#pragma unroll
  for (int j = 0; j < NX; j++) xo[j] = (uint32_t)min(X::row(NX * wave + j, lane), last_m) * (uint32_t)xrb;
#pragma unroll
  for (int j = 0; j < NW; j++) {
    const int b = W::row(NW * wave + j, lane);
    wo[j] = (uint32_t)min((b & ~31) + tile_col(b & 31), last_n) * (uint32_t)wrb;
  }
  // the loads of stage s into st; a chunk past the end of its row: the row's
  // first one (its scale is 0)
  auto issue = [&](int s_, uint8_t* st) {
    const int s = k_first + s_;
    uint32_t ox[X::KINDS], ow[W::KINDS];
#pragma unroll
    for (int v = 0; v < X::KINDS; v++) {
      const uint32_t k = (uint32_t)(s * XB + X::source(v, lane));
      ox[v] = k < (uint32_t)xrb ? k : 0u;
    }
#pragma unroll
    for (int v = 0; v < W::KINDS; v++) {
      const uint32_t k = (uint32_t)(s * WB + W::source(v, lane));
      ow[v] = k < (uint32_t)wrb ? k : 0u;
    }
#pragma unroll
    for (int i = 0; i < NX; i++) dma16(xb + (xo[i] + ox[i % X::KINDS]), st + 1024 * (NX * wave + i));
#pragma unroll
    for (int i = 0; i < NW; i++) dma16(wb + (wo[i] + ow[i % W::KINDS]), st + BM * XB + 1024 * (NW * wave + i));
  };

  // scales: thread t carries rows t, t + 256, .. of x then w (past the last: that one again)
  constexpr int NS = (BM + BN + 255) / 256;
  const uint8_t* sp[NS];
#pragma unroll
  for (int i = 0; i < NS; i++) {
    const int row = min(tid + 256 * i, BM + BN - 1), b = row - BM;
    sp[i] = row < BM ? a.x_sf + (m0 + min(row, last_m)) * nb
                     : a.w_sf + (int64_t)(n0 + min((b & ~31) + tile_col(b & 31), last_n)) * nb;
  }
  const int sc_first = k_first * (KS / 32);  // scale byte of this K group's first stage
  // (one LDS area: every wave has its records of group g in registers since
  // before the first barrier of the group, and g + 1 is put before the last)
  auto put_scales = [&](const u32x4_t (&v)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; i++)
      *reinterpret_cast<u32x4_t*>(smem + S::SC_OFF + 16 * min(tid + 256 * i, BM + BN - 1)) = v[i];
  };

  // (the scales first: what waits for them does not wait for the stages)
  u32x4_t sv[NS];
#pragma unroll
  for (int i = 0; i < NS; i++)
    sv[i] = nb >= 16 ? ld16u(scale_source(sp[i], sc_first, nb)) : scale_short(sp[i], sc_first, nb);
#pragma unroll
  for (int s = 0; s < NBUF; s++) {
    if (s >= KT) break;
    issue(s, smem + s * S::STAGE);
  }
#pragma unroll
  for (int i = 0; i < NS; i++)
    if (nb >= 16) sv[i] = scale_shift(sv[i], sc_first, nb);
  put_scales(sv);

  f32x16_t acc[TN][TM];
#pragma unroll
  for (int n = 0; n < TN; n++)
#pragma unroll
    for (int m = 0; m < TM; m++)
#pragma unroll
      for (int i = 0; i < 16; i++) acc[n][m][i] = 0.0f;
  if (NBUF <= KT) __builtin_amdgcn_s_waitcnt(waitcnt_vm((NBUF - 1) * ND));
  else __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  ring_barrier();

  const int wrow = 32 * TN * wn + r, xrow = 32 * TM * wm + r;
  u32x4_t w0[TN], w1[TN], sw[TN], sx[TM];
  XFrag<XE> x0[TM], x1[TM];
  // fragment read i of 64-K step u
  auto read = [&](const uint8_t* st, int u, int i, u32x4_t (&w)[TN], XFrag<XE> (&x)[TM]) {
    if (i < TN) {
      w[i] = *reinterpret_cast<const u32x4_t*>(st + BM * XB + 32 * WB * i + W::at(wrow, 2 * u + h));
    } else if (XE == 1) {
      x[i - TN].p[0] = *reinterpret_cast<const u32x4_t*>(st + 32 * XB * (i - TN) + X::at(xrow, 2 * u + h));
    } else {
      const int m = (i - TN) >> 1, e = (i - TN) & 1;
      x[m].p[XE == 1 ? 0 : e] =
          *reinterpret_cast<const u32x4_t*>(st + 32 * XB * m + X::at(xrow, 4 * u + 2 * e + h));
    }
  };
  // this lane's scale records of the group in LDS
  auto read_scales = [&]() {
    const uint8_t* sc = smem + S::SC_OFF;
#pragma unroll
    for (int n = 0; n < TN; n++) {
      sw[n] = *reinterpret_cast<const u32x4_t*>(sc + 16 * (BM + wrow + 32 * n));
#pragma unroll
      for (int i = 0; i < 4; i++) sw[n][i] >>= 8 * h;
    }
#pragma unroll
    for (int m = 0; m < TM; m++) {
      sx[m] = *reinterpret_cast<const u32x4_t*>(sc + 16 * (xrow + 32 * m));
#pragma unroll
      for (int i = 0; i < 4; i++) sx[m][i] >>= 8 * h;
    }
  };
  auto pin_all = [&]() {
#pragma unroll
    for (int i = 0; i < NQ; i++) pin<NQ>(acc[i / TM][i % TM]);
  };
  // reads of one step's fragments between the MFMAs of another
  auto order = [&]() {
#pragma unroll
    for (int i = 0; i < (NF > NQ ? NF : NQ); i++) {
      if (i < NF) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (i < NQ) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // Stage s, number I of its group.
  auto stage = [&](int s, auto I_, int next_group) {
    constexpr int I = decltype(I_)::value;
    uint8_t* st = smem + (s % NBUF) * S::STAGE;
    const uint8_t* sn = smem + ((s + 1) % NBUF) * S::STAGE;
    auto step = [&](auto u_, const u32x4_t (&w)[TN], const XFrag<XE> (&x)[TM], u32x4_t (&wn)[TN], XFrag<XE> (&xn)[TM],
                    const uint8_t* from) {
      constexpr int u = decltype(u_)::value, word = I * (4 / GS) + u / 2;
#pragma unroll
      for (int i = 0; i < NF; i++) read(from, (u + 1) % QS, i, wn, xn);
#pragma unroll
      for (int i = 0; i < NQ; i++)
        mfma_one<XE, u & 1>(acc[i / TM][i % TM], w[i / TM], x[i % TM], (int)sw[i / TM][word], (int)sx[i % TM][word]);
      order();
    };
    step(std::integral_constant<int, 0>{}, w0, x0, w1, x1, st);
    if constexpr (QS == 4) {
      step(std::integral_constant<int, 1>{}, w1, x1, w0, x0, st);
      step(std::integral_constant<int, 2>{}, w0, x0, w1, x1, st);
    }
    if (next_group > 0) {
#pragma unroll
      for (int i = 0; i < NS; i++) sv[i] = scale_shift(sv[i], sc_first + 16 * next_group, nb);
      put_scales(sv);
    }
    // stage s + 1 has landed: with the ring full, all but the newest loads
    if (s + NBUF <= KT) __builtin_amdgcn_s_waitcnt(waitcnt_vm((NBUF - 2) * ND));
    else __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    ring_barrier();
    __builtin_amdgcn_sched_barrier(0);
    // every wave has this stage's fragments: refill its buffer
    if (s + NBUF < KT) issue(s + NBUF, st);
    // (past the last stage: reads that are not used)
    step(std::integral_constant<int, QS - 1>{}, w1, x1, w0, x0, sn);
    pin_all();
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2 % GS>;
  using I3 = std::integral_constant<int, 3 % GS>;

#pragma unroll
  for (int i = 0; i < NF; i++) read(smem, 0, i, w0, x0);
  const int groups = nb >= 16 ? KT / GS : 0;
#pragma unroll 1
  for (int g = 0; g < groups; g++) {
    read_scales();
#pragma unroll
    for (int i = 0; i < NS; i++) sv[i] = ld16u(scale_source(sp[i], sc_first + 16 * (g + 1), nb));
    stage(GS * g, I0{}, 0);
    if constexpr (GS == 4) {
      stage(GS * g + 1, I1{}, 0);
      stage(GS * g + 2, I2{}, 0);
      stage(GS * g + 3, I3{}, g + 1);
    } else {
      stage(GS * g + 1, I1{}, g + 1);
    }
  }
  const int s0 = GS * groups;
  if (s0 < KT) {
    read_scales();
    stage(s0, I0{}, 0);
    if (s0 + 1 < KT) stage(s0 + 1, I1{}, 0);
    if (GS == 4 && s0 + 2 < KT) stage(s0 + 2, I2{}, 0);
    if (GS == 4 && s0 + 3 < KT) stage(s0 + 3, I3{}, 0);
  }
  ring_barrier();  // the other waves have read the stages that the joins and the way out overwrite
  // the K groups' sums: the upper half hands its accumulators to the lower
  // one, until the first group has all of them
#pragma unroll
  for (int half = KG / 2; half >= 1; half /= 2) {
    f32x4_t* to = reinterpret_cast<f32x4_t*>(smem_all);
    if (kg >= half && kg < 2 * half) {
#pragma unroll
      for (int i = 0; i < TN * TM; i++)
#pragma unroll
        for (int c = 0; c < 4; c++)
          to[(((kg - half) * 4 + wave) * TN * TM + i) * 256 + 64 * c + lane] =
              f32x4_t{acc[i / TM][i % TM][4 * c], acc[i / TM][i % TM][4 * c + 1], acc[i / TM][i % TM][4 * c + 2],
                      acc[i / TM][i % TM][4 * c + 3]};
    }
    ring_barrier();
    if (kg < half) {
#pragma unroll
      for (int i = 0; i < TN * TM; i++)
#pragma unroll
        for (int c = 0; c < 4; c++) {
          const f32x4_t v = to[((kg * 4 + wave) * TN * TM + i) * 256 + 64 * c + lane];
#pragma unroll
          for (int e = 0; e < 4; e++) acc[i / TM][i % TM][4 * c + e] += v[e];
        }
    }
    ring_barrier();
  }
  if (kg != 0) return;
  store_tiles<WIDE, TM, TN, 2048>(a, acc, m0 + 32 * TM * wm, n0 + 32 * TN * wn, smem + 2048 * wave, lane);
}

template <int XE, bool WIDE, int TM, int TN, int KS, int NBUF, int KG, int PER_CU>
hipError_t launch_tile_as(const LinearParams& p, hipStream_t s) {
  using S = Shape<XE, TM, TN, KS, NBUF, KG>;
  static_assert(S::LDS * PER_CU <= 160 * 1024, "LDS ring exceeds the CU's LDS");
  int cus = 0;
  const hipError_t err = allow_lds<linear_tile_kernel<XE, WIDE, TM, TN, KS, NBUF, KG, PER_CU>>(S::LDS, &cus);
  if (err != hipSuccess) return err;
  const int tm = (p.M + S::BM - 1) / S::BM, tn = (p.N + S::BN - 1) / S::BN;
  const unsigned grid = (unsigned)(((int64_t)tm * tn + 7) / 8 * 8);
  linear_tile_kernel<XE, WIDE, TM, TN, KS, NBUF, KG, PER_CU><<<grid, 256 * KG, S::LDS, s>>>(p, tm, tn);
  return hipGetLastError();
}

// bf16 y that is overwritten, its rows aligned to 16 bytes
bool wide_rows(const LinearParams& p) {
  return !p.y_f32 && !p.accumulate && p.N % 8 == 0 && ((uintptr_t)p.y & 15) == 0;
}

template <int XE, int TM, int TN, int KS, int NBUF, int KG, int PER_CU>
hipError_t launch_tile(const LinearParams& p, hipStream_t s) {
  return wide_rows(p) ? launch_tile_as<XE, true, TM, TN, KS, NBUF, KG, PER_CU>(p, s)
                      : launch_tile_as<XE, false, TM, TN, KS, NBUF, KG, PER_CU>(p, s);
}

// ------------------------------------------------------------- persistent kernel

// 256 x 256 tiles, one workgroup of 8 wavefronts a CU, two a SIMD (one with
// 128 x 128 results would read a third less from LDS, but its accumulators and
// fragments do not fit the registers without spills).  A workgroup walks its
// tiles with one stream of stages: the first stages of the next tile are loaded
// while the last ones of this tile multiply, so that only the first tile waits
// for memory.  A stage of 256 K is 2048 cycles of matrix cores for E2M1, and
// 196 KiB of fragment reads and 64 KiB of loads in LDS, another 2048 cycles if
// nothing overlapped.  16384 x 6144 x 4096: E2M1 207 us at best, 220 - 250 from
// launch to launch (3.3 - 4.0 PFLOP/s, the matrix cores 47% busy at 2.0 GHz), E4M3
// 333 - 374 us (2.2 - 2.5).  Wave priorities and other orders of the reads: the same.  At 8192 x
// 8192 x 8192 E2M1, 264 us: without the loads 221, without the fragment reads
// 223, the instructions alone 176.
template <int XE>
struct Big {
  static constexpr int TM = 2, TN = 4;               // 32-row tiles of a wavefront
  static constexpr int WM = 4, WN = 2;               // wavefronts along m and n
  static constexpr int NT = 64 * WM * WN;
  static constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN;
  static constexpr int KS = XE == 1 ? 256 : 128;     // K per stage: 128-byte lines of an x row
  static constexpr int NBUF = XE == 1 ? 2 : 3;
  static constexpr int XB = 128, WB = KS / 2;        // bytes of a row in a stage
  static constexpr int X_BYTES = BM * XB;
  static constexpr int STAGE = X_BYTES + BN * WB;    // 64 / 48 KiB
  static constexpr int RB = KS / 16;                 // scale record of a row: two stages
  static constexpr int SC = (BM + BN) * RB;          // two areas of records
  static constexpr int SC_OFF = NBUF * STAGE;
  static constexpr int OUT = XE == 1 ? 2048 : 1024;  // a wavefront's way out: rows of 64 bytes
  static constexpr int T_OFF = SC_OFF + 2 * SC;
  static constexpr int LDS = T_OFF + WM * WN * OUT;  // 160 KiB
};

// scale record g (RB bytes) of a row of nb >= RB bytes, in two steps as scale_source / scale_shift
template <int RB>
struct Record {
  uint32_t v[RB / 4];
};
template <int RB>
DEV Record<RB> record_load(const uint8_t* row, int g, int nb) {
  Record<RB> o;
  __builtin_memcpy(&o, row + min(RB * g, nb - RB), RB);
  return o;
}
template <int RB>
DEV Record<RB> record_shift(const Record<RB>& v, int g, int nb) {
  const int over = max(0, RB * (g + 1) - nb);
  const int w = over >> 2, b = 8 * (over & 3);
  Record<RB> o;
#pragma unroll
  for (int i = 0; i < RB / 4; i++) {
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int j = i; j < RB / 4; j++) {
      lo = j == i + w ? v.v[j] : lo;
      hi = j == i + w + 1 ? v.v[j] : hi;
    }
    o.v[i] = (uint32_t)((((uint64_t)hi << 32) | lo) >> b);
  }
  return o;
}

template <int XE>
__global__ __launch_bounds__(Big<XE>::NT, 1) void linear_big_kernel(const LinearParams a, int tiles_m, int tiles_n) {
  using S = Big<XE>;
  constexpr int TM = S::TM, TN = S::TN, BM = S::BM, BN = S::BN, XB = S::XB, WB = S::WB, NT = S::NT, RB = S::RB;
  constexpr int NX = S::X_BYTES / 16 / NT, NW = BN * WB / 16 / NT;  // LDS-DMA loads a wavefront and stage
  constexpr int ND = NX + NW;
  constexpr int NQ = TN * TM;                                       // MFMAs of 64 K
  constexpr int NF = TN + TM * (XE == 1 ? 1 : 2);                   // their fragment reads
  constexpr int QS = S::KS / 64;                                    // 64-K steps of a stage
  constexpr int RW = S::KS / 128;                                   // scale words of a row and stage
  static_assert(S::WN == 2 && NX % 2 == 0 && NW % 2 == 0, "the swizzles go by a load's number");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  const int r = lane & 31, h = lane >> 5;
  const int KT = (a.K + 2 * S::KS - 1) / (2 * S::KS) * 2, nb = a.K / 32;  // whole scale records
  const int xrb = XE == 1 ? a.K / 2 : a.K, wrb = a.K / 2;

  // tiles of this workgroup: XCD b & 7 takes a contiguous run of tiles, its
  // workgroups take them in turn; GM tile rows high, so that the 32 concurrent
  // tiles of an XCD are 8 x 4 and share their rows in its L2
  const int tiles = tiles_m * tiles_n, per = (tiles + 7) / 8, step = gridDim.x >> 3;
  const int first = (blockIdx.x & 7) * per, end = min(first + per, tiles);
  int t = first + (blockIdx.x >> 3);
  if (t >= end) return;
  auto tile_at = [&](int t, int64_t& m0, int& n0) {
    constexpr int GM = 8;
    const int group = t / (GM * tiles_n), in = t % (GM * tiles_n);
    const int rows = min(GM, tiles_m - group * GM);
    m0 = (int64_t)(group * GM + in % rows) * BM;
    n0 = (in / rows) * BN;
  };

  // what the loads of the moment read: tile bases, this lane's row offsets
  // (rows past the end: the last row, whose products are not stored) and this
  // thread's scale row (NT = BM + BN: one each)
  static_assert(NT == BM + BN, "a thread carries one row's scales");
  const uint8_t *xb, *wb, *sp;
  uint32_t xo[NX], wo[NW];
  auto aim = [&](int64_t m0, int n0) {
    xb = a.x + m0 * xrb;
    wb = a.w + (int64_t)n0 * wrb;
    const int last_m = (int)min((int64_t)BM, a.M - m0) - 1, last_n = min(BN, a.N - n0) - 1;
#pragma unroll
    for (int j = 0; j < NX; j++) xo[j] = (uint32_t)min(8 * (NX * wave + j) + (lane >> 3), last_m) * (uint32_t)xrb;
#pragma unroll
    for (int j = 0; j < NW; j++) {
      const int b = WB == 128 ? 8 * (NW * wave + j) + (lane >> 3) : 16 * (NW * wave + j) + (lane >> 2);
      wo[j] = (uint32_t)min((b & ~31) + tile_col(b & 31), last_n) * (uint32_t)wrb;
    }
    const int row = threadIdx.x, b = row - BM;
    sp = row < BM ? a.x_sf + (m0 + min(row, last_m)) * nb
                  : a.w_sf + (int64_t)(n0 + min((b & ~31) + tile_col(b & 31), last_n)) * nb;
  };
  // logical chunk (16 bytes) of the physical one a lane fills: rows of 8
  // chunks are swizzled by row / 2, whose bit 2 is the load's parity; rows of
  // 4 chunks by row / 4
  const int c8 = 16 * ((lane & 7) ^ ((lane >> 4) & 3));
  const int c4 = 16 * ((lane & 3) ^ ((lane >> 4) & 3));
  // K offsets of stage s's loads; a chunk past the end of its row: the row's
  // first one (its scale is 0)
  struct Offs {
    uint32_t w[2], x[2];
  };
  auto offsets = [&](int s) {
    Offs o;
#pragma unroll
    for (int v = 0; v < 2; v++) {
      const uint32_t kw = (uint32_t)(s * WB + (WB == 128 ? c8 ^ (64 * v) : c4)), kx = (uint32_t)(s * XB + (c8 ^ (64 * v)));
      o.w[v] = kw < (uint32_t)wrb ? kw : 0u;
      o.x[v] = kx < (uint32_t)xrb ? kx : 0u;
    }
    return o;
  };
  auto issue_one = [&](const Offs& o, uint8_t* st, int i) {
    if (i < NX) dma16(xb + (xo[i] + o.x[i & 1]), st + 1024 * (NX * wave + i));
    else dma16(wb + (wo[i - NX] + o.w[i & 1]), st + S::X_BYTES + 1024 * (NW * wave + i - NX));
  };

  u32x4_t w0[TN], w1[TN];
  XFrag<XE> x0[TM], x1[TM];
  uint32_t sw[TN][RW], sx[TM][RW], swn[TN][RW], sxn[TM][RW];  // this stage's and the next one's scale words
  Record<RB> sv;
  f32x16_t acc[TN][TM];
  const int wrow = 32 * TN * wn + r, xrow = 32 * TM * wm + r;
  const int sw8 = (r >> 1) & 7, sw4 = (r >> 2) & 3;
  // fragment read i of 64-K step u
  auto read = [&](const uint8_t* st, int u, int i, u32x4_t (&w)[TN], XFrag<XE> (&x)[TM]) {
    if (i < TN) {
      w[i] = *reinterpret_cast<const u32x4_t*>(st + S::X_BYTES + (wrow + 32 * i) * WB +
                                               16 * ((2 * u + h) ^ (WB == 128 ? sw8 : sw4)));
    } else if (XE == 1) {
      x[i - TN].p[0] = *reinterpret_cast<const u32x4_t*>(st + (xrow + 32 * (i - TN)) * XB + 16 * ((2 * u + h) ^ sw8));
    } else {
      const int m = (i - TN) >> 1, e = (i - TN) & 1;
      x[m].p[XE == 1 ? 0 : e] =
          *reinterpret_cast<const u32x4_t*>(st + (xrow + 32 * m) * XB + 16 * ((4 * u + 2 * e + h) ^ sw8));
    }
  };
  auto put_record = [&](int area) {
    *reinterpret_cast<Record<RB>*>(smem + S::SC_OFF + area * S::SC + RB * threadIdx.x) = sv;
  };
  // the scale words of stage I of the records in an area
  auto read_scales = [&](int area, int I) {
    const uint8_t* sc = smem + S::SC_OFF + area * S::SC + 4 * RW * I;
#pragma unroll
    for (int n = 0; n < TN; n++)
#pragma unroll
      for (int i = 0; i < RW; i++) swn[n][i] = reinterpret_cast<const uint32_t*>(sc + RB * (BM + wrow + 32 * n))[i];
#pragma unroll
    for (int m = 0; m < TM; m++)
#pragma unroll
      for (int i = 0; i < RW; i++) sxn[m][i] = reinterpret_cast<const uint32_t*>(sc + RB * (xrow + 32 * m))[i];
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int i = 0; i < RW; i++) {
#pragma unroll
      for (int n = 0; n < TN; n++) sw[n][i] = swn[n][i] >> (8 * h);
#pragma unroll
      for (int m = 0; m < TM; m++) sx[m][i] = sxn[m][i] >> (8 * h);
    }
  };

  int buf = 0, area = 0;
  // One stage, number I (0, 1) of its scale record; `is`: the stage of the
  // aimed-at tile that its loads fetch (NBUF ahead in the stream of stages).
  // I = 0 puts the next record (sv, number `next`), which I = 1 reads.  LAST:
  // the reads of the next stage's first fragments are left out.
  auto stage = [&](auto I_, int is, int next, auto last_) {
    constexpr int I = decltype(I_)::value;
    constexpr bool LAST = decltype(last_)::value;
    uint8_t* st = smem + buf * S::STAGE;
    buf = buf == S::NBUF - 1 ? 0 : buf + 1;
    const uint8_t* sn = smem + buf * S::STAGE;
    take_scales();
    auto step = [&](auto u_, const u32x4_t (&w)[TN], const XFrag<XE> (&x)[TM], u32x4_t (&wn)[TN], XFrag<XE> (&xn)[TM]) {
      constexpr int u = decltype(u_)::value;
#pragma unroll
      for (int i = 0; i < NF; i++) read(st, u + 1, i, wn, xn);
      if constexpr (u == QS - 2) read_scales(I == 0 ? area : area ^ 1, I ^ 1);
#pragma unroll
      for (int i = 0; i < NQ; i++)
        mfma_one<XE, u & 1>(acc[i / TM][i % TM], w[i / TM], x[i % TM], (int)sw[i / TM][u / 2], (int)sx[i % TM][u / 2]);
#pragma unroll
      for (int i = 0; i < NQ; i++) {
        __builtin_amdgcn_sched_group_barrier(0x100, (NF + NQ - 1) / NQ, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    step(std::integral_constant<int, 0>{}, w0, x0, w1, x1);
    if constexpr (QS == 4) {
      step(std::integral_constant<int, 1>{}, w1, x1, w0, x0);
      step(std::integral_constant<int, 2>{}, w0, x0, w1, x1);
    }
    if constexpr (I == 0) {
      sv = record_shift(sv, next, nb);
      put_record(area ^ 1);
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm((S::NBUF - 2) * ND));  // the next stage has landed
    ring_barrier();
    __builtin_amdgcn_sched_barrier(0);
    // every wave has this stage's fragments: refill its buffer
    const Offs o = offsets(is);
    constexpr int DQ = (ND + NQ - 1) / NQ, RQ = (NF + NQ - 1) / NQ;
#pragma unroll
    for (int i = 0; i < NQ; i++) {
#pragma unroll
      for (int j = 0; j < DQ; j++)
        if (DQ * i + j < ND) issue_one(o, st, DQ * i + j);
      mfma_one<XE, 1>(acc[i / TM][i % TM], w1[i / TM], x1[i % TM], (int)sw[i / TM][RW - 1], (int)sx[i % TM][RW - 1]);
#pragma unroll
      for (int j = 0; j < RQ; j++)
        if (!LAST && RQ * i + j < NF) read(sn, 0, RQ * i + j, w0, x0);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (I == 1) area ^= 1;
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  const std::true_type last;
  const std::false_type mid;
  auto pin_all = [&]() {
#pragma unroll
    for (int i = 0; i < NQ; i++) pin<NQ>(acc[i / TM][i % TM]);
  };

  int64_t m0;
  int n0;
  tile_at(t, m0, n0);
  aim(m0, n0);
  sv = record_load<RB>(sp, 0, nb);
#pragma unroll
  for (int s = 0; s < S::NBUF; s++) {
    const Offs o = offsets(s);
#pragma unroll
    for (int i = 0; i < ND; i++) issue_one(o, smem + s * S::STAGE, i);
  }
  sv = record_shift(sv, 0, nb);
  put_record(0);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm((S::NBUF - 1) * ND));
  ring_barrier();
  read_scales(0, 0);

#pragma unroll 1
  for (;;) {
#pragma unroll
    for (int i = 0; i < NF; i++) read(smem + buf * S::STAGE, 0, i, w0, x0);
#pragma unroll
    for (int i = 0; i < NQ; i++)
#pragma unroll
      for (int j = 0; j < 16; j++) acc[i / TM][i % TM][j] = 0.0f;
    const int tn = t + step;
    const bool more = tn < end;
    int64_t mn = m0;
    int nn = n0;
    if (more) tile_at(tn, mn, nn);

    // stages s, s + 1 fetch s + NBUF and s + NBUF + 1; the last NBUF of a tile
    // the first ones of the next tile (without one, of this tile, unread)
    int g = 0;
#pragma unroll 1
    for (; 2 * g + 1 + S::NBUF < KT; g++) {
      sv = record_load<RB>(sp, g + 1, nb);
      stage(I0{}, 2 * g + S::NBUF, g + 1, mid);
      stage(I1{}, 2 * g + 1 + S::NBUF, 0, mid);
    }
    pin_all();
    if constexpr (S::NBUF == 3) {  // KT - 4 .. KT - 1: the first of them still fetches KT - 1
      sv = record_load<RB>(sp, g + 1, nb);
      stage(I0{}, KT - 1, g + 1, mid);
      pin_all();
      aim(mn, nn);
      sv = record_load<RB>(sp, 0, nb);
      stage(I1{}, 0, 0, mid);
      stage(I0{}, 1, 0, mid);
      stage(I1{}, 2, 0, last);
    } else {
      aim(mn, nn);
      sv = record_load<RB>(sp, 0, nb);
      stage(I0{}, 0, 0, mid);
      stage(I1{}, 1, 0, last);
    }
    pin_all();
    store_tiles<true, TM, TN, S::OUT>(a, acc, m0 + 32 * TM * wm, n0 + 32 * TN * wn, smem + S::T_OFF + S::OUT * wave, lane);
    if (!more) break;
    t = tn;
    m0 = mn;
    n0 = nn;
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));  // no LDS-DMA load may be in flight when the workgroup ends
}

template <int XE>
hipError_t launch_big(const LinearParams& p, hipStream_t s) {
  using S = Big<XE>;
  static_assert(S::LDS <= 160 * 1024, "LDS ring exceeds the CU's LDS");
  int cus = 0;
  const hipError_t err = allow_lds<linear_big_kernel<XE>>(S::LDS, &cus);
  if (err != hipSuccess) return err;
  const int tm = (p.M + S::BM - 1) / S::BM, tn = (p.N + S::BN - 1) / S::BN;
  const int grid = cus / 8 * 8 > 8 ? cus / 8 * 8 : 8;  // one workgroup a CU, as many on every XCD
  linear_big_kernel<XE><<<grid, S::NT, S::LDS, s>>>(p, tm, tn);
  return hipGetLastError();
}

// ------------------------------------------------------------- streaming kernel

// 16 rows of x a workgroup (decoding): it streams 16 rows of W once, its
// wavefronts splitting K, straight into registers; their sums meet in LDS in
// a fixed order.  8 x 4096 x 6144 E2M1: 6.8 - 7.0 us for 13.4 MB of W, of which 2.1
// are a kernel's start and end; the rest goes at the 2.8 TB/s (4.7 us) that one
// workgroup a CU asks for, whose eight wavefronts have six steps each under way
// (K = 24576: 21.0 us).  v_mfma_scale_f32_16x16x128_f8f6f4: lane (row or column r
// = lane & 15, group q = lane >> 4) holds block q of each 128 values of an E2M1
// row (16 bytes), or of an E4M3 row its halves 16 q .. and 64 + 16 q .., and
// block q's scale.
constexpr int STREAM_WAVES = 8;

template <int XE>
__global__ __launch_bounds__(64 * STREAM_WAVES) void linear_stream_kernel(const LinearParams a) {
  constexpr int NW = STREAM_WAVES;
  __shared__ f32x4_t part[NW][64];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16;
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  const int nb = a.K / 32, steps = (nb + 3) / 4;
  const int per = (steps + NW - 1) / NW, s_first = wave * per, s_end = min(s_first + per, steps);
  const int64_t wr = min(a.N - 1, n0 + r), xr = min((int64_t)a.M - 1, m0 + r);
  const uint8_t *w = a.w + wr * (a.K / 2) + 16 * q, *wsf = a.w_sf + wr * nb;
  const uint8_t *x = a.x + xr * (XE == 1 ? a.K / 2 : a.K) + 16 * q, *xsf = a.x_sf + xr * nb;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  auto mul = [&](const u32x4_t& wv, int ws, const u32x4_t& lo, const u32x4_t& hi, int xs) {
    const i32x8_t b = {(int)wv[0], (int)wv[1], (int)wv[2], (int)wv[3], 0, 0, 0, 0};
    const i32x8_t c = {(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(c, b, acc, XE == 1 ? 4 : 0, 4, 0, xs, 0, ws);
  };
  // the four scale bytes of a whole step, this lane's lowest
  auto scale4 = [&](const uint8_t* sf, int s) {
    uint32_t v;
    __builtin_memcpy(&v, sf + 4 * s, 4);
    return (int)(v >> (8 * q));
  };
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  constexpr int U = 6;  // steps whose loads go out together
  int s = s_first;
  const int whole = min(s_end, nb / 4);
  for (; s + U <= whole; s += U) {
    u32x4_t wv[U], lo[U], hi[U];
    int ws[U], xs[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      wv[u] = ld16(w + 64 * (s + u));
      ws[u] = scale4(wsf, s + u);
      lo[u] = ld16(x + (XE == 1 ? 64 : 128) * (s + u));
      hi[u] = XE == 1 ? zero : ld16(x + 128 * (s + u) + 64);
      xs[u] = scale4(xsf, s + u);
    }
#pragma unroll
    for (int u = 0; u < U; u++) mul(wv[u], ws[u], lo[u], hi[u], xs[u]);
  }
  for (; s < s_end; s++) {  // the rest, the last step perhaps not whole
    const bool in = 4 * s + q < nb;
    u32x4_t lo = zero, hi = zero;
    if (XE == 1) {
      if (in) lo = ld16(x + 64 * s);
    } else {
      if (128 * s + 16 * q < a.K) lo = ld16(x + 128 * s);
      if (128 * s + 64 + 16 * q < a.K) hi = ld16(x + 128 * s + 64);
    }
    mul(in ? ld16(w + 64 * s) : zero, in ? wsf[4 * s + q] : 0, lo, hi, in ? xsf[4 * s + q] : 0);
  }
  part[wave][lane] = acc;
  __syncthreads();
  // element i of lane (r, q): row 4 q + i, column r
  if (threadIdx.x >= 64 || n0 + r >= a.N) return;
  f32x4_t v = part[0][lane];
#pragma unroll
  for (int k = 1; k < NW; k++) v += part[k][lane];
  const int n = n0 + r;
  const float alpha = a.alpha ? *a.alpha : 1.0f, bias = a.bias ? a.bias[n] : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t row = m0 + 4 * q + i;
    if (row >= a.M) continue;
    const float o = scaled(v[i], alpha, bias);
    const int64_t at = row * a.N + n;
    if (a.y_f32) {
      float* y = reinterpret_cast<float*>(a.y) + at;
      *y = a.accumulate ? *y + o : o;
    } else {
      uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + at;
      *y = f32_to_bf16(a.accumulate ? bf16_to_f32(*y) + o : o);
    }
  }
}

template <int XE>
hipError_t launch(const LinearParams& p, hipStream_t s) {
  constexpr int64_t CUS = 256;
  auto tiles = [&](int m, int n) { return (int64_t)((p.M + m - 1) / m) * ((p.N + n - 1) / n); };
  // The streaming kernel for one row of 16 x 16 tiles, or while there is at
  // most one of them a CU: its K is split eight ways (128 x 300 x 4992, E2M1:
  // 5.4 us against 8.0 us tiled; 32 x 4096 x 6144, two a CU: 13.1 against 8.9).
  if (p.M <= 16 || tiles(16, 16) <= CUS) {
    const dim3 grid((unsigned)((p.N + 15) / 16), (unsigned)((p.M + 15) / 16));
    linear_stream_kernel<XE><<<grid, 64 * STREAM_WAVES, 0, s>>>(p);
    return hipGetLastError();
  }
  // Few tiles: 64 x 64, with K split in two where it is long (E2M1: 128 x 4096
  // x 4096 7.4 us against 8.2; 64 x 8192 x 1024 4.5 against 4.3).
  if (tiles(64, 64) <= CUS)
    return p.K >= 2048 ? launch_tile<XE, 1, 1, 128, 4, 2, 1>(p, s) : launch_tile<XE, 1, 1, 256, 2, 1, 2>(p, s);
  const int64_t t128 = tiles(128, 128);
  // K split in two goes by the shape alone, whatever becomes of the sums: it is
  // in their order.  Sums that leave as fp32, onto y or in narrower pieces have 64 x
  // 128 tiles at every size, whose bound is the trips of the stages and, where rows
  // are not whole 16 bytes, single elements (16384 x 6144 x 4096, E2M1 / E4M3: fp32
  // 448 / 540 us, accumulated bf16 438 / 511, accumulated fp32 534 / 621, N = 6147
  // 424 / 513 and accumulated 794 / 857, against 250 / 355 for aligned bf16 in
  // the same run; 2048 x 4096 x 2048 fp32 27 / 31 against 16 / 22).
  const bool halves = XE == 0 && t128 <= CUS / 2 && p.K >= 2048;
  if (!wide_rows(p)) {
    if constexpr (XE == 0)
      if (halves) return launch_tile_as<0, false, 1, 2, 256, 2, 2, 1>(p, s);
    return launch_tile_as<XE, false, 1, 2, 256, XE == 1 ? 3 : 2, 1, 2>(p, s);
  }
  // 256 x 256 tiles in whole rounds of the CUs, three quarters full at least
  // (2048 x 6144 x 4096, 0.75: 34.7 us against 44.5 in 128 x 128 tiles; 4096 x
  // 5120 x 2048, 0.63: 37.1 against 37.2, E4M3 53.9 against 47.0), and with
  // enough stages to fill its pipeline (8192 x 8192 x 512: 53.0 against 39.9).
  const int64_t big = tiles(256, 256), rounds = (big + CUS - 1) / CUS;
  if (p.K >= 1024 && 4 * big >= 3 * CUS * rounds) return launch_big<XE>(p, s);
  // Between, stages of 256 K load whole lines of W (64 x 128 x 128 stages reach
  // 14 TB/s from L2 into LDS and are bound by it).  E2M1: 64 x 64 tiles, from
  // three quarters of a round of them on 128 x 128 (512 x 4096 x 4096, 128 of
  // them: 11.0 us against 14.6; 1024 x 4096 x 4096, 256: 18.2 against 16.0).
  // E4M3: 64 x 128 tiles, with K split in two up to half a round of 128 x 128
  // (512 x 4096 x 4096: 13.4 against 15.4; 1024 x 4096 x 4096: 25.4 against
  // 21.3), and 128 x 128 above a whole one (2048 x 4096 x 2048: 20.5 against
  // 22.4).
  if constexpr (XE == 1) {
    if (t128 <= CUS * 3 / 4) return launch_tile_as<1, true, 1, 1, 256, 2, 1, 2>(p, s);
    return launch_tile_as<1, true, 2, 2, 256, 2, 1, 2>(p, s);
  } else {
    if (halves) return launch_tile_as<0, true, 1, 2, 256, 2, 2, 1>(p, s);
    if (t128 <= CUS) return launch_tile_as<0, true, 1, 2, 256, 2, 1, 2>(p, s);
    return launch_tile_as<0, true, 2, 2, 128, 3, 1, 2>(p, s);
  }
}

}  // namespace

hipError_t launch_linear_mx(const LinearParams& p, hipStream_t s) {
  return p.x_elem == 1 ? launch<1>(p, s) : launch<0>(p, s);
}

}  // namespace moe
