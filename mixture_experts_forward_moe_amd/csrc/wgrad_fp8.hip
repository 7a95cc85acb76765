// wgrad_fp8.hip -- the gradient of a product's weights, dW = dy^T x, from rows of
// x kept in 8 bits: of one matrix, or of every expert from its rows.
//
// The sum runs over the rows, in which both operands are contiguous the other
// way; gfx950's transposing LDS read (ds_read_b64_tr_b16) turns 4 rows of 16
// values into the fragments that the matrix instruction takes.  x's codes are
// decoded to bf16 once a workgroup, on their way into LDS: a code times a power
// of two is exact there (under the three least scales for the codes that bf16 values
// were quantised to), so the products are exact and the sums fp32.
#include "device_common.h"
#include "dynamic_lds.h"
#include "internal.h"

namespace moe {

namespace {

typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
typedef __attribute__((address_space(3))) u32x4_t lds_u32x4_t;

// LDS at a byte address
template <typename T>
DEV T* lds(uint32_t at) {
  return (T*)(uintptr_t)at;
}

// 16 codes under one E8M0 code as bf16 pairs
DEV void decode16(const u32x4_t& c, uint32_t code, u32x4_t& lo, u32x4_t& hi) {
  const float s = e8m0_scale_operand(code);
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t v = c[i];
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, s, false);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, s, true);
    u32x4_t& o = i < 2 ? lo : hi;
    o[2 * (i & 1)] = __builtin_bit_cast(uint32_t, a);
    o[2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, b);
  }
}

// workgroup barrier over LDS that waits for this wavefront's LDS accesses but the
// newest LEFT (a release fence would also wait for every load in flight)
template <int LEFT>
DEV void stage_barrier() {
  static_assert(LEFT <= 15, "four bits");
  __builtin_amdgcn_s_waitcnt(0xC07F | (LEFT << 8));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int TN_, int TK_, int MG_>
struct Tile {
  static constexpr int MG = MG_;                  // groups of four wavefronts that split the rows
  static constexpr int TN = TN_, TK = TK_;        // 16 x 16 results of a wavefront, four of them as 2 x 2
  static constexpr int BN = 32 * TN, BK = 32 * TK;
  static constexpr int ST = 32;                   // rows of a stage
  static constexpr int PN = 2 * BN, PK = 2 * BK;  // bytes of a row in LDS
  static constexpr int STAGE = ST * (PN + PK);
  static constexpr int BUFFERS = 3 * STAGE;       // of a group
  static constexpr int LDS = MG * BUFFERS;
  static constexpr int ND = ST * PN / 4096;       // 16-byte loads of dy a thread and stage
  static constexpr int NX = ST * BK / 4096;       // and of x
};

// The units of 32 bytes (16 values) of row m are swizzled by this, so that the
// eight rows that half a wavefront's transposing read takes (0 - 3 and 8 - 11
// past a multiple of 16, or four more) lie in different banks.
template <int P>
DEV int swizzle(int m) {
  if constexpr (P >= 256) return (m & 3) | (((m >> 3) & 1) << 2);
  else return ((m >> 1) & 1) | (((m >> 3) & 1) << 1);
}

// One tile of dW a workgroup.  Both operands go through registers: loaded four
// stages ahead, written into LDS two ahead between the multiplications, so that a
// wavefront's fragments of the next stage are on their way at the barrier (with two
// buffers, all of a stage written behind its last read: 16384 x 4096 x 6144 790 us,
// now 735 - 750, 1.1 PFLOP/s; experts of 16384 tokens 1435, now 1200 - 1290; added onto
// what dw holds 764 and 1930).  (LDS-DMA of dy is slower: the
// compiler cannot tell its target from what a transposing read takes, and waits
// for all of it.)  Rows past the end of the range are read as 0: the buffers
// end there.
template <typename S>
__global__ __launch_bounds__(256 * S::MG, S::MG == 4 ? 4 : 2) void wgrad_kernel(const WgradParams a, int tiles_n, int tiles_k) {
  constexpr int TN = S::TN, TK = S::TK, PN = S::PN, PK = S::PK, ND = S::ND, NX = S::NX, MG = S::MG;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_all[];
  const int tid = threadIdx.x & 255, lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wn = wave & 1, wk = wave >> 1;
  const int mg = MG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);

  // tile of this workgroup: an XCD (workgroups are dealt to them round robin) takes
  // a run of every expert's tiles, so that experts with many rows cost all XCDs the
  // same, 8 tiles of n high, so that those it works on share their rows in its L2
  const int tiles = tiles_n * tiles_k, per = (tiles + 7) / 8;
  const int slot = blockIdx.x >> 3, e = slot / per, t = (blockIdx.x & 7) * per + slot - e * per;
  if (e >= a.experts || t >= tiles) return;
  constexpr int GM = 8;
  const int group = t / (GM * tiles_k), in = t - group * GM * tiles_k;
  const int high = min(GM, tiles_n - group * GM);
  const int n0 = (group * GM + in % high) * S::BN, k0 = in / high * S::BK;

  // rows of this group: as many stages for each (past the end they are 0)
  const int64_t all = a.offsets ? ld_uniform(a.counts + e) : a.M;
  if (all == 0 && a.accumulate) return;  // nothing to add
  const int stages = (int)((all + S::ST * MG - 1) / (S::ST * MG));
  const int64_t skip = (int64_t)mg * stages * S::ST, first = (a.offsets ? ld_uniform(a.offsets + e) : 0) + skip;
  const int64_t rows = all - skip;
  const int nb = (a.K + 127) / 128;

  // thread's rows of a stage and the 16 bytes it loads of each: 8 values of dy, 16
  // codes of x (columns past the end of a row of dy: of the next row, not stored)
  constexpr int CD = S::BN / 8, CX = S::BK / 16;  // threads a row
  const int dm = tid / CD, dc = tid % CD, xm = tid / CX, xc = tid % CX;
  const bool inside = k0 + 16 * xc < a.K;
  const uint32_t past = 0x80000000u;  // (reads as 0)
  struct Rows {
    u32x4_t d[ND], q[NX];
    uint32_t sf[NX];
  };
  struct From {  // of a stage: buffers that end with the range
    __amdgpu_buffer_rsrc_t d, q, sf;
  };
  auto from = [&](int s) {
    const int64_t m0 = first + (int64_t)s * S::ST;
    const int left = (int)min((int64_t)S::ST, max((int64_t)0, rows - (int64_t)s * S::ST));
    From o;
    o.d = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(a.dy + m0 * a.N), 0, left * 2 * a.N, 0x00020000);
    o.q = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.x + m0 * a.K), 0, left * a.K, 0x00020000);
    o.sf = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.x_sf + m0 * nb), 0, left * nb, 0x00020000);
    return o;
  };
  const uint32_t d_from = (uint32_t)(dm * 2 * a.N + 2 * n0 + 16 * dc);
  const uint32_t q_from = inside ? (uint32_t)(xm * a.K + k0 + 16 * xc) : past;
  const uint32_t sf_from = inside ? (uint32_t)(xm * nb + ((k0 + 16 * xc) >> 7)) : past;
  auto load_d = [&](const From& f, Rows& o, int i) {
    o.d[i] = __builtin_amdgcn_raw_buffer_load_b128(f.d, d_from + (uint32_t)(256 / CD * i * 2 * a.N), 0, 0);
  };
  auto load_x = [&](const From& f, Rows& o, int i) {
    o.q[i] = __builtin_amdgcn_raw_buffer_load_b128(f.q, q_from + (uint32_t)(256 / CX * i * a.K), 0, 0);
    o.sf[i] = __builtin_amdgcn_raw_buffer_load_b8(f.sf, sf_from + (uint32_t)(256 / CX * i * nb), 0, 0);
  };
  auto load = [&](int s, Rows& o) {
    const From f = from(s);
#pragma unroll
    for (int i = 0; i < NX; i++) load_x(f, o, i);
#pragma unroll
    for (int i = 0; i < ND; i++) load_d(f, o, i);
  };
  // LDS addresses in the first of the group's buffers: where this thread's rows
  // go (those of x are 16 apart and those of dy 16 or 32, so they have one swizzle),
  // and of the fragments of 16 columns, rows 8 q .. 8 q + 7, two reads whose lane
  // addresses 4 columns of one row; column tile j is the first one's address xor 32 j
  static_assert((256 / CX % 16 == 0 || NX == 1) && 256 / CD % 16 == 0, "rows of a thread");
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem_all + mg * S::BUFFERS;
  const uint32_t x_to = base + S::ST * PN + xm * PK + 32 * (xc ^ swizzle<PK>(xm));
  const uint32_t d_to = base + dm * PN + 32 * ((dc >> 1) ^ swizzle<PN>(dm)) + 16 * (dc & 1);
  const int fm = 8 * q + (r >> 2);
  const uint32_t d_at = (base + fm * PN + 32 * swizzle<PN>(fm) + 8 * (r & 3)) ^ (32 * TN * wn);
  const uint32_t x_at = (base + S::ST * PN + fm * PK + 32 * swizzle<PK>(fm) + 8 * (r & 3)) ^ (32 * TK * wk);
  auto store_x = [&](const Rows& o, uint32_t st, int i) {
    u32x4_t lo, hi;
    decode16(o.q[i], o.sf[i], lo, hi);
    lds_u32x4_t* p = lds<lds_u32x4_t>(x_to + st + (uint32_t)(256 / CX * i * PK));
    p[0] = lo;
    p[1] = hi;
  };
  auto store_d = [&](const Rows& o, uint32_t st, int i) {
    *lds<lds_u32x4_t>(d_to + st + (uint32_t)(256 / CD * i * PN)) = o.d[i];
  };
  auto store = [&](const Rows& o, uint32_t st) {
#pragma unroll
    for (int i = 0; i < NX; i++) store_x(o, st, i);
#pragma unroll
    for (int i = 0; i < ND; i++) store_d(o, st, i);
  };
  auto frag = [&](uint32_t at, int pitch) {
    const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds<lds_i16x4_t>(at));
    const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds<lds_i16x4_t>(at + (uint32_t)(4 * pitch)));
    typedef short i16x8_t __attribute__((ext_vector_type(8)));
    const i16x8_t v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8_t, v);
  };

  f32x4_t acc[TK][TN];
#pragma unroll
  for (int i = 0; i < TK; i++)
#pragma unroll
    for (int j = 0; j < TN; j++) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  if (stages > 0) {
    Rows x0, x1;
    load(0, x0);
    load(1, x1);
    store(x0, 0);
    load(2, x0);
    store(x1, S::STAGE);
    load(3, x1);
    stage_barrier<0>();
    constexpr int AHEAD = 3, RING = 4;  // x's fragments
    bf16x8_t d0[TN], d1[TN], f[RING];
    uint32_t b0 = 0, b1 = S::STAGE, b2 = 2 * S::STAGE;  // buffers of this stage, the next one, the one after it
    auto read_d = [&](uint32_t st, int j) { return frag((d_at + st) ^ (32u * j), PN); };
    auto read_x = [&](uint32_t st, int i) { return frag((x_at + st) ^ (32u * i), PK); };
#pragma unroll
    for (int j = 0; j < TN; j++) d0[j] = read_d(0, j);
#pragma unroll
    for (int i = 0; i < AHEAD; i++) f[i] = read_x(0, i);
    // Stage s.  `rows` holds those of s + 2, which go into the third buffer piece by
    // piece between the multiplications, and takes those of s + 4; the first fragments
    // of s + 1, in LDS since the last barrier, are read behind the last of s.
    auto stage = [&](int s, Rows& rows, bf16x8_t (&d)[TN], bf16x8_t (&dn)[TN]) {
      const From o = from(s + 4);
#pragma unroll
      for (int i = 0; i < TK; i++) {
        f[(i + AHEAD) % RING] = i + AHEAD < TK ? read_x(b0, (i + AHEAD) % TK) : read_x(b1, (i + AHEAD) % TK);
        if (i >= TK - 2) {
#pragma unroll
          for (int j = 0; j < TN / 2; j++) dn[TN / 2 * (i - TK + 2) + j] = read_d(b1, TN / 2 * (i - TK + 2) + j);
        }
        constexpr int P = TK - 2, PIECES = NX + ND;  // pieces, in the steps before the last two
#pragma unroll
        for (int c = 0; c < PIECES; c++) {
          if (c * P / PIECES != i) continue;
          if (c < NX) {
            store_x(rows, b2, c % NX);
            load_x(o, rows, c % NX);
          } else {
            store_d(rows, b2, c - NX);
            load_d(o, rows, c - NX);
          }
        }
#pragma unroll
        for (int j = 0; j < TN; j++)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[i % RING], d[j], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      // all LDS accesses but the reads of the last two steps (of the next stage) are done
      stage_barrier<2 * (2 + TN)>();
      const uint32_t t = b0;
      b0 = b1;
      b1 = b2;
      b2 = t;
    };
    int s = 0;
#pragma unroll 1
    for (; s + 1 < stages; s += 2) {
      stage(s, x0, d0, d1);
      stage(s + 1, x1, d1, d0);
    }
    if (s < stages) stage(s, x0, d0, d1);
  }

  // the groups' sums: the upper half hands its own to the lower one, until the first
  // group has all of them (every wavefront is past its reads of the buffers)
#pragma unroll
  for (int half = MG / 2; half >= 1; half /= 2) {
    f32x4_t* to = reinterpret_cast<f32x4_t*>(smem_all);
    const int at = ((mg & (half - 1)) * 4 + wave) * TN * TK * 64 + lane;
    __syncthreads();
    if (mg >= half && mg < 2 * half) {
#pragma unroll
      for (int i = 0; i < TN * TK; i++) to[at + 64 * i] = acc[i / TN][i % TN];
    }
    __syncthreads();
    if (mg < half) {
#pragma unroll
      for (int i = 0; i < TN * TK; i++) acc[i / TN][i % TN] += to[at + 64 * i];
    }
  }
  if constexpr (MG > 1) {
    __syncthreads();  // (what was handed over has been read)
    if (mg > 0) return;
  }

  // element i of lane (r, q): k = 4 q + i, n = r.  Out through a part of LDS of the
  // wavefront's own (what others may still read of the buffers is of no stage), 16 rows
  // at a time, their chunks of 16 bytes swizzled by the row, in lines of 64 TK bytes.
  constexpr int C = 4 * TK, LINES = 64 / C;  // chunks of a row; rows a store
  uint8_t* out = smem_all + wave * 16 * 16 * C;
  const int c = lane % C, k = k0 + 16 * TK * wk + 4 * c;
  float* dw = a.dw + (int64_t)e * a.N * a.K + k;
#pragma unroll
  for (int j = 0; j < TN; j++) {
#pragma unroll
    for (int i = 0; i < TK; i++)
      *reinterpret_cast<f32x4_t*>(out + 16 * (C * r + ((4 * i + q) ^ (r & 7)))) = acc[i][j];
    wave_fence();
    f32x4_t v[16 / LINES];
#pragma unroll
    for (int i = 0; i < 16 / LINES; i++) {
      const int row = LINES * i + lane / C;
      v[i] = *reinterpret_cast<const f32x4_t*>(out + 16 * (C * row + (c ^ (row & 7))));
    }
#pragma unroll
    for (int i = 0; i < 16 / LINES; i++) {
      const int n = n0 + 16 * (TN * wn + j) + LINES * i + lane / C;
      if (n >= a.N || k >= a.K) continue;
      f32x4_t* p = reinterpret_cast<f32x4_t*>(dw + (int64_t)n * a.K);
      *p = a.accumulate ? *p + v[i] : v[i];
    }
    wave_fence();
  }
}

template <typename S>
hipError_t launch(const WgradParams& a, hipStream_t s) {
  const int tn = (a.N + S::BN - 1) / S::BN, tk = (a.K + S::BK - 1) / S::BK;
  int cus = 0;
  const hipError_t err = allow_lds<wgrad_kernel<S>>(S::LDS, &cus);
  if (err != hipSuccess) return err;
  const int64_t grid = ((int64_t)tn * tk + 7) / 8 * 8 * a.experts;
  wgrad_kernel<S><<<(unsigned)grid, 256 * S::MG, S::LDS, s>>>(a, tn, tk);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_wgrad_fp8(const WgradParams& a, hipStream_t s) {
  constexpr int64_t CUS = 256;
  auto tiles = [&](int n, int k) { return (int64_t)a.experts * ((a.N + n - 1) / n) * ((a.K + k - 1) / k); };
  // 128 x 256 tiles while there is one for each CU (4096 x 4096 x 4096, 512 of them:
  // 147 us against 183 in 128 x 128 tiles; 2048 x 4096 x 2048, 256: 48 against 51; 32
  // experts of 512 rows, 4096 x 1536: 347 against 555)
  if (tiles(128, 256) >= CUS) return launch<Tile<4, 8, 1>>(a, s);
  // 128 x 128, rows in two, while that is one for every other CU (1237 x 2056 x 1568,
  // 221 of them: 22.7 us, in 64 x 128 tiles 25.0, in 128 x 256 34; 4096 x 2048 x 2048:
  // 48, 55, 82)
  if (tiles(128, 128) > CUS / 2) return launch<Tile<4, 4, 2>>(a, s);
  // 64 x 128 below, rows in two, or in four where they are many (16384 x 1024 x 1024:
  // 121 us in two, 99 in four; 512 x 1024 x 1024: 9.1, 9.9; 64 x 2048 x 2048: 8.8, 14.5)
  if (a.M / a.experts < 1024) return launch<Tile<2, 4, 2>>(a, s);
  return launch<Tile<2, 4, 4>>(a, s);
}

}  // namespace moe
