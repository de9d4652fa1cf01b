// Products with 4-bit weights: y[r][c] = sum_k x[r][k] W[c][k], W as E2M1 codes
// (two to a byte, the even k in the low half) and one exponent for every 32
// consecutive k, W = code * 2^(exponent - 127).  gfx950 converts two codes and
// their exponent to two 16-bit values in one instruction, exactly, so every
// product is the one of 16-bit weights of these values.
//
// fp4_stream_kernel: a block owns 16 RB rows and 16 NC WN columns; its WK
// groups of WN waves take every WK-th 128-wide chunk of the contraction and add
// their sums in LDS, in order.  Codes (64 bytes of a row and chunk) and rows of
// x go straight into LDS, each load in the order of memory: four lanes to 64
// bytes, a quarter of the cache's work that loads in the order of the matrix
// instruction's operands cost (one lane to 16 bytes, each of another row: 64
// cache accesses a load, which bounded it: 4096 rows over 128 experts' gated
// projections of 2048 -> 768 158 us with both operands loaded that way, 75 so).
// A lane reads 16 bytes of codes of one weight row back, four lanes' 4 x 4
// words are turned by two swaps of lane rows, and each word is a matrix
// instruction's eight weights.  Exponents come four chunks at a time, spread
// over the same four lanes.  Waves that share rows of x (WN > 1) meet at a
// barrier a chunk; with WN = 1 no wave waits for another.
// Bound by the weights' 17/32 byte for few rows (6144 -> 16384, one row: 12
// us, 4.4 TB/s with the launch), by the conversions and the matrix pipe for
// many (16000 rows over 32 experts of 4096 -> 1536: 244 us, 0.8 PFLOP/s).
#include "matmul.h"

namespace moe {

namespace {

constexpr int kChunk = 128;                       // contraction per step of a wave

// Two values from byte SEL of four code bytes, times 2^(exponent of s).
template <bool F16, int SEL>
__device__ __forceinline__ uint32_t widen2(uint32_t codes, float s) {
  if constexpr (F16) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, SEL));
  } else {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, SEL));
  }
}
template <bool F16>
__device__ __forceinline__ u32x4_t widen8(uint32_t codes, float s) {
  return u32x4_t{widen2<F16, 0>(codes, s), widen2<F16, 1>(codes, s), widen2<F16, 2>(codes, s), widen2<F16, 3>(codes, s)};
}
// Scale from byte s of four exponents.  The conversion takes the exponent field alone.
__device__ __forceinline__ float exponent_of(uint32_t e, int s) { return __uint_as_float(s == 3 ? e >> 1 : e << (23 - 8 * s)); }
__device__ __forceinline__ float exponent(uint32_t e) { return __uint_as_float(e << 23); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int size) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, size, 0x00020000);
}
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

// Four registers by four rows of sixteen lanes, turned: register i of row r
// becomes register r of row i.
__device__ __forceinline__ u32x4_t turn(u32x4_t v) {
#ifdef __HIP_DEVICE_COMPILE__
  auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4_t{(uint32_t)c[0], (uint32_t)c[1], (uint32_t)d[0], (uint32_t)d[1]};
#else
  return v;
#endif
}

// NB buffers of a stage (a chunk for each group): NB - 1 stages, or with WN = 1
// NB, are on their way while one is multiplied.  GATED: columns are pairs,
// sixteen of W_gate and their sixteen of W_up.  XREG: rows of x of any
// alignment, which pass through registers (they wait for every load under way).
// BM: rows of a tile, 16 RB or, for few, four: the matrix instruction's other
// twelve repeat them and are dropped, and x is a quarter of the loads and LDS
// reads (128 experts of 2048 -> 768, 64 rows, gated 22.9 -> 18.9 us).
// (Registers stay below 256.  Above, an instance of 4 x 8 blocks in a wave had the
// address of the groups' offsets parked in the other half of the file inside a
// block for some lanes, and the others read their next tile through what was there
// before.  tests/test_compiled_kernels_cpu.py holds every instance to that.)
template <bool F16, int RB, int NC, int WN, int WK, int NB, bool GATED, bool XREG, int BM>
__global__ __launch_bounds__(64 * WN * WK, 2) void fp4_stream_kernel(Fp4Args a) {
  constexpr int NW = WN * WK;
  constexpr int kCols = 16 * NC * WN;             // columns of a block, pairs counted twice
  constexpr int kOut = GATED ? kCols / 2 : kCols;
  constexpr bool FOUR = BM == 4;                  // every wave of a group makes the one load of x, of the same bytes
  constexpr int AX = FOUR ? 1 : 4 * RB / WN;      // loads of x of a wave and stage
  constexpr int kLoads = NC + (XREG ? 0 : AX);    // of these and of codes that a later stage may leave under way
  constexpr int XB = BM * kChunk, WB = NC * 512, STAGE = WK * XB + NW * WB;      // 16-bit words
  constexpr int PART = NW * RB * NC * 512;
  constexpr int G = NB == 3 ? 3 : 4;              // stages that share loaded exponents
  static_assert(NB == 2 || NB == 3, "buffers");
  static_assert((!GATED || NC % 2 == 0) && (FOUR ? RB == 1 && !XREG : BM == 16 * RB && AX * WN == 4 * RB), "whole pairs and loads");
  __shared__ __align__(16) uint16_t s0[STAGE > PART ? STAGE : PART];
  __shared__ __align__(16) uint16_t s1[STAGE];
  __shared__ __align__(16) uint16_t s2[NB > 2 ? STAGE : 8];
  const MatmulArgs& p = a.mm;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave / WN, wn = wave % WN;
  const int fr = lane & 15, fg = lane >> 4;
  const int cpitch = p.k / 2, epitch = p.k / 32;
  MmTile t;
  for (int step = 0; mm_find_tile<false, BM, kOut>(p, lane, step, t); ++step) {
    mm_scalar(t);
    const int chunks = ceil_div(p.k, kChunk), n = ceil_div(chunks, WK);
    const int64_t row = (int64_t)t.e * p.n + t.col0;
    const uint8_t* w0 = a.codes[0] + row * cpitch;
    const uint8_t* w1 = GATED ? a.codes[1] + row * cpitch : w0;
    const uint16_t* x0 = p.a + (int64_t)(t.g0 + t.row0) * p.lda;
    const __amdgpu_buffer_rsrc_t er = mm_rsrc(a.exps[0] + row * epitch);
    const __amdgpu_buffer_rsrc_t er2 = GATED ? mm_rsrc(a.exps[1] + row * epitch) : er;
    const int x_first = FOUR ? 0 : 4 * wn * AX;     // this wave's rows of x
    uint32_t co[NC], eo[NC], xo[AX];
    const int wpiece = (lane & 3) ^ ((lane >> 4) & 3);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int first = GATED ? 16 * (wn * (NC / 2) + (j >> 1)) : 16 * (wn * NC + j);  // of its matrix
      co[j] = t.col0 + first + (lane >> 2) < p.n ? (uint32_t)((first + (lane >> 2)) * cpitch + wpiece * 16) : kMmOut;
      eo[j] = t.col0 + first + fr < p.n ? (uint32_t)((first + fr) * epitch) : kMmOut;
    }
#pragma unroll
    for (int i = 0; i < AX; ++i) {
      const int r = x_first + 4 * i + fg;
      xo[i] = r < t.nrows ? (uint32_t)r * (uint32_t)(2 * p.lda) + (uint32_t)((fr ^ (r & 15)) * 16) : kMmOut;
    }
    f32x4_t acc[NC][RB];
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int b = 0; b < RB; ++b) acc[j][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto put_x = [&](__amdgpu_buffer_rsrc_t rx, uint32_t off, uint32_t at, uint16_t* to) __attribute__((always_inline)) {
      if constexpr (XREG) *reinterpret_cast<u32x4_t*>(to + lane * 8) = load16(rx, off, at);
      else mm_dma16(rx, off, at, to);
    };
    // stage c of this wave's part of the contraction is chunk wk + WK c
    auto load = [&](uint16_t* buf, int c) __attribute__((always_inline)) {
      const int k0 = (wk + WK * c) * kChunk;
      // past the end: buffers of no bytes, which read as zeros
      const int size = k0 < p.k ? (int)kMmBytes : 0;
      const __amdgpu_buffer_rsrc_t rw = rsrc(w0, size), rw2 = GATED ? rsrc(w1, size) : rw, rx = rsrc(x0, size);
      uint16_t* bw = buf + WK * XB + wave * WB;
      uint16_t* bx = buf + wk * XB + x_first * kChunk;
      if (k0 + kChunk <= p.k || size == 0) {
#pragma unroll
        for (int j = 0; j < NC; ++j) mm_dma16(GATED && (j & 1) ? rw2 : rw, co[j], (uint32_t)k0 / 2, bw + j * 512);
#pragma unroll
        for (int i = 0; i < AX; ++i) put_x(rx, xo[i], (uint32_t)k0 * 2, bx + i * 512);
      } else {
#pragma unroll
        for (int j = 0; j < NC; ++j)
          mm_dma16(GATED && (j & 1) ? rw2 : rw, k0 + wpiece * 32 < p.k ? co[j] : kMmOut, (uint32_t)k0 / 2, bw + j * 512);
#pragma unroll
        for (int i = 0; i < AX; ++i) {
          const int xk = (fr ^ ((x_first + 4 * i + fg) & 15)) * 8;
          put_x(rx, k0 + xk < p.k ? xo[i] : kMmOut, (uint32_t)k0 * 2, bx + i * 512);
        }
      }
    };
    uint32_t er4[NC];
    u32x4_t ex[NC];
    // exponents of four chunks from c on, the fg-th in the lanes of fg (four bytes
    // at any address: buffer loads need no alignment)
    auto load_e = [&](int c) __attribute__((always_inline)) {
      const int at = (wk + WK * (c + fg)) * 4;
      if ((epitch & 3) == 0) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
          er4[j] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(GATED && (j & 1) ? er2 : er, at < epitch ? eo[j] + at : kMmOut, 0, 0);
      } else {
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          er4[j] = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            er4[j] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(GATED && (j & 1) ? er2 : er,
                                                                    at + q < epitch ? eo[j] + at + q : kMmOut, 0, 0) << (8 * q);
        }
      }
    };
    const int xr = FOUR ? fr & 3 : fr;
    u32x4_t x[RB][4], w[NC];
    auto read = [&](const uint16_t* buf) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NC; ++j)
        w[j] = *reinterpret_cast<const u32x4_t*>(buf + WK * XB + wave * WB + j * 512 + fr * 32 + ((fg ^ ((fr >> 2) & 3)) << 3));
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int b = 0; b < RB; ++b)
          x[b][s] = *reinterpret_cast<const u32x4_t*>(buf + wk * XB + (16 * b + xr) * kChunk + (((4 * s + fg) ^ xr) << 3));
    };
    auto multiply = [&](int q) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const u32x4_t k = turn(w[j]);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const u32x4_t f = widen8<F16>(k[s], exponent_of(ex[j][q], s));
#pragma unroll
          for (int b = 0; b < RB; ++b) acc[j][b] = mm_mfma<F16>(f, x[b][s], acc[j][b]);
        }
      }
    };
#define FP4_WAIT(N) __builtin_amdgcn_s_waitcnt(((N) & 15) | (((N) >> 4) << 14) | 0x0F70)
#define FP4_BUF(I) ((I) % NB == 0 ? s0 : (I) % NB == 1 ? s1 : s2)
    load_e(0);
#pragma unroll
    for (int i = 0; i < (WN == 1 ? NB : NB - 1); ++i) load(FP4_BUF(i), i);
    for (int c = 0; c < n; c += G) {
#pragma unroll
      for (int j = 0; j < NC; ++j) ex[j] = turn(u32x4_t{er4[j], er4[j], er4[j], er4[j]});
      load_e(c + G);
#pragma unroll
      for (int d = 0; d < G; ++d) {
        if (c + d >= n) break;
        if constexpr (WN == 1) {
          FP4_WAIT((NB - 1) * kLoads);
          __builtin_amdgcn_sched_barrier(0);
          read(FP4_BUF(d));
          __builtin_amdgcn_s_waitcnt(0xC07F);
          __builtin_amdgcn_sched_barrier(0);
          load(FP4_BUF(d), c + d + NB);
          multiply(d);
        } else {
          FP4_WAIT((NB - 2) * kLoads);
          __builtin_amdgcn_s_waitcnt(0xC07F);
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_sched_barrier(0);
          load(FP4_BUF(d + NB - 1), c + d + NB - 1);
          read(FP4_BUF(d));
          multiply(d);
        }
      }
    }
    FP4_WAIT(0);                                  // loads past the last stage land
    __syncthreads();
    // partial sums [group][16 RB rows][columns of the block]; column c of row r
    // at c ^ 4 (r & 3), for the banks
    float* part = reinterpret_cast<float*>(s0) + wk * (RB * 16 * kCols);
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int j = 0; j < NC; ++j)
        *reinterpret_cast<f32x4_t*>(part + (16 * b + fr) * kCols + 16 * (wn * NC + j) + 4 * (fg ^ (fr & 3))) = acc[j][b];
    __syncthreads();
    // eight columns of a row to a thread
    for (int i = tid; i < BM * (kOut / 8); i += 64 * NW) {
      const int row = i / (kOut / 8), c = i % (kOut / 8), col = t.col0 + 8 * c, sw = 4 * (row & 3);
      if (row >= t.nrows || col >= p.n) continue;
      const int at = GATED ? 32 * (c >> 1) + 8 * (c & 1) : 8 * c;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < WK; ++q) {
        const float* s = reinterpret_cast<const float*>(s0) + (q * RB * 16 + row) * kCols;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4_t f = *reinterpret_cast<const f32x4_t*>(s + ((at + 4 * h) ^ sw));
#pragma unroll
          for (int k = 0; k < 4; ++k) v[4 * h + k] += f[k];
          if constexpr (GATED) {
            const f32x4_t g = *reinterpret_cast<const f32x4_t*>(s + 16 + ((at + 4 * h) ^ sw));
#pragma unroll
            for (int k = 0; k < 4; ++k) u[4 * h + k] += g[k];
          }
        }
      }
      if constexpr (GATED) {
        mm_gate8<F16>(p, v, u, (int64_t)t.g0 + t.row0 + row, col);
      } else {
        float bias[8];
        mm_bias8<F16>(p, col, bias);
        mm_finish8<F16, true>(p, v, bias, (int64_t)t.g0 + t.row0 + row, col, 0);
      }
    }
    __syncthreads();                              // the sums are read before they are written again
  }
#undef FP4_WAIT
#undef FP4_BUF
}

template <bool F16, int RB, int NC, int WN, int WK, int NB, bool GATED, bool XREG = false, int BM = 16 * RB>
hipError_t stream_go(const Fp4Args& a, hipStream_t st) {
  const MatmulArgs& p = a.mm;
  const long long groups = p.offsets != nullptr ? (p.E < p.rows ? p.E : p.rows) : 1;
  const long long cols = ceil_div(p.n, (GATED ? 8 : 16) * NC * WN);
  long long grid = (((long long)p.rows + BM - 1) / BM + (p.offsets != nullptr ? groups : 0)) * cols;
  grid = (grid + 7) / 8 * 8;
  if (grid > (1 << 20)) grid = 1 << 20;
  hipLaunchKernelGGL((fp4_stream_kernel<F16, RB, NC, WN, WK, NB, GATED, XREG, BM>), dim3((unsigned)grid), dim3(64 * WN * WK), 0, st, a);
  return hipGetLastError();
}
int64_t mean_rows(const MatmulArgs& p) {
  return p.offsets != nullptr ? ((int64_t)p.rows + p.E - 1) / p.E : p.rows;
}

// Groups go by their mean rows, us on 128 experts of 2048 -> 768 unless stated.
// Up to two: tiles of four rows.  Up to eight: 16-row tiles of 64 columns (8 rows
// each to 8 experts of 4096 -> 4096 16.9, 20.8 with 32-row tiles).  Up to 28: 32 rows x
// 256 columns, whose eight waves share x, where that leaves a block for most CUs
// (16 each 34.6, 44.0 with 16 x 64, 37.0 with 32 x 128; gated, 23 each 63.3 and 68.9 with 32 x
// 128), else as up to eight, and from 17 to 40 32 x 128 in two parts of the
// contraction (31 each to 8 experts of 4096 -> 4096 27.7, 31.5 with 48 x 128).
// More: 48 x 128 (64 each 56.8, 64.8 with 64 x 128; gated 100 and 106), and gated from 97 on
// 96 x 128 (128 each 154, 163 with 48 x 128).
// Dense: up to sixteen rows take narrow blocks, with eight waves along the
// contraction where that leaves fewer blocks than CUs (8 rows, 4096 x 4096 6.3 us
// with 16 columns, 7.0 with 32; one row, 6144 -> 16384 17 and 12.3).  More rows
// take the first of ever larger blocks, a block's time growing with them, of which
// every CU gets one at most (6784 -> 112, 256 rows 8.2 us with 16 x 16, 14.9 with 32 x 64;
// 8192 -> 2048, 128 rows 12.7 with 32 x 32, 18.2 with 32 x 64; 5120 x 5120: 96 rows 14.1 us with 32 x 64, 15.9 with 48 x 64;
// 128 rows 25.6 and 15.9; 256 rows 24.6 with 48 x 128, 28.2 with 64 x 128; 512 rows 35.6 with 96 x
// 128, 42.1 with 64 x 128 as follows), and else 64 x 128 or 96 x 128 without waves along
// the contraction, two blocks to a CU, by the rounds over the card at 1 : 1.35 (5120 x
// 5120, 900 rows 71.6 us by 64, 60.4 by 96).
template <bool F16, bool GATED>
hipError_t stream_rows(const Fp4Args& a, hipStream_t st) {
  const MatmulArgs& p = a.mm;
  const int64_t rows = mean_rows(p), n = (int64_t)p.n * (GATED ? 2 : 1);
  const bool x16 = (reinterpret_cast<uintptr_t>(p.a) & 15) == 0 && p.lda % 8 == 0;
  if (!x16) {
    if (rows <= 16) return stream_go<F16, 1, 2, 2, 2, 2, GATED, true>(a, st);
    return stream_go<F16, 4, 2, 4, 2, 2, GATED, true>(a, st);
  }
  if (p.offsets != nullptr) {
    if (rows <= 2) return stream_go<F16, 1, 2, 2, 2, 2, GATED, false, 4>(a, st);
    const bool wide = p.E * ((n + 255) / 256) >= 192;
    if (wide && rows > 8 && rows <= 28) return stream_go<F16, 2, 2, 8, 1, 3, GATED>(a, st);
    if (rows <= 16) return stream_go<F16, 1, 2, 2, 2, 2, GATED>(a, st);
    if (!wide && rows <= 40) return stream_go<F16, 2, 2, 4, 2, 2, GATED>(a, st);
    if constexpr (GATED)
      if (rows > 96) return stream_go<F16, 6, 2, 4, 1, 2, GATED>(a, st);
    return stream_go<F16, 3, 2, 4, 1, 2, GATED>(a, st);
  }
  if (rows <= 4) {
    if (n >= 6144) return stream_go<F16, 1, 2, 1, 4, 2, GATED, false, 4>(a, st);
    if constexpr (GATED) return stream_go<F16, 1, 2, 1, 8, 2, GATED, false, 4>(a, st);
    else return stream_go<F16, 1, 1, 1, 8, 2, GATED, false, 4>(a, st);
  }
  if (rows <= 16) {
    if (n >= 6144) return stream_go<F16, 1, 2, 1, 4, 2, GATED>(a, st);
    if constexpr (GATED) return stream_go<F16, 1, 2, 1, 8, 2, GATED>(a, st);
    else return stream_go<F16, 1, 1, 1, 8, 2, GATED>(a, st);
  }
  auto blocks = [&](int64_t bm, int64_t bn) { return (rows + bm - 1) / bm * ((n + bn - 1) / bn); };
  auto fits = [&](int64_t bm, int64_t bn) { return blocks(bm, bn) <= 256; };
  if constexpr (!GATED)
    if (fits(16, 16)) return stream_go<F16, 1, 1, 1, 8, 2, GATED>(a, st);
  if (fits(16, 32)) return stream_go<F16, 1, 2, 1, 4, 2, GATED>(a, st);
  if (fits(32, 32)) return stream_go<F16, 2, 2, 1, 4, 2, GATED>(a, st);
  if (fits(32, 64)) return stream_go<F16, 2, 2, 2, 4, 2, GATED>(a, st);
  if (fits(48, 64)) return stream_go<F16, 3, 2, 2, 4, 2, GATED>(a, st);
  if (fits(64, 64)) return stream_go<F16, 4, 2, 2, 4, 2, GATED>(a, st);
  if (fits(32, 128)) return stream_go<F16, 2, 2, 4, 2, 2, GATED>(a, st);
  if (fits(48, 128)) return stream_go<F16, 3, 2, 4, 2, 2, GATED>(a, st);
  if (fits(64, 128)) return stream_go<F16, 4, 2, 4, 2, 2, GATED>(a, st);
  if (fits(96, 128)) return stream_go<F16, 6, 2, 4, 2, 2, GATED>(a, st);
  if (27 * ((blocks(96, 128) + 511) / 512) < 20 * ((blocks(64, 128) + 511) / 512))
    return stream_go<F16, 6, 2, 4, 1, 2, GATED>(a, st);
  return stream_go<F16, 4, 2, 4, 1, 3, GATED>(a, st);
}

// -------------------------------------------------------------- many rows

// w = the codes' values in 16 bits; a thread widens eight.
template <bool F16>
__global__ __launch_bounds__(256) void widen_kernel(const uint8_t* codes, const uint8_t* exps, uint16_t* w, int64_t pieces) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
    uint32_t c;
    __builtin_memcpy(&c, __builtin_assume_aligned(codes + 4 * i, 4), 4);
    *reinterpret_cast<u32x4_t*>(w + 8 * i) = widen8<F16>(c, exponent(exps[i >> 2]));
  }
}
hipError_t launch_widen(bool f16, const uint8_t* codes, const uint8_t* exps, uint16_t* w, int64_t pieces, hipStream_t st) {
  const int64_t blocks = (pieces + 255) / 256;
  const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
  if (f16) hipLaunchKernelGGL(widen_kernel<true>, grid, dim3(256), 0, st, codes, exps, w, pieces);
  else hipLaunchKernelGGL(widen_kernel<false>, grid, dim3(256), 0, st, codes, exps, w, pieces);
  return hipGetLastError();
}

// Whether the weights are better widened first: 2.53 bytes a weight, products
// at 1.4 PFLOP/s in place of 1.0, and about 12 us of launches and tiles that fill
// the card less well, which many rows or many weights make up for (us without and
// with: 5120 x 5120, 1200 rows 74 and 79, 2048 rows 115 and 99; 2048 x 2048, 2048 rows 23 and
// 28, 4096 rows 42 and 36; 32 experts of 4096 -> 1536, gated, 850 rows each 670 and 692, 1300
// rows 999 and 935).  Rows of x at an odd pitch pass through registers at half the
// rate; the products of 16-bit weights copy them (5120 x 5120: 600 rows 103 us, 1400
// rows widened 85), but not those of groups.
bool widens(const MatmulArgs& p) {
  const int64_t weights = (int64_t)p.E * p.n * p.k * (p.gated ? 2 : 1);
  if (p.lda % 8 == 0) return mean_rows(p) > 900 + 12000000000LL / weights;
  return mean_rows(p) > (p.offsets != nullptr ? 640 : 300) + 6000000000LL / weights;
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
size_t matrix_bytes(const MatmulArgs& p) { return up256((size_t)p.E * p.n * p.k * 2); }

// ------------------------------------------------------------ quantisation

// A thread takes 32 consecutive weights of a row: the least exponent that
// leaves no magnitude above 7 (which rounds to 6, the largest code), codes to
// nearest, ties to the even code.  fp16: exponents at which every code is an
// fp16 number.
template <bool F16>
__global__ __launch_bounds__(256) void quantize_fp4_kernel(const uint16_t* w, int64_t groups, uint8_t* codes, uint8_t* exps) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= groups) return;
  float f[32];
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float g[8];
    mm_unpack8<F16>(*reinterpret_cast<const u32x4_t*>(w + 32 * i + 8 * q), g);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[8 * q + k] = g[k];
      top = max(top, __float_as_uint(g[k]) & 0x7fffffffu);
    }
  }
  const int e = min(max((int)((top + 0x1FFFFFu) >> 23) - 2, F16 ? 104 : 1), F16 ? 140 : 252);
  const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
  u32x4_t out{0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const float a = fabsf(f[k]) * inv;
    const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.f);
    out[k >> 3] |= (c | ((__float_as_uint(f[k]) >> 28) & 8u)) << (4 * (k & 7));
  }
  *reinterpret_cast<u32x4_t*>(codes + 16 * i) = out;
  exps[i] = (uint8_t)e;
}

}  // namespace

hipError_t launch_quantize_fp4(const uint16_t* w, long long rows, int cols, int f16, uint8_t* codes, uint8_t* exps,
                               hipStream_t st) {
  const int64_t groups = rows * (cols / 32);
  const dim3 grid((unsigned)((groups + 255) / 256));
  if (f16) hipLaunchKernelGGL(quantize_fp4_kernel<true>, grid, dim3(256), 0, st, w, groups, codes, exps);
  else hipLaunchKernelGGL(quantize_fp4_kernel<false>, grid, dim3(256), 0, st, w, groups, codes, exps);
  return hipGetLastError();
}

size_t fp4_workspace_bytes(const Fp4Args& a) {
  if (!widens(a.mm)) return 0;
  MatmulArgs p = a.mm;
  p.ldb = p.k;
  return matrix_bytes(p) * (p.gated ? 2 : 1) + matmul_workspace_bytes(kMmForward, p);
}

hipError_t launch_fp4(const Fp4Args& a, void* ws, hipStream_t st) {
  if (a.mm.rows == 0) return hipSuccess;
  if (!widens(a.mm)) {
    if (a.mm.gated) return a.mm.f16 ? stream_rows<true, true>(a, st) : stream_rows<false, true>(a, st);
    return a.mm.f16 ? stream_rows<true, false>(a, st) : stream_rows<false, false>(a, st);
  }
  MatmulArgs p = a.mm;
  char* w = static_cast<char*>(ws);
  const int64_t pieces = (int64_t)p.E * p.n * p.k / 8;
  for (int i = 0; i < (p.gated ? 2 : 1); ++i) {
    uint16_t* to = reinterpret_cast<uint16_t*>(w);
    if (hipError_t e = launch_widen(p.f16 != 0, a.codes[i], a.exps[i], to, pieces, st)) return e;
    (i ? p.b2 : p.b) = to;
    w += matrix_bytes(p);
  }
  p.ldb = p.k;
  p.b_group = (int64_t)p.n * p.k;
  return launch_matmul(kMmForward, p, w, st);
}

}  // namespace moe
