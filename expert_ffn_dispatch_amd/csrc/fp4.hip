// Products with 4-bit weights: y[r][c] = sum_k x[r][k] W[c][k], W as E2M1 codes
// (two to a byte, the even k in the low half) and one exponent for every 32
// consecutive k, W = code * 2^(exponent - 127).  gfx950 converts two codes and
// their exponent to two 16-bit values in one instruction, exactly, so every
// product is the one of 16-bit weights of these values.
//
// Few rows to a group of weights: fp4_stream_kernel.  A block owns 16 NC
// columns and 16 RB rows; its NW waves take every NW-th 128-wide chunk of the
// contraction and add their sums in LDS, in wave order.  A lane loads 16 bytes
// of codes, 32 consecutive k of one weight row, so that it needs one exponent
// for all of them; they are the operands of four matrix instructions, each
// with 8 of every lane's 32 k.  That is a permutation of the chunk's k, which
// the sums do not mind as long as the rows of x are read in the same one.
// Nothing passes through LDS on the way and no wave waits for another.
// Bound by the weights' 17/32 byte.
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
__device__ __forceinline__ float exponent(uint32_t e) { return __uint_as_float(e << 23); }

__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

// D chunks of codes and one of x are on their way while one is multiplied.
template <bool F16, int RB, int NC, int NW, int D, bool GATED>
__global__ __launch_bounds__(64 * NW) void fp4_stream_kernel(Fp4Args a) {
  constexpr int kOut = GATED ? 8 * NC : 16 * NC;  // output columns of a block
  static_assert(!GATED || NC % 2 == 0, "pairs of columns");
  __shared__ __align__(16) float s_part[NW][RB * NC * 256];
  const MatmulArgs& p = a.mm;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, fg = lane >> 4;
  const int cpitch = p.k / 2, epitch = p.k / 32;
  MmTile t;
  for (int step = 0; mm_find_tile<false, 16 * RB, kOut>(p, lane, step, t); ++step) {
    mm_scalar(t);
    const int chunks = ceil_div(p.k, kChunk);
    const int n = wave < chunks ? (chunks - wave + NW - 1) / NW : 0;   // this wave's
    const int64_t row = (int64_t)t.e * p.n + t.col0;
    const __amdgpu_buffer_rsrc_t cr = mm_rsrc(a.codes[0] + row * cpitch), er = mm_rsrc(a.exps[0] + row * epitch);
    const __amdgpu_buffer_rsrc_t cr2 = GATED ? mm_rsrc(a.codes[1] + row * cpitch) : cr;
    const __amdgpu_buffer_rsrc_t er2 = GATED ? mm_rsrc(a.exps[1] + row * epitch) : er;
    const __amdgpu_buffer_rsrc_t xr = mm_rsrc(p.a + (int64_t)(t.g0 + t.row0) * p.lda);
    uint32_t co[NC], eo[NC], xo[RB];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int r = (GATED ? 16 * (j >> 1) : 16 * j) + fr;             // of its matrix
      const bool in = t.col0 + r < p.n;
      co[j] = in ? (uint32_t)(r * cpitch + fg * 16) : kMmOut;
      eo[j] = in ? (uint32_t)(r * epitch + fg) : kMmOut;
    }
#pragma unroll
    for (int b = 0; b < RB; ++b)
      xo[b] = 16 * b + fr < t.nrows ? (uint32_t)(16 * b + fr) * (uint32_t)(2 * p.lda) + (uint32_t)(fg * 64) : kMmOut;
    f32x4_t acc[NC][RB];
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int b = 0; b < RB; ++b) acc[j][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // chunk c of this wave starts at k = 128 (wave + NW c); past the end lanes
    // take zeros
    u32x4_t w[D][NC];
    uint32_t e[D][NC];
    auto load_w = [&](u32x4_t (&cw)[NC], uint32_t (&ce)[NC], int c) __attribute__((always_inline)) {
      const int at = wave + NW * c;
      const bool in = at * kChunk + 32 * fg < p.k;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const bool second = GATED && (j & 1);
        cw[j] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(second ? cr2 : cr, in ? co[j] : kMmOut,
                                                                                  (uint32_t)at * (kChunk / 2), 0));
        ce[j] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(second ? er2 : er, in ? eo[j] : kMmOut,
                                                              (uint32_t)at * (kChunk / 32), 0);
      }
    };
    auto load_x = [&](u32x4_t (&x)[RB][4], int c) __attribute__((always_inline)) {
      const int at = wave + NW * c;
      const bool in = at * kChunk + 32 * fg < p.k;
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int s = 0; s < 4; ++s) x[b][s] = load16(xr, in ? xo[b] + 16 * s : kMmOut, (uint32_t)at * (2 * kChunk));
    };
    auto multiply = [&](const u32x4_t (&cw)[NC], const uint32_t (&ce)[NC], const u32x4_t (&x)[RB][4]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const float sc = exponent(ce[j]);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const u32x4_t f = widen8<F16>(cw[j][s], sc);
#pragma unroll
          for (int b = 0; b < RB; ++b) acc[j][b] = mm_mfma<F16>(f, x[b][s], acc[j][b]);
        }
      }
    };
    u32x4_t xa[2][RB][4];
#pragma unroll
    for (int d = 0; d < D; ++d) load_w(w[d], e[d], d);
    load_x(xa[0], 0);
    static_assert(D % 2 == 0, "the rows' two buffers alternate with the codes'");
    for (int c = 0; c < n; c += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (c + d >= n) break;
        load_x(xa[(d + 1) & 1], c + d + 1);
        multiply(w[d], e[d], xa[d & 1]);
        load_w(w[d], e[d], c + d + D);
      }
    }
    // partial sums [wave][16 RB rows][16 NC columns]; column c of row r at
    // c ^ 4 (r & 3), for the banks
    float* part = s_part[wave];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int j = 0; j < NC; ++j)
        *reinterpret_cast<f32x4_t*>(part + (16 * b + fr) * 16 * NC + 16 * j + 4 * (fg ^ (fr & 3))) = acc[j][b];
    __syncthreads();
    for (int i = tid; i < RB * 16 * kOut; i += 64 * NW) {
      const int row = i / kOut, c = i % kOut, col = t.col0 + c;
      const int at = row * 16 * NC + (GATED ? 32 * (c >> 4) + ((c & 15) ^ (4 * (row & 3))) : c ^ (4 * (row & 3)));
      float v = 0.f, u = 0.f;
#pragma unroll
      for (int q = 0; q < NW; ++q) {
        v += s_part[q][at];
        if constexpr (GATED) u += s_part[q][at + 16];
      }
      if (row < t.nrows && col < p.n) {
        if constexpr (GATED) gate1<F16>(p, v, u, (int64_t)t.g0 + t.row0 + row, col);
        else finish1<F16>(p, v, (int64_t)t.g0 + t.row0 + row, col);
      }
    }
    __syncthreads();                              // the sums are read before they are written again
  }
}

template <bool F16, int RB, int NC, int NW, int D, bool GATED>
hipError_t stream_go(const Fp4Args& a, hipStream_t st) {
  const MatmulArgs& p = a.mm;
  const long long groups = p.offsets != nullptr ? (p.E < p.rows ? p.E : p.rows) : 1;
  const long long BM = 16 * RB, cols = ceil_div(p.n, GATED ? 8 * NC : 16 * NC);
  long long grid = ((p.rows + BM - 1) / BM + (p.offsets != nullptr ? groups : 0)) * cols;
  grid = (grid + 7) / 8 * 8;
  if (grid > (1 << 20)) grid = 1 << 20;
  hipLaunchKernelGGL((fp4_stream_kernel<F16, RB, NC, NW, D, GATED>), dim3((unsigned)grid), dim3(64 * NW), 0, st, a);
  return hipGetLastError();
}
template <bool F16, bool GATED>
hipError_t stream_rows(const Fp4Args& a, hipStream_t st) {
  const MatmulArgs& p = a.mm;
  const long long mean = p.offsets != nullptr ? (p.rows + p.E - 1) / p.E : p.rows;
  if (mean <= 16) return stream_go<F16, 1, 2, 8, 2, GATED>(a, st);
  if (mean <= 32) return stream_go<F16, 2, 4, 4, 2, GATED>(a, st);
  return stream_go<F16, 4, 4, 4, 2, GATED>(a, st);
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

// Whether the weights are better widened first: a pass of 0.53 + 2 bytes and
// the product's reading of 2 instead of 0.53.
bool widens(const MatmulArgs& p) {
  const long long mean = p.offsets != nullptr ? (p.rows + p.E - 1) / p.E : p.rows;
  return mean > 64;
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
