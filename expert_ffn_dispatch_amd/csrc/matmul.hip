// What the three forms share: the choice of contraction slices, the sum of
// their partial results, and the gradients of the activation (with the bias
// gradient) and of the gated projections' activation and product.
#include <algorithm>

#include "matmul.h"

namespace moe {

namespace {

// out = epilogue(sum over the slices, in order) of the tiles that were cut;
// parts [tail][splits][B][B] fp32.  A block takes 2048 values of a tile, a
// thread eight columns of a row.  Bound by reading the parts, from L2 mostly.
template <bool F16, bool WG, int B>
__global__ __launch_bounds__(256) void matmul_join_kernel(MatmulArgs p) {
  constexpr int kPer = B * B / 2048;
  const int j = blockIdx.x / kPer;
  MmTile t;
  const int64_t tiles = (int64_t)ceil_div(p.m, B) * ceil_div(p.n, B) * (WG ? p.E : 1);
  mm_plain_tile<WG, B, B>(p, (int)(tiles - p.tail) + j, t);
  const int at = (blockIdx.x - j * kPer) * 2048 + threadIdx.x * 8;
  const int row = at / B, col = t.col0 + at % B;
  if (row >= t.nrows || col >= p.n) return;
  const float* src = p.parts + (int64_t)j * p.splits * (B * B) + at;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s, src += B * B) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t*>(src), b = *reinterpret_cast<const f32x4_t*>(src + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] += a[q];
      v[4 + q] += b[q];
    }
  }
  float bias[8];
  mm_bias8<F16>(p, col, bias);
  int e = t.e;
  if (WG && p.b2_half) {
    if (e & 1) p.out = p.out2;
    e >>= 1;
  }
  mm_finish8<F16, !WG>(p, v, bias, (int64_t)t.row0 + row, col, WG ? (int64_t)e * p.out_group : 0);
}

// The same for the gated projections, forward: of every 32 columns of a part
// the first sixteen are gates, the others their ups.  A thread takes eight
// columns of a row, a block 1024 values of a tile's output.
template <bool F16, int B>
__global__ __launch_bounds__(128) void matmul_join_gated_kernel(MatmulArgs p) {
  constexpr int kPer = B * B / 2048, kRow = B / 16;
  const int j = blockIdx.x / kPer;
  MmTile t;
  const int64_t tiles = (int64_t)ceil_div(p.m, B) * ceil_div(p.n, B / 2);
  mm_plain_tile<false, B, B / 2>(p, (int)(tiles - p.tail) + j, t);
  const int i = (blockIdx.x - j * kPer) * 128 + threadIdx.x;
  const int row = i / kRow, c = i % kRow, col = t.col0 + 8 * c;
  if (row >= t.nrows || col >= p.n) return;
  const float* src = p.parts + (int64_t)j * p.splits * (B * B) + row * B + 32 * (c >> 1) + 8 * (c & 1);
  float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s, src += B * B) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4_t a = *reinterpret_cast<const f32x4_t*>(src + 4 * h), b = *reinterpret_cast<const f32x4_t*>(src + 16 + 4 * h);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        g[4 * h + q] += a[q];
        u[4 * h + q] += b[q];
      }
    }
  }
  mm_gate8<F16>(p, g, u, (int64_t)t.row0 + row, col);
}

template <int B>
hipError_t launch_join_gated(const MatmulArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.tail * (B * B / 2048)));
  if (a.f16) hipLaunchKernelGGL((matmul_join_gated_kernel<true, B>), grid, dim3(128), 0, st, a);
  else hipLaunchKernelGGL((matmul_join_gated_kernel<false, B>), grid, dim3(128), 0, st, a);
  return hipGetLastError();
}

template <bool WG, int B>
hipError_t launch_join(const MatmulArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.tail * (B * B / 2048)));
  if (a.f16) hipLaunchKernelGGL((matmul_join_kernel<true, WG, B>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((matmul_join_kernel<false, WG, B>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

// s = 1 / (1 + e^-u) and c = 1 - s, from one exponential and one reciprocal.
__device__ __forceinline__ void logistic(float u, float& s, float& c) {
  const float e = __expf(-fabsf(u)), r = __builtin_amdgcn_rcpf(1.f + e), q = e * r;
  s = u < 0.f ? q : r;
  c = u < 0.f ? r : q;
}

// act'(z) in fp32.  Past |z| = 128 every form is 0 or 1 to the last bit, and z
// is cut there: powers of a larger z overflow, and inf times 0 is no number.
// Gelu's distribution and density share an exponential (gradients of 4000 x
// 64 -> 5120: 68 us, relu 64; with the library's error function 11 more).
__device__ __forceinline__ float act_grad(float z, int act) {
  if (fabsf(z) > 128.f) z = copysignf(128.f, z);
  switch (act) {
    case kActRelu: return z > 0.f ? 1.f : 0.f;
    case kActGelu: {
      const float e = __expf(-0.5f * z * z);
      return mm_normal(z, e) + z * 0.39894228040143268f * e;
    }
    case kActGeluTanh: {
      // z s(2u), s the logistic function: s + z s (1 - s) 2u'
      float s, c;
      logistic(1.5957691216057307f * (z + 0.044715f * z * z * z), s, c);
      return s + z * s * c * 1.5957691216057307f * (1.f + 0.134145f * z * z);
    }
    case kActSilu: {
      float s, c;
      logistic(z, s, c);
      return s + z * s * c;
    }
    default: return 1.f;
  }
}

// act(z) and act'(z) of eight values together: one exponential and one
// reciprocal each, and one branch for all, so that they overlap (777 x 2222 with
// gelu (tanh) 11 us with a branch for each value).  z is cut as in act_grad; above
// zero the value is z's own.
__device__ __forceinline__ void act_both(const float (&z)[8], int act, float (&value)[8], float (&slope)[8]) {
#define ACT_EACH                                                               \
  _Pragma("unroll") for (int q = 0; q < 8; ++q) {                              \
    const float w = fabsf(z[q]) > 128.f ? copysignf(128.f, z[q]) : z[q], y = z[q] < 0.f ? w : z[q];
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        slope[q] = z[q] > 0.f ? 1.f : 0.f;
        value[q] = z[q] > 0.f || z[q] != z[q] ? z[q] : 0.f;
      }
      break;
    case kActGelu:
      ACT_EACH
        const float e = __expf(-0.5f * w * w), n = mm_normal(w, e);
        value[q] = y * n;
        slope[q] = n + w * 0.39894228040143268f * e;
      }
      break;
    case kActGeluTanh:
      ACT_EACH
        float s, c;
        logistic(1.5957691216057307f * (w + 0.044715f * w * w * w), s, c);
        value[q] = y * s;
        slope[q] = s + w * s * c * 1.5957691216057307f * (1.f + 0.134145f * w * w);
      }
      break;
    case kActSilu:
      ACT_EACH
        float s, c;
        logistic(w, s, c);
        value[q] = y * s;
        slope[q] = s + w * s * c;
      }
      break;
    default:
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        value[q] = z[q];
        slope[q] = 1.f;
      }
  }
#undef ACT_EACH
}

// A saved product times f.  An infinite one stands for a finite sum past its
// type's range (fp16: 65504): times 0 it is 0, where the formula in numbers that
// hold the sum has 0.
__device__ __forceinline__ float saved_times(float v, float f) {
  return f == 0.f && fabsf(v) == __builtin_inff() ? f : v * f;
}

// The rows of the groups (offsets as mm_bounds clamps them): where they
// decrease they still lie between the least and the greatest.  Every wave looks
// through the offsets itself (at most five a lane).
__device__ __forceinline__ void group_rows(const int32_t* offsets, int E, int64_t rows, int64_t& first, int64_t& end) {
  int lo = (int)rows, hi = 0;
  for (int e = threadIdx.x & 63; e <= E; e += 64) {
    const int o = min(max(offsets[e], 0), (int)rows);
    if (e < E) lo = min(lo, o);
    hi = max(hi, o);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    lo = min(lo, __shfl_xor(lo, d));
    hi = max(hi, __shfl_xor(hi, d));
  }
  first = lo;
  end = hi;
}

// Eight 16-bit values from p on, zeros from the n-th on.
__device__ __forceinline__ u32x4_t load8(const uint16_t* p, int n) {
  u32x4_t v{0, 0, 0, 0};
  if (n >= 8) {
    __builtin_memcpy(&v, p, 16);                  // one load: unaligned access is on
  } else if (n > 0) {
#pragma unroll
    for (int q = 0; q < 7; ++q)
      if (q < n) v[q >> 1] |= (uint32_t)p[q] << (16 * (q & 1));
  }
  return v;
}

// A block covers 512 columns (eight per lane) and a run of rows; its four
// waves take four neighbouring rows each at a time, loaded together.  Lanes
// keep fp32 sums of their columns, which the waves add up in LDS; partial sums
// [runs][n], and dbias_join_kernel adds the runs in order.
// g has a row pitch of ldg; columns n..ldg-1 become zeros.
// g is rounded to the operands' 16 bits, which is what the matrix instruction
// takes (a second term for the rest would double both products); the bias
// gradient sums the unrounded values.
template <bool F16>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs p, float* part, int run) {
  __shared__ float s_sum[4][512];
  constexpr int U = 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 512 + lane * 8;
  const int r0 = blockIdx.y * run, r1 = min(r0 + run, p.rows);
  const int left = p.n - col;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int r = r0 + wave * U; r < r1; r += 4 * U) {
    u32x4_t dv[U], zv[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int n = r + k < r1 ? left : 0;
      dv[k] = load8(p.dy + (int64_t)(r + k) * p.ldd + col, n);
      zv[k] = u32x4_t{0, 0, 0, 0};
      if (p.act != kActNone) zv[k] = load8(p.pre + (int64_t)(r + k) * p.ldp + col, n);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      float d[8], z[8];
      mm_unpack8<F16>(dv[k], d);
      if (p.act != kActNone) {
        mm_unpack8<F16>(zv[k], z);
#pragma unroll
        for (int q = 0; q < 8; ++q) d[q] *= act_grad(z[q], p.act);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) sum[q] += d[q]; // zeros past the ends
      // (the pitch is a multiple of 8, and what lies past the width is zero)
      if (p.g && r + k < r1 && col < p.ldg)
        *reinterpret_cast<u32x4_t*>(p.g + (int64_t)(r + k) * p.ldg + col) =
            u32x4_t{mm_pack2<F16>(d[0], d[1]), mm_pack2<F16>(d[2], d[3]), mm_pack2<F16>(d[4], d[5]),
                    mm_pack2<F16>(d[6], d[7])};
    }
  }
  if (!p.dbias) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) s_sum[wave][q * 64 + lane] = sum[q];
  __syncthreads();
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int c = blockIdx.x * 512 + (i & 63) * 8 + (i >> 6);
    if (c < p.n) part[(int64_t)blockIdx.y * p.n + c] = (s_sum[0][i] + s_sum[1][i]) + (s_sum[2][i] + s_sum[3][i]);
  }
}

template <bool F16>
__global__ __launch_bounds__(1024) void dbias_join_kernel(ActGradArgs p, const float* part, int runs) {
  // 64 columns per block; each wave sums every sixteenth run, LDS joins them
  __shared__ float s_sum[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < p.n) {
#pragma unroll 8
    for (int r = wave; r < runs; r += 16) s += part[(int64_t)r * p.n + c];
  }
  s_sum[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < p.n) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) v += s_sum[w][lane];
    if (p.dbias_f32) static_cast<float*>(p.dbias)[c] = v;
    else static_cast<uint16_t*>(p.dbias)[c] = mm_store1<F16>(v);
  }
}

// Rows first to end of a copy, over the blocks in x; a thread moves eight columns.
__device__ __forceinline__ void pack_rows(const PackJob& j, int64_t first, int64_t end) {
  const int chunks = j.pitch / 8;
  for (int64_t i = first * chunks + (int64_t)blockIdx.x * 256 + threadIdx.x; i < end * chunks;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / chunks;
    const int c = (int)(i - r * chunks) * 8;
    *reinterpret_cast<u32x4_t*>(j.out + r * j.pitch + c) = load8(j.in + r * j.ld + c, j.width - c);
  }
}
int64_t pack_blocks(const PackJob& j) { return (j.rows * (j.pitch / 8) + 255) / 256; }

// dgate = dh up act'(gate) and dup = dh act(gate), rounded to the operands' 16
// bits (as g above: a matrix instruction takes no more, and two operands for the
// rest of the bits would double the products; gradients are 0.0024 from 64 bits
// in bf16 and 0.00029 in fp16, with unrounded factors 0.0017 and 0.00021), side by side: g [rows][2 half], dup from column `half`
// on (whole stages of the contraction), zeros past n.  A thread takes eight
// columns of a row.  Bound by its five passes over rows x n.
// The products' padded copies (x's rows are the groups', weights are copied
// without groups only) are further rows of the grid: each is too short for a
// launch of its own (777 x 1111 x 2222, fp16: the backward pass 71.3 us
// with two launches for them, 62.6 so).
template <bool F16>
__global__ __launch_bounds__(256) void gated_grad_kernel(GatedGradArgs p) {
  const uint32_t chunks = (uint32_t)p.half / 8;
  int64_t first = 0, end = p.rows;
  if (p.offsets != nullptr) group_rows(p.offsets, p.E, p.rows, first, end);
  if (blockIdx.y > 0) {
    const PackJob j = p.jobs[blockIdx.y - 1];
    return pack_rows(j, p.offsets != nullptr ? first : 0, p.offsets != nullptr ? end : j.rows);
  }
  const int64_t last = (end - first) * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < last; i += (int64_t)gridDim.x * 256) {
    const int64_t k = last <= 0xffffffffLL ? (int64_t)((uint32_t)i / chunks) : i / chunks;
    const int64_t r = first + k;
    const int c = (int)(i - k * chunks) * 8, n = p.n - c;
    const u32x4_t dv = load8(p.dh + r * p.ldd + c, n), zv = load8(p.gate + r * p.ldg + c, n),
                  uv = load8(p.up + r * p.ldu + c, n);
    float d[8], z[8], u[8], value[8], slope[8];
    mm_unpack8<F16>(dv, d);
    mm_unpack8<F16>(zv, z);
    mm_unpack8<F16>(uv, u);
    act_both(z, p.act, value, slope);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      u[q] = saved_times(u[q], d[q] * slope[q]);
      z[q] = saved_times(value[q], d[q]);
    }
    uint16_t* o = p.g + r * 2 * p.half + c;
    *reinterpret_cast<u32x4_t*>(o) = u32x4_t{mm_pack2<F16>(u[0], u[1]), mm_pack2<F16>(u[2], u[3]),
                                             mm_pack2<F16>(u[4], u[5]), mm_pack2<F16>(u[6], u[7])};
    *reinterpret_cast<u32x4_t*>(o + p.half) = u32x4_t{mm_pack2<F16>(z[0], z[1]), mm_pack2<F16>(z[2], z[3]),
                                                      mm_pack2<F16>(z[4], z[5]), mm_pack2<F16>(z[6], z[7])};
  }
}

// Rows per run: about 1024 blocks over the card, at least 16 rows each.
int act_grad_run(int64_t rows, int64_t n) {
  const int64_t col_blocks = (n + 511) / 512;
  const int64_t want = (1024 + col_blocks - 1) / col_blocks;
  const int64_t run = (rows + want - 1) / want;
  return (int)((run + 15) / 16 * 16 < 16 ? 16 : (run + 15) / 16 * 16);
}

}  // namespace

size_t act_grad_workspace_bytes(int64_t rows, int64_t n) {
  const int64_t run = act_grad_run(rows, n);
  return (size_t)((rows + run - 1) / run) * (size_t)n * sizeof(float);
}

hipError_t launch_act_grad(const ActGradArgs& a, void* ws, hipStream_t st) {
  const int run = act_grad_run(a.rows, a.n);
  const int runs = ceil_div(a.rows, run);
  float* part = static_cast<float*>(ws);
  if (runs > 0) {
    const dim3 grid((unsigned)ceil_div(a.n, 512), (unsigned)runs);
    if (a.f16) hipLaunchKernelGGL(act_grad_kernel<true>, grid, dim3(256), 0, st, a, part, run);
    else hipLaunchKernelGGL(act_grad_kernel<false>, grid, dim3(256), 0, st, a, part, run);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (a.dbias) {
    const dim3 grid((unsigned)ceil_div(a.n, 64));
    if (a.f16) hipLaunchKernelGGL(dbias_join_kernel<true>, grid, dim3(1024), 0, st, a, part, runs);
    else hipLaunchKernelGGL(dbias_join_kernel<false>, grid, dim3(1024), 0, st, a, part, runs);
    return hipGetLastError();
  }
  return hipSuccess;
}

hipError_t launch_gated_grad(const GatedGradArgs& a, hipStream_t st) {
  int64_t blocks = ((int64_t)a.rows * (a.half / 8) + 255) / 256;
  for (int i = 0; i < a.n_jobs; ++i) blocks = std::max(blocks, pack_blocks(a.jobs[i]));
  const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384), (unsigned)(1 + a.n_jobs));
  if (a.rows <= 0) return hipSuccess;
  if (a.f16) hipLaunchKernelGGL(gated_grad_kernel<true>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(gated_grad_kernel<false>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

namespace {

// How a call without ragged groups is cut into tiles: their size, and into how
// many slices of the contraction the tiles of the last, partial round over the
// card are cut (all tiles, where there is less than a round).
struct Plan {
  int big;
  int tail;
  int splits;
  size_t bytes;
};

// The cheapest of both tile sizes and up to 32 slices by a model of the time
// in us, from measurements: a 64-wide stage takes 1.2 us with a 256 x 256 tile
// per CU and 1.07 us with two 128 x 128 tiles per CU (0.65 with one), a tile
// costs 8 (6) us besides, partial sums pass twice through memory at 4 TB/s and
// joining them costs a launch.
Plan matmul_plan(MatmulForm f, int E, int64_t rows, int64_t m, int64_t n, int64_t k, bool aligned, bool whole) {
  const int64_t len = f == kMmWeightGrad ? (rows + E - 1) / E : k;
  const int64_t stages = len > kMmK ? (len + kMmK - 1) / kMmK : 1;
  Plan best{0, 0, 1, 0};
  double best_us = 0;
  for (int big = 0; big < 2; ++big) {
    if (big && (!aligned || m <= 128 || n <= 128)) continue;
    const int64_t B = big ? 256 : 128, slots = big ? 256 : 512;
    const int64_t tiles = (f == kMmWeightGrad ? E : 1) * ((m + B - 1) / B) * ((n + B - 1) / B);
    const int64_t rest = tiles % slots, rounds = tiles / slots;
    const double fixed = big ? 8 : 6;
    for (int64_t s = 1; s <= 32 && (s == 1 || (s * 4 <= stages && !whole)); ++s) {
      const int64_t items = rest * s, per = (stages + s - 1) / s;
      const double stage = big ? 1.2 : rounds > 0 || items > 256 ? 1.07 : 0.65;
      double us = rounds * (stages * (big ? 1.2 : 1.07) + fixed) + (items + slots - 1) / slots * (per * stage + fixed);
      if (s > 1) us += 5 + (double)items * B * B * 8 / 4e6;
      if ((big == 0 && s == 1) || us < best_us) {
        best_us = us;
        best = Plan{big, s > 1 ? (int)rest : 0, (int)s, s > 1 ? (size_t)(items * B * B) * sizeof(float) : 0};
      }
      if (rest == 0) break;
    }
  }
  return best;
}

}  // namespace

namespace {

// With groups (offsets [E+1], as mm_bounds clamps them) only the rows from the
// first group's first to the last group's last: the others belong to no
// product, and are neither read nor worth the time.
// A grid of two rows does the same for a second matrix.
__global__ __launch_bounds__(256) void pack_kernel(PackJob j, PackJob j2, const int32_t* offsets, int E) {
  int64_t first = 0, end = j.rows;
  if (offsets != nullptr) {
    group_rows(offsets, E, j.rows, first, end);
  }
  pack_rows(blockIdx.y == 1 ? j2 : j, first, end);
}

// Operands that do not take 16-byte loads are copied with padded rows where
// that costs less than the products gain: a product runs at 1000 TFLOP/s with
// such loads and at 440 without, and takes about 1 us less a stage where it is
// bound by latency; a copy passes twice through memory at 4 TB/s and takes a
// launch (2000 x 7041 x 7041 448 us without, and 8 + 30 us for the copies).
struct Packing {
  bool a, b;
  int wa, wb, pa, pb;        // widths, pitches
  int64_t ra, rb;            // rows
  size_t bytes_a, bytes_b;   // bytes_b: of each matrix
  int mats;
};
size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
Packing packing(MatmulForm f, const MatmulArgs& q) {
  Packing k{};
  k.wa = f == kMmWeightGrad ? q.m : q.k;
  k.wb = f == kMmForward ? q.k : q.n;
  k.ra = q.rows;
  k.rb = f == kMmForward ? q.n : f == kMmRowGrad ? q.k : q.rows;
  if (q.whole || (f != kMmWeightGrad && q.offsets != nullptr)) return k;
  const int mats = q.gated && f != kMmWeightGrad ? 2 : 1;   // of the columns' operand
  const int groups = q.b2_half ? q.E / 2 : q.E;
  const bool a = !(q.lda % 8 == 0 && (q.a_padded || k.wa % 8 == 0)), b = !(q.ldb % 8 == 0 && (q.b_padded || k.wb % 8 == 0));
  if (!a && !b) return k;
  auto pitch = [](int w) { return w >= 512 ? (w + 63) / 64 * 64 : (w + 7) / 8 * 8; };
  k.pa = pitch(k.wa);
  k.pb = pitch(k.wb);
  const size_t na = (size_t)k.ra * k.pa * 2, nb = (size_t)k.rb * k.pb * 2;
  const int64_t len = f == kMmWeightGrad ? q.rows / groups : q.k, stages = len / kMmK;
  const double flops = (q.gated ? 4.0 : 2.0) * q.rows * (f == kMmForward ? (double)q.n * q.k : f == kMmRowGrad ? (double)q.k * q.n : (double)q.m * q.n);
  const double gain = flops * 1.2e-9 + (stages < 16 ? stages : 16);
  const double cost = (a ? na * 2 / 4e6 + 4 : 0) + (b ? mats * nb * 2 / 4e6 + 4 : 0);
  if (gain <= cost) return k;
  k.a = a;
  k.b = b;
  k.bytes_a = a ? up256(na) : 0;
  k.bytes_b = b ? up256(nb) : 0;
  k.mats = mats;
  return k;
}
hipError_t launch_pack(const PackJob* jobs, int n, const int32_t* offsets, int E, hipStream_t st) {
  const int64_t blocks = pack_blocks(jobs[0]);
  hipLaunchKernelGGL(pack_kernel, dim3((unsigned)(blocks < 16384 ? blocks : 16384), (unsigned)n), dim3(256), 0, st,
                     jobs[0], jobs[n - 1], offsets, E);
  return hipGetLastError();
}
// b's copies, in their places from `to` on.
int b_jobs(const MatmulArgs& a, const Packing& k, char* to, PackJob* jobs) {
  const uint16_t* in[2] = {a.b, a.b2};
  for (int i = 0; i < k.mats; ++i)
    jobs[i] = PackJob{in[i], to != nullptr ? reinterpret_cast<uint16_t*>(to + i * k.bytes_b) : nullptr, a.ldb, k.rb, k.wb, k.pb};
  return k.mats;
}
void use_b_copies(MatmulArgs& a, const PackJob* jobs, int n) {
  a.b = jobs[0].out;
  if (n == 2) a.b2 = jobs[1].out;
  a.ldb = jobs[0].pitch;
}
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The plan of a call.  Gated: a tile's columns are gates and ups, the rows'
// gradient has both contractions one after the other, and every group of rows
// two weight gradients.
Plan plan_of(MatmulForm f, const MatmulArgs& a, bool aligned) {
  const bool g = a.gated != 0;
  return matmul_plan(f, a.E, (int64_t)a.rows * (a.b2_half ? 2 : 1), a.m, (int64_t)a.n * (g && f == kMmForward ? 2 : 1),
                     g && f == kMmRowGrad ? 2 * (((int64_t)a.k + kMmK - 1) / kMmK * kMmK) : a.k, aligned, a.whole != 0);
}

}  // namespace

size_t matmul_workspace_bytes(MatmulForm f, const MatmulArgs& a) {
  if (a.whole || (f != kMmWeightGrad && a.offsets != nullptr)) return 0;
  const Packing k = packing(f, a);
  // the pointers' alignment is not known here: either plan may run
  const size_t x = plan_of(f, a, true).bytes, y = plan_of(f, a, false).bytes;
  return k.bytes_a + k.mats * k.bytes_b + up256(x > y ? x : y);
}

size_t matmul_pack_jobs(MatmulForm f, MatmulArgs& a, void* to, PackJob* jobs, int& n) {
  const Packing k = packing(f, a);
  if (!k.b || k.a) return 0;                      // (with k.a, launch_matmul copies both)
  const int mats = b_jobs(a, k, static_cast<char*>(to), jobs + n);
  use_b_copies(a, jobs + n, mats);
  a.b_padded = 1;
  n += mats;
  return mats * k.bytes_b;
}

hipError_t launch_matmul(MatmulForm f, MatmulArgs a, void* ws, hipStream_t st) {
  if (a.m == 0 || (f != kMmWeightGrad && a.rows == 0)) return hipSuccess;
  const Packing k = packing(f, a);
  const bool a16 = al16(a.a) && a.lda % 8 == 0 && (a.a_padded || k.wa % 8 == 0);
  const bool b16 = al16(a.b) && (a.b2 == nullptr || al16(a.b2)) && a.ldb % 8 == 0 && (a.b_padded || k.wb % 8 == 0);
  a.aligned = (a16 || k.a) && (b16 || k.b);
  char* w = static_cast<char*>(ws);
  const int groups = a.b2_half ? a.E / 2 : a.E;
  if (a.aligned && a.rows > 0) {
    if (k.a) {
      const PackJob j{a.a, reinterpret_cast<uint16_t*>(w), a.lda, k.ra, k.wa, k.pa};
      if (hipError_t e = launch_pack(&j, 1, a.offsets, groups, st)) return e;
      a.a = j.out;
      a.lda = k.pa;
    }
    if (k.b) {
      PackJob jobs[2];
      const int n = b_jobs(a, k, w + k.bytes_a, jobs);
      if (hipError_t e = launch_pack(jobs, n, a.offsets, groups, st)) return e;
      use_b_copies(a, jobs, n);
    }
  }
  a.parts = reinterpret_cast<float*>(w + k.bytes_a + k.mats * k.bytes_b);
  if (f == kMmForward && matmul_streams(a)) return launch_matmul_stream(a, st);
  if (f != kMmWeightGrad && a.offsets != nullptr) {
    // ragged: 256 x 256 tiles where the mean group would fill the card with
    // them, else 128 x 128
    const int64_t mean = (a.rows + a.E - 1) / a.E, n = (int64_t)a.n * (a.gated && f == kMmForward ? 2 : 1);
    a.big = mean > 128 && n > 128 && a.E * ((mean + 255) / 256) * ((n + 255) / 256) >= 192;
    a.tail = 0;
    a.splits = 1;
  } else {
    const Plan plan = plan_of(f, a, a.aligned != 0);
    a.big = plan.big;
    a.tail = plan.tail;
    a.splits = plan.splits;
  }
  if (hipError_t e = a.gated ? (f == kMmForward   ? launch_matmul_gated_forward(a, st)
                                : f == kMmRowGrad ? launch_matmul_gated_row_grad(a, st)
                                                  : launch_matmul_gated_weight_grad(a, st))
                     : f == kMmForward ? launch_matmul_forward(a, st)
                     : f == kMmRowGrad ? launch_matmul_row_grad(a, st)
                                       : launch_matmul_weight_grad(a, st))
    return e;
  if (a.tail == 0) return hipSuccess;
  if (a.gated && f == kMmForward) return a.big ? launch_join_gated<256>(a, st) : launch_join_gated<128>(a, st);
  if (f == kMmWeightGrad) return a.big ? launch_join<true, 256>(a, st) : launch_join<true, 128>(a, st);
  return a.big ? launch_join<false, 256>(a, st) : launch_join<false, 128>(a, st);
}

}  // namespace moe
