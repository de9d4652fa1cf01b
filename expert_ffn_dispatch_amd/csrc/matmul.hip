// What the three forms share: the choice of contraction slices, the sum of
// their partial results, and the activation's gradient with the bias gradient.
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
  mm_finish8<F16, !WG>(p, v, bias, (int64_t)t.row0 + row, col, WG ? (int64_t)t.e * p.out_group : 0);
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

// out[r] = in[r], widened to `pitch` with zeros; a thread moves eight columns.
// With groups (offsets [E+1], as mm_bounds clamps them) only the rows from the
// first group's first to the last group's last: the others belong to no
// product, and are neither read nor worth the time.
__global__ __launch_bounds__(256) void pack_kernel(const uint16_t* in, int64_t ld, int64_t rows, int width,
                                                   uint16_t* out, int pitch, const int32_t* offsets, int E) {
  const int chunks = pitch / 8;
  int64_t first = 0, end = rows;
  if (offsets != nullptr) {
    // every wave looks through the offsets itself (at most five a lane); where
    // they decrease the groups' rows still lie between the least and the greatest
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
  for (int64_t i = first * chunks + (int64_t)blockIdx.x * 256 + threadIdx.x; i < end * chunks;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / chunks;
    const int c = (int)(i - r * chunks) * 8;
    *reinterpret_cast<u32x4_t*>(out + r * pitch + c) = load8(in + r * ld + c, width - c);
  }
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
  size_t bytes_a, bytes_b;
};
size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
Packing packing(MatmulForm f, const MatmulArgs& q) {
  Packing k{};
  k.wa = f == kMmWeightGrad ? q.m : q.k;
  k.wb = f == kMmForward ? q.k : q.n;
  k.ra = q.rows;
  k.rb = f == kMmForward ? q.n : f == kMmRowGrad ? q.k : q.rows;
  if (q.whole || (f != kMmWeightGrad && q.offsets != nullptr)) return k;
  const bool a = !(q.lda % 8 == 0 && (q.a_padded || k.wa % 8 == 0)), b = !(q.ldb % 8 == 0 && k.wb % 8 == 0);
  if (!a && !b) return k;
  auto pitch = [](int w) { return w >= 512 ? (w + 63) / 64 * 64 : (w + 7) / 8 * 8; };
  k.pa = pitch(k.wa);
  k.pb = pitch(k.wb);
  const size_t na = (size_t)k.ra * k.pa * 2, nb = (size_t)k.rb * k.pb * 2;
  const int64_t len = f == kMmWeightGrad ? q.rows / q.E : q.k, stages = len / kMmK;
  const double flops = 2.0 * q.rows * (f == kMmForward ? (double)q.n * q.k : f == kMmRowGrad ? (double)q.k * q.n : (double)q.m * q.n);
  const double gain = flops * 1.2e-9 + (stages < 16 ? stages : 16);
  const double cost = (a ? na * 2 / 4e6 + 4 : 0) + (b ? nb * 2 / 4e6 + 4 : 0);
  if (gain <= cost) return k;
  k.a = a;
  k.b = b;
  k.bytes_a = a ? up256(na) : 0;
  k.bytes_b = b ? up256(nb) : 0;
  return k;
}
hipError_t launch_pack(const uint16_t* in, int64_t ld, int64_t rows, int width, void* out, int pitch,
                       const int32_t* offsets, int E, hipStream_t st) {
  const int64_t blocks = (rows * (pitch / 8) + 255) / 256;
  hipLaunchKernelGGL(pack_kernel, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), 0, st, in, ld, rows,
                     width, static_cast<uint16_t*>(out), pitch, offsets, E);
  return hipGetLastError();
}
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

size_t matmul_workspace_bytes(MatmulForm f, const MatmulArgs& a) {
  if (a.whole || (f != kMmWeightGrad && a.offsets != nullptr)) return 0;
  const Packing k = packing(f, a);
  // the pointers' alignment is not known here: either plan may run
  const size_t x = matmul_plan(f, a.E, a.rows, a.m, a.n, a.k, true, false).bytes;
  const size_t y = matmul_plan(f, a.E, a.rows, a.m, a.n, a.k, false, false).bytes;
  return k.bytes_a + k.bytes_b + up256(x > y ? x : y);
}

hipError_t launch_matmul(MatmulForm f, MatmulArgs a, void* ws, hipStream_t st) {
  if (a.m == 0 || (f != kMmWeightGrad && a.rows == 0)) return hipSuccess;
  const Packing k = packing(f, a);
  const bool a16 = al16(a.a) && a.lda % 8 == 0 && (a.a_padded || k.wa % 8 == 0);
  const bool b16 = al16(a.b) && a.ldb % 8 == 0 && k.wb % 8 == 0;
  a.aligned = (a16 || k.a) && (b16 || k.b);
  char* w = static_cast<char*>(ws);
  if (a.aligned && a.rows > 0) {
    if (k.a) {
      if (hipError_t e = launch_pack(a.a, a.lda, k.ra, k.wa, w, k.pa, a.offsets, a.E, st)) return e;
      a.a = reinterpret_cast<const uint16_t*>(w);
      a.lda = k.pa;
    }
    if (k.b) {
      if (hipError_t e = launch_pack(a.b, a.ldb, k.rb, k.wb, w + k.bytes_a, k.pb, a.offsets, a.E, st)) return e;
      a.b = reinterpret_cast<const uint16_t*>(w + k.bytes_a);
      a.ldb = k.pb;
    }
  }
  a.parts = reinterpret_cast<float*>(w + k.bytes_a + k.bytes_b);
  if (f == kMmForward && matmul_streams(a)) return launch_matmul_stream(a, st);
  if (f != kMmWeightGrad && a.offsets != nullptr) {
    // ragged: 256 x 256 tiles where the mean group would fill the card with
    // them, else 128 x 128
    const int64_t mean = (a.rows + a.E - 1) / a.E;
    a.big = mean > 128 && a.n > 128 && a.E * ((mean + 255) / 256) * ((a.n + 255) / 256) >= 192;
    a.tail = 0;
    a.splits = 1;
  } else {
    const Plan plan = matmul_plan(f, a.E, a.rows, a.m, a.n, a.k, a.aligned != 0, a.whole != 0);
    a.big = plan.big;
    a.tail = plan.tail;
    a.splits = plan.splits;
  }
  if (hipError_t e = f == kMmForward ? launch_matmul_forward(a, st)
                     : f == kMmRowGrad ? launch_matmul_row_grad(a, st)
                                       : launch_matmul_weight_grad(a, st))
    return e;
  if (a.tail == 0) return hipSuccess;
  if (f == kMmWeightGrad) return a.big ? launch_join<true, 256>(a, st) : launch_join<true, 128>(a, st);
  return a.big ? launch_join<false, 256>(a, st) : launch_join<false, 128>(a, st);
}

}  // namespace moe
