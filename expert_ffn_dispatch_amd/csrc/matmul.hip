// What the three forms share: the choice of contraction slices, the sum of
// their partial results, and the activation's gradient with the bias gradient.
#include "matmul.h"

namespace moe {

namespace {

// out = epilogue(sum over slices, in slice order).  parts [E][splits][m][n]
// fp32; one thread per eight columns.  Bound by HBM / L2 reads of the parts.
template <bool F16>
__global__ __launch_bounds__(256) void matmul_join_kernel(MatmulArgs p, const float* parts, int splits) {
  const int chunks = ceil_div(p.n, 8);
  const long long total = (long long)p.E * p.m * chunks;
  const int64_t one = (int64_t)p.m * p.n;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const int64_t row = i / chunks;               // over all groups
    const int col = (int)(i - row * chunks) * 8;
    const int64_t e = row / p.m;
    const float* src = parts + e * splits * one + (row - e * p.m) * p.n + col;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s, src += one) {
      if ((p.n & 7) == 0) {
        const f32x4_t a = *reinterpret_cast<const f32x4_t*>(src), b = *reinterpret_cast<const f32x4_t*>(src + 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[q] += a[q];
          v[4 + q] += b[q];
        }
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (col + q < p.n) v[q] += src[q];
      }
    }
    float bias[8];
    mm_bias8<F16>(p, col, bias);
    mm_finish8<F16>(p, v, bias, row, col, 0);
  }
}

// act'(z) in fp32.
__device__ __forceinline__ float act_grad(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.f ? 1.f : 0.f;
    case kActGelu:
      return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * 0.39894228040143268f * __expf(-0.5f * z * z);
    case kActGeluTanh: {
      // z s(2u), s the logistic function: s + z s (1 - s) 2u'; 1 - s = s(-2u)
      const float u2 = 1.5957691216057307f * (z + 0.044715f * z * z * z);
      const float s = 1.f / (1.f + __expf(-u2)), c = 1.f / (1.f + __expf(u2));
      return s + z * s * c * 1.5957691216057307f * (1.f + 0.134145f * z * z);
    }
    case kActSilu: {
      const float s = 1.f / (1.f + __expf(-z)), c = 1.f / (1.f + __expf(z));
      return s + z * s * c;
    }
    default: return 1.f;
  }
}

// A block covers 512 columns (two per lane of each wave... 64 lanes x 8) and
// a run of rows: wave w takes rows w, w + 4, ... of the run; lanes hold eight
// columns each and their fp32 sums, which the four waves add up in LDS.
// Partial sums [row runs][n]; dbias_join adds the runs in order.
template <bool F16>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs p, float* part, int run, int vec) {
  __shared__ float s_sum[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 512 + lane * 8;
  const int r0 = blockIdx.y * run, r1 = min(r0 + run, p.rows);
  const int left = p.n - col;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int r = r0 + wave; r < r1; r += 4) {
    float d[8], z[8];
    const uint16_t* dp = p.dy + (int64_t)r * p.ldd + col;
    const uint16_t* zp = p.act != kActNone ? p.pre + (int64_t)r * p.ldp + col : nullptr;
    if (vec && left >= 8) {
      mm_unpack8<F16>(*reinterpret_cast<const u32x4_t*>(dp), d);
      if (zp) mm_unpack8<F16>(*reinterpret_cast<const u32x4_t*>(zp), z);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        d[q] = q < left ? mm_load1<F16>(dp[q]) : 0.f;
        z[q] = (zp && q < left) ? mm_load1<F16>(zp[q]) : 0.f;
      }
    }
    if (zp) {
#pragma unroll
      for (int q = 0; q < 8; ++q) d[q] *= act_grad(z[q], p.act);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[q] += d[q];
    if (p.g) {
      uint16_t* gp = p.g + (int64_t)r * p.n + col;
      if (vec && left >= 8) {
        *reinterpret_cast<u32x4_t*>(gp) = u32x4_t{mm_pack2<F16>(d[0], d[1]), mm_pack2<F16>(d[2], d[3]),
                                                  mm_pack2<F16>(d[4], d[5]), mm_pack2<F16>(d[6], d[7])};
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < left) gp[q] = mm_store1<F16>(d[q]);
      }
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
__global__ __launch_bounds__(256) void dbias_join_kernel(ActGradArgs p, const float* part, int runs) {
  // 64 columns per block; each wave sums every fourth run, LDS joins the four
  __shared__ float s_sum[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < p.n)
    for (int r = wave; r < runs; r += 4) s += part[(int64_t)r * p.n + c];
  s_sum[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < p.n) {
    const float v = (s_sum[0][lane] + s_sum[1][lane]) + (s_sum[2][lane] + s_sum[3][lane]);
    if (p.dbias_f32) static_cast<float*>(p.dbias)[c] = v;
    else static_cast<uint16_t*>(p.dbias)[c] = mm_store1<F16>(v);
  }
}

// Rows per run: about 1024 blocks over the card, at least 16 rows each.
int act_grad_run(int64_t rows, int64_t n) {
  const int64_t col_blocks = (n + 511) / 512;
  const int64_t want = (1024 + col_blocks - 1) / col_blocks;
  int64_t run = (rows + want - 1) / want;
  return (int)(run < 16 ? 16 : run);
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
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const int vec = al(a.dy) && a.ldd % 8 == 0 && (a.act == kActNone || (al(a.pre) && a.ldp % 8 == 0)) &&
                  (a.g == nullptr || (al(a.g) && a.n % 8 == 0));
  if (runs > 0) {
    const dim3 grid((unsigned)ceil_div(a.n, 512), (unsigned)runs);
    if (a.f16) hipLaunchKernelGGL(act_grad_kernel<true>, grid, dim3(256), 0, st, a, part, run, vec);
    else hipLaunchKernelGGL(act_grad_kernel<false>, grid, dim3(256), 0, st, a, part, run, vec);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (a.dbias) {
    const dim3 grid((unsigned)ceil_div(a.n, 64));
    if (a.f16) hipLaunchKernelGGL(dbias_join_kernel<true>, grid, dim3(256), 0, st, a, part, runs);
    else hipLaunchKernelGGL(dbias_join_kernel<false>, grid, dim3(256), 0, st, a, part, runs);
    return hipGetLastError();
  }
  return hipSuccess;
}

int matmul_splits(MatmulForm f, int E, bool ragged, int64_t rows, int64_t m, int64_t n, int64_t k) {
  if (ragged && f != kMmWeightGrad) return 1;
  const int64_t groups = f == kMmWeightGrad ? E : 1;
  const int64_t tiles = groups * ((m + 127) / 128) * ((n + 127) / 128);
  const int64_t len = f == kMmWeightGrad ? (rows + E - 1) / E : k;
  const int64_t stages = (len + kMmK - 1) / kMmK;
  // two 128 x 128 blocks fit a CU: slice until about 512 blocks, four stages
  // at least to a slice
  int64_t s = 512 / (tiles > 0 ? tiles : 1);
  if (s > stages / 4) s = stages / 4;
  if (s > 32) s = 32;
  return s < 2 ? 1 : (int)s;
}

size_t matmul_workspace_bytes(MatmulForm f, int E, bool ragged, int64_t rows, int64_t m, int64_t n, int64_t k) {
  const int s = matmul_splits(f, E, ragged, rows, m, n, k);
  if (s == 1) return 0;
  return (size_t)s * (f == kMmWeightGrad ? E : 1) * (size_t)m * (size_t)n * sizeof(float);
}

hipError_t launch_matmul(MatmulForm f, MatmulArgs a, void* ws, hipStream_t st) {
  if (a.m == 0 || (f != kMmWeightGrad && a.rows == 0)) return hipSuccess;
  if (f == kMmForward && matmul_streams(a)) {
    a.splits = 1;
    return launch_matmul_stream(a, st);
  }
  const int64_t s = a.whole ? 1 : matmul_splits(f, a.E, a.offsets != nullptr, a.rows, a.m, a.n, a.k);
  auto launch = [&](const MatmulArgs& q) {
    return f == kMmForward ? launch_matmul_forward(q, st)
           : f == kMmRowGrad ? launch_matmul_row_grad(q, st)
                             : launch_matmul_weight_grad(q, st);
  };
  a.splits = (int)s;
  if (s == 1) return launch(a);
  MatmulArgs part = a;
  part.out = ws;
  part.out_f32 = 1;
  part.ldo = a.n;
  part.out_group = (int64_t)a.m * a.n;
  part.vec = a.n % 4 == 0;
  part.bias = nullptr;
  part.act = kActNone;
  part.residual = nullptr;
  part.pre = nullptr;
  if (hipError_t e = launch(part)) return e;
  if (f != kMmWeightGrad) a.E = 1;
  const long long work = (long long)a.E * a.m * ceil_div(a.n, 8);
  const long long blocks = (work + 255) / 256;
  const unsigned grid = (unsigned)(blocks < 8192 ? blocks : 8192);
  if (a.f16) hipLaunchKernelGGL(matmul_join_kernel<true>, dim3(grid), dim3(256), 0, st, a, static_cast<const float*>(ws), (int)s);
  else hipLaunchKernelGGL(matmul_join_kernel<false>, dim3(grid), dim3(256), 0, st, a, static_cast<const float*>(ws), (int)s);
  return hipGetLastError();
}

}  // namespace moe
