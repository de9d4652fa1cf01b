// Layer norm and its gradient, in fp32 arithmetic over bf16, fp16 or fp32 rows.
//
//   n = (x - mu) rstd,  rstd = (mean((x - mu)^2) + eps)^-1/2,  y = n gamma + beta
//   dx = rstd (g - mean(g) - n mean(g n)),  g = dy gamma
//   dgamma = sum_rows dy n,  dbeta = sum_rows dy
// Root-mean-square form: mu = 0, and dx has no mean(g).
//
// Bound by HBM: the forward pass reads x and writes y, the backward pass reads
// x and dy and writes dx, each once.  A row is held in registers from its one
// read, so the variance is that of the centred values (no difference of large
// sums) at no further read.
#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

template <int TYPE>
struct NormElem;                                  // storage type and conversions
template <>
struct NormElem<kTypeBf16> {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(T v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ T put(float f) { return f32_to_bf16(f); }
};
template <>
struct NormElem<kTypeF16> {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(T v) { return static_cast<float>(__builtin_bit_cast(_Float16, v)); }
  static __device__ __forceinline__ T put(float f) { return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f)); }
};
template <>
struct NormElem<kTypeF32> {
  typedef float T;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float f) { return f; }
};

// tpr threads share a row, and each holds NCH groups of eight values of it.  VEC: group i of thread
// t is columns 8 (i tpr + t) ..+7, moved in 16-byte pieces; otherwise value q
// of group i is column (8 i + q) tpr + t, moved one by one (any width, stride
// and alignment, still contiguous across the lanes).
template <bool VEC>
__device__ __forceinline__ int norm_col(int i, int q, int t, int tpr) {
  return VEC ? 8 * (i * tpr + t) + q : (8 * i + q) * tpr + t;
}

template <class E, bool VEC, int NCH>
__device__ __forceinline__ void norm_load(const typename E::T* p, int cols, int t, int tpr, typename E::T (&v)[NCH][8]) {
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    if constexpr (VEC) {
      const int c = norm_col<VEC>(i, 0, t, tpr);
      constexpr int W = sizeof(typename E::T) * 8 / 16;    // 16-byte pieces
      u32x4_t w[W];
#pragma unroll
      for (int k = 0; k < W; ++k) w[k] = u32x4_t{0, 0, 0, 0};
      if (c < cols) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[k] = reinterpret_cast<const u32x4_t*>(p + c)[k];
      }
      __builtin_memcpy(&v[i][0], &w[0], sizeof(w));
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int c = norm_col<VEC>(i, q, t, tpr);
        v[i][q] = c < cols ? p[c] : typename E::T(0);
      }
    }
  }
}

// Eight values of column group i of a parameter vector, `dflt` where null.
template <class E, bool VEC>
__device__ __forceinline__ void norm_param(const void* base, bool f32, int cols, int i, int t, int tpr, float dflt, float (&f)[8]) {
  if (base == nullptr) {
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = dflt;
    return;
  }
  if (f32) {
    float v[1][8];
    const float* p = static_cast<const float*>(base) + 8 * i * tpr;
    norm_load<NormElem<kTypeF32>, VEC, 1>(p, cols - 8 * i * tpr, t, tpr, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = v[0][q];
  } else {
    typename E::T v[1][8];
    const typename E::T* p = static_cast<const typename E::T*>(base) + 8 * i * tpr;
    norm_load<E, VEC, 1>(p, cols - 8 * i * tpr, t, tpr, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = E::get(v[0][q]);
  }
}

template <class E, bool VEC>
__device__ __forceinline__ void norm_store(typename E::T* p, int cols, int i, int t, int tpr, const float (&f)[8]) {
  typename E::T v[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = E::put(f[q]);
  if constexpr (VEC) {
    const int c = norm_col<VEC>(i, 0, t, tpr);
    constexpr int W = sizeof(typename E::T) * 8 / 16;
    u32x4_t w[W];
    __builtin_memcpy(&w[0], &v[0], sizeof(w));
    if (c < cols) {
#pragma unroll
      for (int k = 0; k < W; ++k) reinterpret_cast<u32x4_t*>(p + c)[k] = w[k];
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int c = norm_col<VEC>(i, q, t, tpr);
      if (c < cols) p[c] = v[q];
    }
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Sum over the TPR threads of a row; red: one float per wave of the block,
// another buffer each time it is called between two barriers of its own.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    const int w0 = wave / NW * NW;
    v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[w0 + w];
  }
  return v;
}

// One row per TPR threads, 256 threads per block.  TPR = 64 (a wave per row,
// no barrier) where there are rows enough to fill the card with waves; 256
// for few or wide rows.
template <class E, bool VEC, int TPR, int NCH>
__global__ __launch_bounds__(256) void norm_forward_kernel(NormArgs p) {
  __shared__ float red[2][4];
  constexpr int tpr = TPR;
  const int t = threadIdx.x % TPR;
  const int row = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  if (TPR == 64 && row >= p.rows) return;         // (TPR = 256: one row per block, always live)
  typename E::T v[NCH][8];
  norm_load<E, VEC, NCH>(static_cast<const typename E::T*>(p.x) + (int64_t)row * p.ldx, p.cols, t, tpr, v);
  const float inv = 1.f / (float)p.cols;
  float mu = 0.f;
  if (!p.rms) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) s += E::get(v[i][q]);
    mu = row_sum<TPR>(s, red[0]) * inv;
  }
  float s2 = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float d = E::get(v[i][q]) - mu;
      s2 += norm_col<VEC>(i, q, t, tpr) < p.cols ? d * d : 0.f;
    }
  const float rstd = 1.f / sqrtf(row_sum<TPR>(s2, red[1]) * inv + p.eps);
  if (t == 0) {
    if (p.mean) p.mean[row] = mu;
    if (p.rstd) p.rstd[row] = rstd;
  }
  typename E::T* out = static_cast<typename E::T*>(p.out) + (int64_t)row * p.ldo;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    if (8 * i * tpr >= p.cols) break;
    float g[8], b[8], y[8];
    norm_param<E, VEC>(p.gamma, p.param_f32, p.cols, i, t, tpr, 1.f, g);
    norm_param<E, VEC>(p.beta, p.param_f32, p.cols, i, t, tpr, 0.f, b);
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] = (E::get(v[i][q]) - mu) * rstd * g[q] + b[q];
    norm_store<E, VEC>(out + 8 * i * tpr, p.cols - 8 * i * tpr, 0, t, tpr, y);
  }
}

// Backward: blocks of `gr` groups of tpr threads (1024 threads or a little
// less), each group walking rows group, group + (all groups), ...; a thread
// keeps the fp32 sums of dgamma and dbeta for its columns over all its rows,
// the block adds its groups' sums in LDS at the end and writes one partial
// row, and norm_join_kernel adds the blocks' partials in order (no atomics:
// the result does not depend on the schedule).  At most 16 columns per
// thread, so that two rows' values and the sums fit 128 registers at sixteen
// waves per CU.
template <class E, bool VEC, int NCH>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormArgs p, float* part, int tpr, int gr) {
  typedef typename E::T T;
  __shared__ float red[2][2][16];
  __shared__ float s_sum[8 * 1024];
  const int grp = threadIdx.x / tpr, t = threadIdx.x - grp * tpr;
  const int step = gridDim.x * gr;
  const float inv = 1.f / (float)p.cols;
  float dg[NCH][8], db[NCH][8];
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) dg[i][q] = db[i][q] = 0.f;
  int par = 0;
  // every group makes the same number of trips (barriers); a row past the
  // end loads nothing and adds zeros
  for (int base = blockIdx.x * gr; base < p.rows; base += step, par ^= 1) {
    const int row = base + grp;
    const bool live = row < p.rows;
    const int cols = live ? p.cols : 0;
    const int64_t rr = live ? row : 0;
    T x[NCH][8], d[NCH][8];
    norm_load<E, VEC, NCH>(static_cast<const T*>(p.x) + rr * p.ldx, cols, t, tpr, x);
    norm_load<E, VEC, NCH>(static_cast<const T*>(p.dy) + rr * p.ldd, cols, t, tpr, d);
    const float mu = (live && !p.rms) ? p.mean[rr] : 0.f;
    const float rs = live ? p.rstd[rr] : 0.f;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      float g[8];
      norm_param<E, VEC>(p.gamma, p.param_f32, p.cols, i, t, tpr, 1.f, g);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const bool in = norm_col<VEC>(i, q, t, tpr) < cols;
        const float dyv = E::get(d[i][q]), n = (E::get(x[i][q]) - mu) * rs;
        s1 += in ? dyv * g[q] : 0.f;
        s2 += in ? dyv * g[q] * n : 0.f;
        dg[i][q] += in ? dyv * n : 0.f;
        db[i][q] += dyv;                          // zero past the ends
      }
    }
    float m1 = wave_sum(s1), m2 = wave_sum(s2);
    if (tpr > 64) {
      const int wave = threadIdx.x >> 6, nw = tpr >> 6;
      if ((threadIdx.x & 63) == 0) {
        red[par][0][wave] = m1;
        red[par][1][wave] = m2;
      }
      __syncthreads();
      m1 = m2 = 0.f;
      for (int w = grp * nw; w < (grp + 1) * nw; ++w) {
        m1 += red[par][0][w];
        m2 += red[par][1][w];
      }
    }
    m1 = p.rms ? 0.f : m1 * inv;
    m2 *= inv;
    if (p.out != nullptr && live) {
      T* out = static_cast<T*>(p.out) + (int64_t)row * p.ldo;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        float g[8], o[8];
        norm_param<E, VEC>(p.gamma, p.param_f32, p.cols, i, t, tpr, 1.f, g);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float n = (E::get(x[i][q]) - mu) * rs;
          o[q] = rs * (E::get(d[i][q]) * g[q] - m1 - n * m2);
        }
        norm_store<E, VEC>(out + 8 * i * tpr, p.cols - 8 * i * tpr, 0, t, tpr, o);
      }
    }
  }
  if (part == nullptr) return;
  // the block's groups, in order, eight columns per thread at a time
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float s[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] = which ? db[i][q] : dg[i][q];
      __syncthreads();
      if (grp > 0) {
#pragma unroll
        for (int q = 0; q < 8; ++q) s_sum[((grp - 1) * 8 + q) * tpr + t] = s[q];
      }
      __syncthreads();
      if (grp == 0) {
        for (int k = 0; k < gr - 1; ++k)
#pragma unroll
          for (int q = 0; q < 8; ++q) s[q] += s_sum[(k * 8 + q) * tpr + t];
        float* o = part + ((int64_t)blockIdx.x * 2 + which) * p.cols;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int c = norm_col<VEC>(i, q, t, tpr);
          if (c < p.cols) o[c] = s[q];
        }
      }
    }
  }
}

// dgamma (blockIdx.y = 0) and dbeta (1): sums over the partial rows, 64
// columns per block, its sixteen waves every sixteenth row.
template <class E>
__global__ __launch_bounds__(1024) void norm_join_kernel(NormArgs p, const float* part, int parts) {
  __shared__ float s_sum[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane, which = blockIdx.y;
  float s = 0.f;
  if (c < p.cols) {
#pragma unroll 4
    for (int r = wave; r < parts; r += 16) s += part[((int64_t)r * 2 + which) * p.cols + c];
  }
  s_sum[wave][lane] = s;
  __syncthreads();
  void* out = which ? p.dbeta : p.dgamma;
  if (wave == 0 && c < p.cols && out != nullptr) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) v += s_sum[w][lane];
    if (p.param_f32) static_cast<float*>(out)[c] = v;
    else static_cast<typename E::T*>(out)[c] = E::put(v);
  }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool vec_ok(const NormArgs& a) {
  const int64_t w = a.type == kTypeF32 ? 4 : 8;
  return a.cols % 8 == 0 && a.ldx % w == 0 && al16(a.x) && (a.out == nullptr || (a.ldo % w == 0 && al16(a.out))) &&
         (a.dy == nullptr || (a.ldd % w == 0 && al16(a.dy))) && al16(a.gamma) && al16(a.beta);
}

template <class E, bool VEC, int TPR, int NCH>
hipError_t forward_go(const NormArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)ceil_div(a.rows, 256 / TPR);
  hipLaunchKernelGGL((norm_forward_kernel<E, VEC, TPR, NCH>), dim3(grid), dim3(256), 0, st, a);
  return hipGetLastError();
}
template <class E, bool VEC>
hipError_t forward_pick(const NormArgs& a, hipStream_t st) {
  if (a.cols <= 4096 && (a.rows >= 1024 || a.cols <= 512)) {
    if (a.cols <= 512) return forward_go<E, VEC, 64, 1>(a, st);
    if (a.cols <= 1024) return forward_go<E, VEC, 64, 2>(a, st);
    if (a.cols <= 2048) return forward_go<E, VEC, 64, 4>(a, st);
    return forward_go<E, VEC, 64, 8>(a, st);
  }
  if (a.cols <= 2048) return forward_go<E, VEC, 256, 1>(a, st);
  if (a.cols <= 4096) return forward_go<E, VEC, 256, 2>(a, st);
  if (a.cols <= 8192) return forward_go<E, VEC, 256, 4>(a, st);
  return forward_go<E, VEC, 256, 8>(a, st);
}
template <class E>
hipError_t forward_type(const NormArgs& a, hipStream_t st) {
  return vec_ok(a) ? forward_pick<E, true>(a, st) : forward_pick<E, false>(a, st);
}

// Threads per row of the backward launch (eight columns each up to 2048,
// then sixteen), row groups per block, and blocks: at most one per CU.
constexpr int kNormBlocks = 256;
int backward_chunks(int64_t cols) { return cols <= 2048 ? 1 : 2; }
int backward_tpr(int64_t cols) {
  const int64_t per = 512 * backward_chunks(cols);
  return (int)((cols + per - 1) / per * 64);
}
int backward_groups(int64_t cols) { return 1024 / backward_tpr(cols); }
int backward_blocks(int64_t rows, int64_t cols) {
  const int64_t g = backward_groups(cols);
  const int64_t b = (rows + g - 1) / g;
  return (int)(b < kNormBlocks ? b : kNormBlocks);
}

template <class E, bool VEC>
hipError_t backward_pick(const NormArgs& a, float* part, hipStream_t st) {
  const int tpr = backward_tpr(a.cols), gr = backward_groups(a.cols);
  const dim3 grid((unsigned)backward_blocks(a.rows, a.cols)), block(tpr * gr);
  if (backward_chunks(a.cols) == 1)
    hipLaunchKernelGGL((norm_backward_kernel<E, VEC, 1>), grid, block, 0, st, a, part, tpr, gr);
  else
    hipLaunchKernelGGL((norm_backward_kernel<E, VEC, 2>), grid, block, 0, st, a, part, tpr, gr);
  return hipGetLastError();
}
template <class E>
hipError_t backward_type(const NormArgs& a, float* part, hipStream_t st) {
  const bool sums = a.dgamma != nullptr || a.dbeta != nullptr;
  if (!sums) part = nullptr;
  if (a.rows > 0) {
    if (hipError_t e = vec_ok(a) ? backward_pick<E, true>(a, part, st) : backward_pick<E, false>(a, part, st)) return e;
  }
  if (!sums) return hipSuccess;
  hipLaunchKernelGGL((norm_join_kernel<E>), dim3((unsigned)ceil_div(a.cols, 64), 2), dim3(1024), 0, st, a, part,
                     a.rows > 0 ? backward_blocks(a.rows, a.cols) : 0);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_forward(const NormArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  switch (a.type) {
    case kTypeBf16: return forward_type<NormElem<kTypeBf16>>(a, st);
    case kTypeF16: return forward_type<NormElem<kTypeF16>>(a, st);
    default: return forward_type<NormElem<kTypeF32>>(a, st);
  }
}

size_t norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  return (size_t)backward_blocks(rows, cols) * 2 * (size_t)cols * sizeof(float);
}

hipError_t launch_norm_backward(const NormArgs& a, void* ws, hipStream_t st) {
  switch (a.type) {
    case kTypeBf16: return backward_type<NormElem<kTypeBf16>>(a, static_cast<float*>(ws), st);
    case kTypeF16: return backward_type<NormElem<kTypeF16>>(a, static_cast<float*>(ws), st);
    default: return backward_type<NormElem<kTypeF32>>(a, static_cast<float*>(ws), st);
  }
}

}  // namespace moe
