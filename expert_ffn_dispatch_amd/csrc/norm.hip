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
// sums) at no further read.  8192 x 4096 bf16 forward: 23.4 us, 5.7 TB/s;
// 4096 x 5120 bf16 backward with fp32 parameters: 31.3 us, 4.0 TB/s, of which the
// launch that joins the parameters' partial sums takes 4.  One row is all
// latency: a kernel of 2.6 us, 7.6 us from the binding.
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

// tpr threads share a row, and each holds NCH groups of eight values of it:
// group i of thread t is columns 8 (i tpr + t) ..+7.  Groups move in 16-byte
// pieces at whatever alignment the row has (unaligned access is on, and whole
// cache lines are used either way); only the last group of a width that is no
// multiple of 8 goes by elements.
__device__ __forceinline__ int norm_col(int i, int t, int tpr) { return 8 * (i * tpr + t); }
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));

// One thread's values of a row, kept as stored (two 16-bit values to a
// register) and widened at use.
template <class E, int NCH>
struct NormVals {
  typedef typename E::T T;
  static constexpr int W = sizeof(T) * 8 / 16;    // 16-byte pieces per group
  u32x4_t r[NCH][W];
  __device__ __forceinline__ float get(int i, int q) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(r[i][q >> 2][q & 3]);
    else return E::get((uint16_t)(r[i][0][q >> 1] >> (16 * (q & 1))));
  }
  __device__ __forceinline__ void set(int i, int q, T v) {
    if constexpr (sizeof(T) == 4) r[i][q >> 2][q & 3] = __builtin_bit_cast(uint32_t, v);
    else r[i][0][q >> 1] |= (uint32_t)v << (16 * (q & 1));
  }
  // p: column 0; columns from `cols` on are zero
  __device__ __forceinline__ void load(const T* p, int cols, int t, int tpr) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = norm_col(i, t, tpr), n = cols - c;
#pragma unroll
      for (int k = 0; k < W; ++k) r[i][k] = u32x4_t{0, 0, 0, 0};
      if (n >= 8) {
#pragma unroll
        for (int k = 0; k < W; ++k) r[i][k] = reinterpret_cast<const u32x4_any_t*>(p + c)[k];
      } else if (n > 0) {
#pragma unroll
        for (int q = 0; q < 7; ++q)
          if (q < n) set(i, q, p[c + q]);
      }
    }
  }
};

// Eight values of column group i of a parameter vector, `dflt` where null.
template <class E>
__device__ __forceinline__ void norm_param(const void* base, bool f32, int cols, int i, int t, int tpr, float dflt, float (&f)[8]) {
  if (base == nullptr) {
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = dflt;
    return;
  }
  const int first = 8 * i * tpr;
  if (f32) {
    NormVals<NormElem<kTypeF32>, 1> v;
    v.load(static_cast<const float*>(base) + first, cols - first, t, tpr);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = v.get(0, q);
  } else {
    NormVals<E, 1> v;
    v.load(static_cast<const typename E::T*>(base) + first, cols - first, t, tpr);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = v.get(0, q);
  }
}

// Group i of a row whose column 0 is p.  Non-temporal: a written row is not
// read again by the launch (2000 x 16384 bf16 forward 38.0 -> 30.6 us, 8192 x
// 1024 9.6 -> 8.4; the hint on the loads lost up to half).
template <class E>
__device__ __forceinline__ void norm_store(typename E::T* p, int cols, int i, int t, int tpr, const float (&f)[8]) {
  const int c = norm_col(i, t, tpr), n = cols - c;
  if (n >= 8) {
    NormVals<E, 1> v;
    if constexpr (sizeof(typename E::T) == 2) v.r[0][0] = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 8; ++q) v.set(0, q, E::put(f[q]));
#pragma unroll
    for (int k = 0; k < NormVals<E, 1>::W; ++k)
      __builtin_nontemporal_store(v.r[0][k], reinterpret_cast<u32x4_any_t*>(p + c) + k);
  } else if (n > 0) {
#pragma unroll
    for (int q = 0; q < 7; ++q)
      if (q < n) p[c + q] = E::put(f[q]);
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// A block barrier for LDS alone: __syncthreads would also wait for the loads
// of the next row and the stores of the last.
__device__ __forceinline__ void lds_sync() {
  __builtin_amdgcn_s_waitcnt(0xC07F);             // lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
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

// One row per TPR threads, blocks of 256 threads or of one row.
template <class E, int TPR, int NCH>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_forward_kernel(NormArgs p) {
  __shared__ float red[2][TPR / 64];
  constexpr int tpr = TPR, kRows = TPR >= 256 ? 1 : 256 / TPR;
  const int t = threadIdx.x % TPR;
  const int row = blockIdx.x * kRows + threadIdx.x / TPR;
  if (kRows > 1 && row >= p.rows) return;         // (one row per block: always live)
  NormVals<E, NCH> v;
  v.load(static_cast<const typename E::T*>(p.x) + (int64_t)row * p.ldx, p.cols, t, tpr);
  const float inv = 1.f / (float)p.cols;
  float mu = 0.f;
  if (!p.rms) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) s += v.get(i, q);
    mu = row_sum<TPR>(s, red[0]) * inv;
  }
  float s2 = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float d = v.get(i, q) - mu;
      s2 += norm_col(i, t, tpr) + q < p.cols ? d * d : 0.f;
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
    norm_param<E>(p.gamma, p.param_f32, p.cols, i, t, tpr, 1.f, g);
    norm_param<E>(p.beta, p.param_f32, p.cols, i, t, tpr, 0.f, b);
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] = (v.get(i, q) - mu) * rstd * g[q] + b[q];
    norm_store<E>(out, p.cols, i, t, tpr, y);
  }
}

// Backward: blocks of `gr` groups of tpr threads, each group walking rows
// group, group + (all groups), ...; a thread keeps the fp32 sums of dgamma and
// dbeta for its columns over all its rows, the block adds its groups' sums in
// LDS at the end and writes one partial row, and norm_join_kernel adds the
// blocks' partials in order (no atomics: the result does not depend on the
// schedule).  The next row's x and dy are in flight while a row is reduced
// and stored.  BLK: the most threads of a block; it bounds the registers.
template <class E, int NCH, int BLK>
__global__ __launch_bounds__(BLK) void norm_backward_kernel(NormArgs p, float* part, int tpr, int gr) {
  typedef typename E::T T;
  __shared__ float red[2][2][16];
  __shared__ float s_sum[8 * BLK];
  const int grp = threadIdx.x / tpr, t = threadIdx.x - grp * tpr;
  const int step = gridDim.x * gr;
  const float inv = 1.f / (float)p.cols;
  float dg[NCH][8], db[NCH][8];
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) dg[i][q] = db[i][q] = 0.f;
  // gamma stays in registers: loaded for each row, its wait (loads complete in
  // order) was a wait for the next row as well
  float g[NCH][8];
#pragma unroll
  for (int i = 0; i < NCH; ++i) norm_param<E>(p.gamma, p.param_f32, p.cols, i, t, tpr, 1.f, g[i]);
  NormVals<E, NCH> x, d, xn, dn;
  float mu, rs, mun, rsn;
  // every group makes the same number of trips (barriers); a row past the
  // end loads nothing and adds zeros
  auto fetch = [&](int row, NormVals<E, NCH>& xv, NormVals<E, NCH>& dv, float& m, float& r) __attribute__((always_inline)) {
    const bool live = row < p.rows;
    const int cols = live ? p.cols : 0;
    const int64_t rr = live ? row : 0;
    xv.load(static_cast<const T*>(p.x) + rr * p.ldx, cols, t, tpr);
    dv.load(static_cast<const T*>(p.dy) + rr * p.ldd, cols, t, tpr);
    m = (live && !p.rms) ? p.mean[rr] : 0.f;
    r = live ? p.rstd[rr] : 0.f;
  };
  constexpr bool kAhead = NCH * sizeof(T) <= 8;   // (32 fp32 columns: two rows would spill)
  if constexpr (kAhead) fetch(blockIdx.x * gr + grp, x, d, mu, rs);
  int par = 0;
  for (int base = blockIdx.x * gr; base < p.rows; base += step, par ^= 1) {
    const int row = base + grp;
    const bool live = row < p.rows;
    if constexpr (kAhead) fetch(row + step, xn, dn, mun, rsn);
    else fetch(row, x, d, mu, rs);
    float s1 = 0.f, s2 = 0.f;
    auto add = [&](int i, int q) __attribute__((always_inline)) {
      const float dyv = d.get(i, q), n = (x.get(i, q) - mu) * rs, gv = dyv * g[i][q];
      s1 += gv;
      s2 += gv * n;
      dg[i][q] += dyv * n;
      db[i][q] += dyv;
    };
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      // nothing past the last column: dy is zero there, but -mu rstd, and so
      // what it adds, need not be finite where n is; a row past the end adds zeros
      const int left = p.cols - norm_col(i, t, tpr);
      if (left >= 8) {
#pragma unroll
        for (int q = 0; q < 8; ++q) add(i, q);
      } else if (left > 0) {
#pragma unroll
        for (int q = 0; q < 7; ++q)
          if (q < left) add(i, q);
      }
    }
    float m1 = wave_sum(s1), m2 = wave_sum(s2);
    if (tpr > 64) {
      const int wave = threadIdx.x >> 6, nw = tpr >> 6;
      if ((threadIdx.x & 63) == 0) {
        red[par][0][wave] = m1;
        red[par][1][wave] = m2;
      }
      lds_sync();
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
        float o[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float n = (x.get(i, q) - mu) * rs;
          o[q] = rs * (d.get(i, q) * g[i][q] - m1 - n * m2);
        }
        norm_store<E>(out, p.cols, i, t, tpr, o);
      }
    }
    if constexpr (kAhead) {
      x = xn;
      d = dn;
      mu = mun;
      rs = rsn;
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
        const int c = norm_col(i, t, tpr);
        float* o = part + ((int64_t)blockIdx.x * 2 + which) * p.cols + c;
        if (c + 8 <= p.cols) {
          typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));
          reinterpret_cast<f32x4_any_t*>(o)[0] = f32x4_t{s[0], s[1], s[2], s[3]};
          reinterpret_cast<f32x4_any_t*>(o)[1] = f32x4_t{s[4], s[5], s[6], s[7]};
        } else {
#pragma unroll
          for (int q = 0; q < 7; ++q)
            if (c + q < p.cols) o[q] = s[q];
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
#pragma unroll 16
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

template <class E, int TPR, int NCH>
hipError_t forward_go(const NormArgs& a, hipStream_t st) {
  constexpr int kRows = TPR >= 256 ? 1 : 256 / TPR;
  hipLaunchKernelGGL((norm_forward_kernel<E, TPR, NCH>), dim3((unsigned)ceil_div(a.rows, kRows)),
                     dim3(TPR * kRows), 0, st, a);
  return hipGetLastError();
}
// A wave per row (no barrier) up to 2048 columns where there are rows enough,
// else a block (8192 x 4096 bf16: 38.4 us by waves, 28.6 by blocks; 8192 x 1024
// 9.6 against 13.7), of 1024 threads above 8192 columns (2000 x 16384 25.7 us,
// 30.7 with 256).
template <class E>
hipError_t forward_type(const NormArgs& a, hipStream_t st) {
  if (a.cols <= 512) return forward_go<E, 64, 1>(a, st);
  if (a.rows >= 1024) {
    if (a.cols <= 1024) return forward_go<E, 64, 2>(a, st);
    if (a.cols <= 2048) return forward_go<E, 64, 4>(a, st);
  }
  if (a.cols <= 2048) return forward_go<E, 256, 1>(a, st);
  if (a.cols <= 4096) return forward_go<E, 256, 2>(a, st);
  if (a.cols <= 8192) return forward_go<E, 256, 4>(a, st);
  return forward_go<E, 1024, 2>(a, st);
}
// Backward launch: 8 columns per thread up to 2048, 16 up to 8192, then 32;
// blocks of at most 768 threads (three waves per SIMD, 168 registers), with 32
// columns 512 (256 registers); at most one block per CU.
constexpr int kNormBlocks = 256;
int backward_chunks(int64_t cols) { return cols <= 2048 ? 1 : cols <= 8192 ? 2 : 4; }
int backward_tpr(int64_t cols) {
  const int64_t per = 512 * backward_chunks(cols);
  return (int)((cols + per - 1) / per * 64);
}
int backward_groups(int64_t cols) { return (backward_chunks(cols) == 4 ? 512 : 768) / backward_tpr(cols); }
int backward_blocks(int64_t rows, int64_t cols) {
  const int64_t g = backward_groups(cols);
  const int64_t b = (rows + g - 1) / g;
  return (int)(b < kNormBlocks ? b : kNormBlocks);
}

template <class E>
hipError_t backward_pick(const NormArgs& a, float* part, hipStream_t st) {
  const int tpr = backward_tpr(a.cols), gr = backward_groups(a.cols);
  const dim3 grid((unsigned)backward_blocks(a.rows, a.cols)), block(tpr * gr);
  switch (backward_chunks(a.cols)) {
    case 1: hipLaunchKernelGGL((norm_backward_kernel<E, 1, 768>), grid, block, 0, st, a, part, tpr, gr); break;
    case 2: hipLaunchKernelGGL((norm_backward_kernel<E, 2, 768>), grid, block, 0, st, a, part, tpr, gr); break;
    default: hipLaunchKernelGGL((norm_backward_kernel<E, 4, 512>), grid, block, 0, st, a, part, tpr, gr); break;
  }
  return hipGetLastError();
}
template <class E>
hipError_t backward_type(const NormArgs& a, float* part, hipStream_t st) {
  const bool sums = a.dgamma != nullptr || a.dbeta != nullptr;
  if (!sums) part = nullptr;
  if (a.rows > 0) {
    if (hipError_t e = backward_pick<E>(a, part, st)) return e;
  }
  if (!sums) return hipSuccess;
  hipLaunchKernelGGL((norm_join_kernel<E>), dim3((unsigned)ceil_div(a.cols, 64), 2), dim3(1024), 0, st, a, part,
                     a.rows > 0 ? backward_blocks(a.rows, a.cols) : 0);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_forward(const NormArgs& all, hipStream_t st) {
  // a launch takes at most 2^21 rows (of up to 1024 threads: 2^31)
  constexpr int kMost = 1 << 21;
  const int64_t size = all.type == kTypeF32 ? 4 : 2;
  for (int r0 = 0; r0 < all.rows; r0 += kMost) {
    NormArgs a = all;
    a.rows = all.rows - r0 < kMost ? all.rows - r0 : kMost;
    a.x = static_cast<const char*>(all.x) + r0 * all.ldx * size;
    a.out = static_cast<char*>(all.out) + r0 * all.ldo * size;
    if (all.mean) a.mean = all.mean + r0;
    if (all.rstd) a.rstd = all.rstd + r0;
    hipError_t e;
    switch (a.type) {
      case kTypeBf16: e = forward_type<NormElem<kTypeBf16>>(a, st); break;
      case kTypeF16: e = forward_type<NormElem<kTypeF16>>(a, st); break;
      default: e = forward_type<NormElem<kTypeF32>>(a, st); break;
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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
