// AdamW step over many tensors in one launch.  With g = grad * grad_scale:
//   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,
//   p = p (1 - lr decay) - lr / c1 * m / (sqrt(v) / sqrt(c2) + eps),
//   c1 = 1 - beta1^step, c2 = 1 - beta2^step,
// in fp32; p is rounded once to its own type and once to the copy's.
//
// States in 32 bits, or in 8: m and sqrt(v) as E4M3 codes with one exponent for
// every 128 values of a tensor, value = code * 2^(exponent - 127).  sqrt(v)
// and not v, so that the codes' 2^18 of range are 2^36 of v's.  A step moves
// an average by less than half a step of its code (1 - beta2 of v, where codes
// are 1/8 to 1/16 apart), so rounding to nearest would leave it where it is
// for good; codes round up or down instead, by a number below 2^16 that is a
// function of the value's place and the step, and are right on average.  The
// update itself takes the unrounded m and v.  Right on average are m and sqrt(v):
// the square of a rounded root is larger by the rounding's variance, so v settles
// 2.5, 4.0 and 4.0 % high at beta2 = 0.95, 0.99 and 0.999 with normal gradients,
// a single root 11, 14 and 15 % rms from what 32 bits hold.
//
// A block takes a chunk of one tensor; the list of tensors comes with the
// launch's arguments (no copy to the device, nothing to keep for a graph).
// Bound by memory: 28 bytes a value with fp32 masters, bf16 gradients and
// copies and 32-bit states, 16 with states in 8.  302M values: 1379 us (6.1
// TB/s) and 826 us (5.9 TB/s).  What the blocks under way read lies closer
// together the smaller the blocks are (one after the other on another card, us with
// states in 32 and in 8 bits): 1024 values to a block 1417 and 889, 2048 1474 and
// 889, 8192 1569 and 948, 32768 1663 and 998.  Stores, and with 32-bit states loads, carry the non-temporal hint
// (1544 without it on loads); with 8-bit states the loads are better without
// (889 -> 841).
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

#pragma clang fp contract(off)                    // the averages as written, so that states do not depend on fusing

template <int BYTES> struct Raw;
template <> struct Raw<4> { typedef uint32_t type; };
template <> struct Raw<8> { typedef uint32_t type __attribute__((ext_vector_type(2))); };
template <> struct Raw<16> { typedef uint32_t type __attribute__((ext_vector_type(4))); };

// V values of a type from memory, zeros from the n-th on; and back.  At any
// alignment of the elements.  NT: loads with the non-temporal hint.
template <int TYPE, int V, bool NT = true>
struct Values {
  static constexpr int kSize = TYPE == kTypeF32 ? 4 : 2;
  static constexpr int kPiece = V * kSize < 16 ? V * kSize : 16, kPieces = V * kSize / kPiece;
  typedef typename Raw<kPiece>::type raw_t;
  typedef raw_t any_t __attribute__((aligned(kSize)));
  raw_t raw[kPieces];
  __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
    const char* a = static_cast<const char*>(p) + i * kSize;
    if (n >= V) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const any_t* piece = reinterpret_cast<const any_t*>(a + k * kPiece);
        raw[k] = NT ? __builtin_nontemporal_load(piece) : *piece;
      }
    } else {
      uint32_t w[V * kSize / 4] = {};
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (k < n) {
          if constexpr (kSize == 4) w[k] = reinterpret_cast<const uint32_t*>(a)[k];
          else w[k / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(a)[k] << (16 * (k & 1));
        }
      __builtin_memcpy(raw, w, sizeof(w));
    }
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
    uint32_t w[V * kSize / 4];
    __builtin_memcpy(w, raw, sizeof(w));
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if constexpr (TYPE == kTypeF32) f[k] = __uint_as_float(w[k]);
      else if constexpr (TYPE == kTypeBf16) f[k] = bf16_to_f32((uint16_t)(w[k / 2] >> (16 * (k & 1))));
      else f[k] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[k / 2] >> (16 * (k & 1))));
    }
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, int n, const float (&f)[V]) {
    char* a = static_cast<char*>(p) + i * kSize;
    uint32_t w[V * kSize / 4] = {};
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if constexpr (TYPE == kTypeF32) w[k] = __float_as_uint(f[k]);
      else if constexpr (TYPE == kTypeBf16) w[k / 2] |= (uint32_t)f32_to_bf16(f[k]) << (16 * (k & 1));
      else w[k / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f[k]) << (16 * (k & 1));
    }
    if (n >= V) {
      raw_t r[kPieces];
      __builtin_memcpy(r, w, sizeof(w));
#pragma unroll
      for (int k = 0; k < kPieces; ++k) __builtin_nontemporal_store(r[k], reinterpret_cast<any_t*>(a + k * kPiece));
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (k < n) {
          if constexpr (kSize == 4) reinterpret_cast<uint32_t*>(a)[k] = w[k];
          else reinterpret_cast<uint16_t*>(a)[k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
        }
    }
  }
};

// What all values of a call share.
struct Hyper {
  float b1, a1, b2, a2;      // beta1, 1 - beta1, ...
  float keep, size, root, eps, scale;
  uint32_t salt;             // of the rounding
};

// beta^t by squaring, in 64 bits.
__device__ __forceinline__ double power(double b, uint32_t t) {
  double r = 1.0;
  for (; t != 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

__device__ __forceinline__ Hyper hyper(const AdamWArgs& a) {
  Hyper h{a.b1, a.a1, a.b2, a.a2, a.keep, a.size, a.root, a.eps, 1.f, (uint32_t)a.step * 0x9E3779B9u};
  if (a.step_dev != nullptr || a.lr_dev != nullptr) {
    const double lr = a.lr_dev != nullptr ? (double)*a.lr_dev : a.lr;
    const int step = a.step_dev != nullptr ? max(*a.step_dev, 1) : a.step;
    h.keep = (float)(1.0 - lr * a.decay);
    h.size = (float)(lr / (1.0 - power(a.beta1, step)));
    h.root = (float)(1.0 / sqrt(1.0 - power(a.beta2, step)));
    h.salt = (uint32_t)step * 0x9E3779B9u;
  }
  if (a.grad_scale != nullptr) h.scale = *a.grad_scale;
  return h;
}

__device__ __forceinline__ void step1(const Hyper& h, float grad, float& p, float& m, float& v, float& root) {
  const float g = grad * h.scale;
  m = m * h.b1 + g * h.a1;
  v = v * h.b2 + g * g * h.a2;
  // within 1 ulp, as the reciprocal: both far below the step's own rounding
  // (the instruction takes numbers below 2^-126 for zeros, which shows where eps is 0)
  const bool low = v < 0x1p-96f;
  root = __builtin_amdgcn_sqrtf(v * (low ? 0x1p64f : 1.f)) * (low ? 0x1p-32f : 1.f);
  p = p * h.keep - m * __builtin_amdgcn_rcpf(root * h.root + h.eps) * h.size;
}

// ------------------------------------------------------------- 8-bit states

// A number below 2^32 from a value's place in its tensor and the step: two
// rounds of a multiplication and a shifted exclusive or.
__device__ __forceinline__ uint32_t draw(uint32_t at, uint32_t salt) {
  uint32_t z = at + salt;
  z = (z ^ (z >> 16)) * 0x6C8E9CF5u;
  z = (z ^ (z >> 15)) * 0x2B7E1517u;
  return z ^ (z >> 16);
}

// Largest of 16 neighbouring lanes' values, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));    // quad_perm 1 0 3 2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));    // quad_perm 2 3 0 1
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));   // row_half_mirror
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));   // row_mirror
  return v;
}

// Biased exponent of a block whose largest magnitude has the bits `top`: the
// least power of two that brings it to 448 or below.  255: the block holds a
// value that is no finite number, and all of it is NaN.
__device__ __forceinline__ uint32_t block_exponent(uint32_t top) {
  return top >= 0x7f800000u ? 255u : (uint32_t)max((int)((top + 0x1FFFFFu) >> 23) - 8, 1);
}

// Byte K of `codes`: the E4M3 code of f, |f| <= 448, the neighbour further from
// zero where the bits of f below the code's last, plus the upper bits of `seed`
// at their place, carry into it (gfx950's conversion with such a rounding;
// whole-number arithmetic took ten instructions more).
template <int K>
__device__ __forceinline__ uint32_t e4m3(uint32_t codes, float f, uint32_t seed) {
  return (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(f, seed, codes, K);
}

__device__ __forceinline__ void widen8(uint2 c, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = i ? c.y : c.x;
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    f[4 * i] = lo[0];
    f[4 * i + 1] = lo[1];
    f[4 * i + 2] = hi[0];
    f[4 * i + 3] = hi[1];
  }
}

// Eight codes from p on (at any alignment), zeros from the n-th on; and back.
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int n) {
  typedef uint32_t any_t __attribute__((ext_vector_type(2), aligned(1)));
  if (n >= 8) {
    const any_t v = *reinterpret_cast<const any_t*>(p);
    return uint2{v[0], v[1]};
  }
  uint2 c{0, 0};
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (k < n) (k < 4 ? c.x : c.y) |= (uint32_t)p[k] << (8 * (k & 3));
  return c;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int n, uint2 c) {
  typedef uint32_t vec_t __attribute__((ext_vector_type(2)));
  typedef vec_t any_t __attribute__((aligned(1)));
  if (n >= 8) {
    __builtin_nontemporal_store(vec_t{c.x, c.y}, reinterpret_cast<any_t*>(p));
    return;
  }
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (k < n) p[k] = (uint8_t)((k < 4 ? c.x : c.y) >> (8 * (k & 3)));
}

// -------------------------------------------------------------- the kernel

constexpr int kThreads = 128;
constexpr int kStep = 1024;                       // values of a block's turn; chunks are whole turns

template <int PT, int V>
__device__ __forceinline__ void write_back(const AdamWTensor& t, int64_t i, int n, const float (&p)[V]) {
  Values<PT, V>::store(t.param, i, n, p);
  if (t.copy == nullptr) return;
  if (t.copy_type == kTypeBf16) Values<kTypeBf16, V>::store(t.copy, i, n, p);
  else Values<kTypeF16, V>::store(t.copy, i, n, p);
}

// 32-bit states: four values a lane, two such pieces in flight.
template <int PT, int GT>
__device__ __forceinline__ void chunk32(const AdamWTensor& t, const Hyper& h, int64_t begin, int64_t end) {
  constexpr int V = 4, U = kStep / (kThreads * V);
  for (int64_t at = begin + threadIdx.x * V; at - (int64_t)threadIdx.x * V < end; at += kStep) {
    Values<PT, V> p[U];
    Values<GT, V> g[U];
    Values<kTypeF32, V> m[U], v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t i = at + k * kThreads * V;
      const int n = (int)min(end - i, (int64_t)V);
      p[k].load(t.param, i, n);
      g[k].load(t.grad, i, n);
      m[k].load(t.m, i, n);
      v[k].load(t.v, i, n);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t i = at + k * kThreads * V;
      const int n = (int)min(end - i, (int64_t)V);
      float pf[V], gf[V], mf[V], vf[V], root;
      p[k].get(pf);
      g[k].get(gf);
      m[k].get(mf);
      v[k].get(vf);
#pragma unroll
      for (int q = 0; q < V; ++q) step1(h, gf[q], pf[q], mf[q], vf[q], root);
      if (n <= 0) continue;
      write_back<PT>(t, i, n, pf);
      Values<kTypeF32, V>::store(t.m, i, n, mf);
      Values<kTypeF32, V>::store(t.v, i, n, vf);
    }
  }
}

// 8-bit states: eight values a lane, sixteen lanes to a block of 128.
template <int PT, int GT>
__device__ __forceinline__ void chunk8(const AdamWTensor& t, const Hyper& h, int64_t begin, int64_t end) {
  constexpr int V = 8;
  static_assert(kThreads * V == kStep, "one turn");
  uint8_t* mc = static_cast<uint8_t*>(t.m);
  uint8_t* vc = static_cast<uint8_t*>(t.v);
  for (int64_t at = begin; at < end; at += kStep) {
    const int64_t i = at + threadIdx.x * V;
    const int n = (int)max(min(end - i, (int64_t)V), (int64_t)0);
    const bool any = n > 0;                       // the block has values here: lane 0 of its sixteen does
    Values<PT, V, false> p;
    Values<GT, V, false> g;
    p.load(t.param, i, n);
    g.load(t.grad, i, n);
    const uint2 mw = load_codes(mc + i, n), vw = load_codes(vc + i, n);
    const uint32_t me = any ? t.m_exp[i >> 7] : 0u, ve = any ? t.v_exp[i >> 7] : 0u;
    float pf[V], gf[V], m[V], v[V], root[V];
    p.get(pf);
    g.get(gf);
    widen8(mw, m);
    widen8(vw, v);
    const float ms = __uint_as_float(me << 23), vs = __uint_as_float(ve << 23);
#pragma unroll
    for (int q = 0; q < V; ++q) {
      m[q] *= ms;
      v[q] *= vs;
      v[q] *= v[q];
      step1(h, gf[q], pf[q], m[q], v[q], root[q]);
    }
    if (n < V) {                                  // zero past the end, also with a gradient scale that is no number
#pragma unroll
      for (int q = 0; q < V; ++q) {
        m[q] = q < n ? m[q] : 0.f;
        v[q] = q < n ? v[q] : 0.f;
      }
    }
    uint32_t mt = 0, vt = 0;
#pragma unroll
    for (int q = 0; q < V; ++q) {
      mt = max(mt, __float_as_uint(m[q]) & 0x7fffffffu);
      vt = max(vt, __float_as_uint(v[q]) & 0x7fffffffu);
    }
    mt = max16(mt);
    vt = max16(vt);
    // the block's largest root, correctly rounded: its exponent is exact
    vt = vt >= 0x7f800000u ? vt : __float_as_uint(sqrtf(__uint_as_float(vt)));
    const uint32_t mn = block_exponent(mt), vn = block_exponent(vt);
    const float mi = __uint_as_float((254u - mn) << 23), vi = __uint_as_float((254u - vn) << 23);
    uint2 mo{0, 0}, vo{0, 0};
    auto encode = [&](auto k, uint32_t& mw, uint32_t& vw, int q) __attribute__((always_inline)) {
      constexpr int K = decltype(k)::value;
      const uint32_t z = draw((uint32_t)i + q, h.salt);
      mw = e4m3<K>(mw, m[q] * mi, z << 16);
      // no divisor that was there is lost, and a root one bit too large stays a code
      vw = e4m3<K>(vw, fminf(fmaxf(root[q] * vi, v[q] > 0.f ? 0x1p-9f : 0.f), 448.f), z & 0xffff0000u);
    };
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t& mw = w ? mo.y : mo.x;
      uint32_t& vw = w ? vo.y : vo.x;
      encode(std::integral_constant<int, 0>{}, mw, vw, 4 * w);
      encode(std::integral_constant<int, 1>{}, mw, vw, 4 * w + 1);
      encode(std::integral_constant<int, 2>{}, mw, vw, 4 * w + 2);
      encode(std::integral_constant<int, 3>{}, mw, vw, 4 * w + 3);
      if (mn == 255u) mw = 0x7f7f7f7fu;
      if (vn == 255u) vw = 0x7f7f7f7fu;
    }
    if (!any) continue;
    write_back<PT>(t, i, n, pf);
    store_codes(mc + i, n, mo);
    store_codes(vc + i, n, vo);
    if ((threadIdx.x & 15) == 0) {
      t.m_exp[i >> 7] = (uint8_t)mn;
      t.v_exp[i >> 7] = (uint8_t)vn;
    }
  }
}

template <bool FP8, int PT, int GT>
__device__ __forceinline__ void chunk(const AdamWTensor& t, const Hyper& h, int64_t begin, int64_t end) {
  if constexpr (FP8) chunk8<PT, GT>(t, h, begin, end);
  else chunk32<PT, GT>(t, h, begin, end);
}
template <bool FP8, int PT>
__device__ __forceinline__ void chunk_of(const AdamWTensor& t, const Hyper& h, int64_t begin, int64_t end) {
  if (t.grad_type == kTypeBf16) chunk<FP8, PT, kTypeBf16>(t, h, begin, end);
  else if (t.grad_type == kTypeF16) chunk<FP8, PT, kTypeF16>(t, h, begin, end);
  else chunk<FP8, PT, kTypeF32>(t, h, begin, end);
}

template <bool FP8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamWArgs a) {
  // the tensor whose chunks this block's index is among: the last that starts
  // at or before it
  const int lane = threadIdx.x & 63;
  const uint32_t first = lane < a.count ? a.tensor[lane].first_chunk : 0xffffffffu;
  const int k = 63 - __builtin_clzll(__ballot(lane < a.count && first <= blockIdx.x));
  const AdamWTensor& t = a.tensor[k];
  const int64_t begin = (int64_t)(blockIdx.x - t.first_chunk) * a.chunk, end = min(begin + a.chunk, t.numel);
  const Hyper h = hyper(a);
  if (t.param_type == kTypeBf16) chunk_of<FP8, kTypeBf16>(t, h, begin, end);
  else if (t.param_type == kTypeF16) chunk_of<FP8, kTypeF16>(t, h, begin, end);
  else chunk_of<FP8, kTypeF32>(t, h, begin, end);
}

}  // namespace

hipError_t launch_adamw(AdamWArgs& a, hipStream_t st) {
  int64_t total = 0;
  for (int i = 0; i < a.count; ++i) total += a.tensor[i].numel;
  // chunks of one turn, or of as many as keep the grid at about 2^20 blocks
  a.chunk = kStep * (int)(1 + (total >> 30));
  uint32_t chunks = 0;
  for (int i = 0; i < a.count; ++i) {
    a.tensor[i].first_chunk = chunks;
    chunks += (uint32_t)((a.tensor[i].numel + a.chunk - 1) / a.chunk);
  }
  if (chunks == 0) return hipSuccess;
  if (a.fp8) hipLaunchKernelGGL(adamw_kernel<true>, dim3(chunks), dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL(adamw_kernel<false>, dim3(chunks), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace moe
