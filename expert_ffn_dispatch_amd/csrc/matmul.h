// Matrix products on bf16 / fp16 MFMA (gfx950, fp32 accumulate) behind the
// linear layer and the products grouped by expert, in the three forms a layer
// and its gradients need.  W is [out][in], the contraction index is k:
//   forward      y[r][c]     = sum_k x[r][k] W_e[c][k]     (e: r's group)
//   row grad     dx[r][c]    = sum_k dy[r][k] W_e[k][c]
//   weight grad  dW_e[r][c]  = sum_k dy[k][r] x[k][c],  k over e's rows
// An operand is stored with k contiguous ("KC": x, dy and W of the first
// form) or with k as its row index ("KS": W of the second, both of the third).
//
// One kernel: a block multiplies BM x BN tiles over 64-wide stages of k that go
// straight into LDS (columns two stages ahead in three buffers, rows one ahead
// in two), 16x16x32 MFMA, sums in fp32 registers, one rounding at the store.
// KS operands are turned by LDS's transposing reads, so no form needs a
// transposed copy.  Resident blocks start their next tile's loads before they
// store the last one.
//
// Bound by the matrix pipes, whose clock falls with the power that the
// operands' switching costs: 8192 x 8192 x 8192 takes 773 us (1.42 PFLOP/s) of
// random bf16 values and 627 us (1.75) of zeros.  With 32x32x16 MFMA and with
// products not in snake order (below) a loop of products on registers alone
// reached 1.68 PFLOP/s on random values, with 16x16x32 in snake order 1.95.
// 256 x 256 tiles (8 waves of 128 x 64) read 1/128 of an operand byte per flop
// and fill one CU each; 128 x 128 tiles (4 waves of 64 x 64, two blocks a CU)
// fill the card with a quarter of the work.  Four waves of 128 x 128 each,
// and tiles of 128 x 256, were slower at every size tried.
#pragma once
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace moe {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr int kMmK = 64;                          // contraction per stage
constexpr uint32_t kMmBytes = 0x7fffff00u;        // buffer size of a tile's resource
constexpr uint32_t kMmOut = 0x80000000u;          // an offset past it: the load returns zeros

// ------------------------------------------------------------ small helpers

template <bool F16>
__device__ __forceinline__ f32x4_t mm_mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                  0, 0, 0);
  else
    return mfma16(a, b, c);
}

template <bool F16>
__device__ __forceinline__ float mm_load1(uint16_t v) {
  if constexpr (F16) return static_cast<float>(__builtin_bit_cast(_Float16, v));
  else return bf16_to_f32(v);
}
template <bool F16>
__device__ __forceinline__ uint16_t mm_store1(float v) {
  if constexpr (F16) return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  else return f32_to_bf16(v);
}
template <bool F16>
__device__ __forceinline__ uint32_t mm_pack2(float lo, float hi) {
  if constexpr (F16) return (uint32_t)mm_store1<true>(lo) | ((uint32_t)mm_store1<true>(hi) << 16);
  else return pack_bf16x2(lo, hi);
}
template <bool F16>
__device__ __forceinline__ void mm_unpack8(u32x4_t v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = mm_load1<F16>((uint16_t)(v[i] & 0xffffu));
    f[2 * i + 1] = mm_load1<F16>((uint16_t)(v[i] >> 16));
  }
}

// 16 bytes / one element from an integer address in global memory (through a
// pointer without that address space these would be flat loads, which every
// wait for LDS waits for too).
__device__ __forceinline__ u32x4_t mm_global16(uint64_t a) {
#ifdef __HIP_DEVICE_COMPILE__
  typedef uint32_t any_t __attribute__((ext_vector_type(4), aligned(2)));   // unaligned access is on
  return *reinterpret_cast<const __attribute__((address_space(1))) any_t*>(a);
#else
  return u32x4_t{0, 0, 0, 0};
#endif
}
__device__ __forceinline__ uint16_t mm_global2(uint64_t a) {
#ifdef __HIP_DEVICE_COMPILE__
  return *reinterpret_cast<const __attribute__((address_space(1))) uint16_t*>(a);
#else
  return 0;
#endif
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t mm_rsrc(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)kMmBytes, 0x00020000);
}
__device__ __forceinline__ void mm_dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint16_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds, 16, voff, soff, 0, 0);
}
// The same with the non-temporal hint, for weights read once.
__device__ __forceinline__ void mm_dma16_nt(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint16_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds, 16, voff, soff, 0, 2);
}
// 4 x 16 transposing read of 16-bit values: within each 16 lanes, lane l
// names the 8 bytes (row l >> 2, columns 4 (l & 3) ..+3) of a 4 x 16 block and
// receives the block's column l, rows 0..3 (checked on the device).
__device__ __forceinline__ s16x4_t mm_read_tr(const uint16_t* lds) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4_t*)(const_cast<uint16_t*>(lds)));
}
__device__ __forceinline__ void mm_lds_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);             // lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Normal distribution at z, e = exp(-z^2 / 2): the tail Q(z) e^(z^2 / 2) as
// eight powers of 1 / (1 + 0.305 |z|), fitted for the least greatest relative
// error over 0 <= z <= 14.5 (1.0e-7).  In fp32, with an exact e and reciprocal,
// it is within 4.7e-7 of the value itself over |z| <= 13 (2.0e-7 absolute); e
// adds its own z^2 2^-24.  Below zero there is no difference of near numbers, so
// gelu keeps its bits far out, where 1 + erf has none left.
__device__ __forceinline__ float mm_normal(float z, float e) {
  const float t = __builtin_amdgcn_rcpf(1.f + 0.305f * fabsf(z));
  float h = 0.036638856f;
  h = -0.15274605f + t * h;
  h = 0.18531486f + t * h;
  h = -0.037620641f + t * h;
  h = 0.12084039f + t * h;
  h = 0.10347370f + t * h;
  h = 0.12245868f + t * h;
  h = 0.12164024f + t * h;
  h *= t;
  return z < 0.f ? h * e : 1.f - h * e;
}

// Activation of the linear layer, in fp32, of N values: one branch for all, so
// that their exponentials overlap (8192 x 4096 -> 16384, gelu (tanh) and the
// pre-activation saved: 916 us with a branch for each value, 855 so; with
// gelu 944 and 840, and 859 with the tail that keeps its bits).  One reciprocal instruction (1 ulp) in place of a division: the
// result is rounded to 16 bits next.
template <int N>
__device__ __forceinline__ void mm_act(float (&v)[N], int act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int q = 0; q < N; ++q) v[q] = v[q] > 0.f ? v[q] : (v[q] != v[q] ? v[q] : 0.f);
      break;
    case kActGelu:
#pragma unroll
      for (int q = 0; q < N; ++q) v[q] *= mm_normal(v[q], __expf(-0.5f * v[q] * v[q]));
      break;
    case kActGeluTanh:
#pragma unroll
      for (int q = 0; q < N; ++q) {
        // 0.5 z (1 + tanh u) = z / (1 + e^-2u)
        const float z = v[q], u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
        v[q] = z * __builtin_amdgcn_rcpf(1.f + __expf(-2.f * u));
      }
      break;
    case kActSilu:
#pragma unroll
      for (int q = 0; q < N; ++q) v[q] *= __builtin_amdgcn_rcpf(1.f + __expf(-v[q]));
      break;
    default: break;
  }
}

// ------------------------------------------------- operand staging in LDS

// 16-byte chunk c of row r of a KC stage (64 k = 8 chunks a row) sits at
// c ^ mm_swz(r): the 32 rows that a fragment read touches at one chunk fall
// on distinct bank groups.
__device__ __forceinline__ int mm_swz(int row) { return ((row >> 1) ^ ((row & 1) << 2)) & 7; }
// KS stage: rows are k, R columns each; chunk c of row r sits at c ^ mm_kswz(r).
// A transposing read of 32 lanes covers 32 bytes of the four rows 8 g ..+3
// (or +4 ..+7) for two neighbouring g: r & 3 picks a quarter of the 64 banks
// and the parity of g a half of it, so the eight pieces do not meet.
__device__ __forceinline__ int mm_kswz(int krow) { return ((krow & 3) << 2) | (((krow >> 3) & 1) << 1); }

// How one operand's 64-wide stages reach LDS.  KC: stage [R rows][64 k]; KS:
// stage [64 k][R columns].  Either way a stage is R * 128 bytes and each of
// the NI loads of a wave fills 1 KB of it, lane l the bytes 16 l ..+15.
// ALIGNED: 16-byte loads straight into LDS (rows of 16-byte pitch and
// alignment, widths in multiples of 8).  Otherwise any strides and sizes: the
// 16 bytes of a piece are loaded unaligned into registers at the start of a
// stage and written to LDS at its end.
// Rows, columns and k past the ends become zeros (ALIGNED: by an offset past
// the buffer, which reads no memory).
template <bool KC, int R, int NW, bool ALIGNED>
struct MmOperand {
  static constexpr int NI = R / (8 * NW);
  static constexpr int C = KC ? 8 : R / 8;        // chunks per LDS row
  uint64_t base;                                  // byte address of the tile's first element
  uint32_t pitch;                                 // row pitch in bytes
  uint32_t off[NI];                               // per lane: byte offset within a stage
  int kk[NI];                                     // per lane: first k of the piece within a stage
  int wave;
  int lim;                                        // rows (KC) or columns (KS) left in the matrix
  int before;                                     // elements of the row in front of the tile

  // KC: p = element (first row of the tile, first k), ext = live rows.
  // KS: p = element (first k, first column), ext = columns left in the matrix.
  // front: elements of a row in front of p.
  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld, int ext, int front, int wave_, int lane) {
    base = reinterpret_cast<uint64_t>(p);
    before = front;
    lim = ext;
    pitch = (uint32_t)ld * 2u;
    wave = wave_;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int piece = wave * NI + i;
      if constexpr (KC) {
        const int r = 8 * piece + (lane >> 3);
        const int ch = (lane & 7) ^ mm_swz(r);
        off[i] = r < ext ? (uint32_t)r * pitch + (uint32_t)(ch * 16) : kMmOut;
        kk[i] = ch * 8;
      } else {
        const int kr = piece * (64 / C) + lane / C;
        const int ch = (lane % C) ^ mm_kswz(kr);
        off[i] = ch * 8 < ext ? (uint32_t)kr * pitch + (uint32_t)(ch * 16) : kMmOut;
        kk[i] = kr;
      }
    }
  }
  // k is contiguous (KC) or steps by the pitch (KS).  The advance to stage kt
  // goes into the 64-bit scalar base, so lane offsets stay within one stage.
  __device__ __forceinline__ uint64_t at(int kt) const {
    return base + (KC ? (uint64_t)kt * (2 * kMmK) : (uint64_t)kt * kMmK * (uint64_t)pitch);
  }
  // ALIGNED: pieces I0..I1-1 of stage kt into `buf`; kend: the contraction's length
  template <int I0, int I1>
  __device__ __forceinline__ void loads(uint16_t* buf, int kt, int kend) const {
    if constexpr (ALIGNED && I0 < I1) {
      mm_dma16(mm_rsrc(reinterpret_cast<const void*>(at(kt))), kk[I0] < kend - kt * kMmK ? off[I0] : kMmOut, 0,
               buf + (wave * NI + I0) * 512);
      loads<I0 + 1, I1>(buf, kt, kend);
    }
  }
  // !ALIGNED: elements of piece i of stage kt inside the matrix (at most 0:
  // none, at least 8: all)
  __device__ __forceinline__ int inside(int i, int kt, int kend, int lane) const {
    if (off[i] == kMmOut) return 0;
    const int left = kend - kt * kMmK;
    if constexpr (KC) return left - kk[i];
    else return kk[i] < left ? lim - chunk(i, lane) * 8 : 0;
  }
  // every piece of the stage is whole (the same for the whole block)
  __device__ __forceinline__ bool interior(int kt, int kend) const { return lim >= R && kend - kt * kMmK >= kMmK; }
  __device__ __forceinline__ int chunk(int i, int lane) const {
    return (lane % C) ^ mm_kswz((wave * NI + i) * (64 / C) + lane / C);
  }
  // A piece of n elements (1..7) at the matrix's edge is read as the last
  // eight elements of its row and shifted down; true where the row has them.
  __device__ __forceinline__ bool back(int i, int kt, int n, int lane) const {
    return before + (KC ? kt * kMmK + kk[i] : chunk(i, lane) * 8) >= 8 - n;
  }
  // The pieces of stage kt into registers (nothing waits for them here), and
  // from there to LDS.  (With the edge's elements loaded one by one, the tiles
  // that have an edge took microseconds a stage: a weight gradient of 261 x
  // 320 over 20110 rows of 4 groups 53 us.)
  __device__ __forceinline__ void fetch(u32x4_t (&v)[NI], int kt, int kend, int lane) const {
    if constexpr (!ALIGNED) {
      const uint64_t b = at(kt);
      if (interior(kt, kend)) {
#pragma unroll
        for (int i = 0; i < NI; ++i) v[i] = mm_global16(b + off[i]);
        return;
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int n = inside(i, kt, kend, lane);
        v[i] = u32x4_t{0, 0, 0, 0};
        if (n >= 8 || (n > 0 && back(i, kt, n, lane))) v[i] = mm_global16(b + off[i] - (n < 8 ? 2 * (8 - n) : 0));
      }
    }
  }
  __device__ __forceinline__ void put(u32x4_t (&v)[NI], uint16_t* buf, int kt, int kend, int lane) const {
    if constexpr (!ALIGNED) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int n = interior(kt, kend) ? 8 : inside(i, kt, kend, lane);
        if (n > 0 && n < 8) {
          uint64_t lo = v[i][0] | ((uint64_t)v[i][1] << 32), hi = v[i][2] | ((uint64_t)v[i][3] << 32);
          if (back(i, kt, n, lane)) {
            const int sh = 16 * (8 - n);
            lo = sh < 64 ? (lo >> sh) | (hi << (64 - sh)) : hi >> (sh - 64);
            hi = sh < 64 ? hi >> sh : 0;
          } else {                                // a row of fewer than eight elements
            const uint64_t src = at(kt) + off[i];
#pragma nounroll
            for (int j = 0; j < n; ++j) {
              const uint64_t e = (uint64_t)mm_global2(src + 2 * j) << (16 * (j & 3));
              if (j < 4) lo |= e;
              else hi |= e;
            }
          }
          v[i] = u32x4_t{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
        }
        *reinterpret_cast<u32x4_t*>(buf + (wave * NI + i) * 512 + lane * 8) = v[i];
      }
    }
  }
};

// Fragments of a 16-wide block: lane l supplies row / column (l & 15) and the
// k of 8 (l >> 4) ..+7 within each 32-wide step.
template <bool KC, int R>
struct MmFrag {
  int o[KC ? 2 : 1];
  // m0: first row / column of this wave's blocks within the tile (a multiple of 64)
  __device__ __forceinline__ void init(int m0, int lane) {
    const int fr = lane & 15, fg = lane >> 4;
    if constexpr (KC) {
#pragma unroll
      for (int s = 0; s < 2; ++s) o[s] = (m0 + fr) * kMmK + (((4 * s + fg) ^ mm_swz(fr)) << 3);
    } else {
      const int kr = 8 * fg + (fr >> 2);
      o[0] = kr * R + ((((m0 >> 3) + ((fr & 3) >> 1)) ^ mm_kswz(kr)) << 3) + 4 * (fr & 1);
    }
  }
  // fragment of block I in step S
  template <int S, int I>
  __device__ __forceinline__ u32x4_t get(const uint16_t* buf) const {
    if constexpr (KC) {
      return *reinterpret_cast<const u32x4_t*>(buf + o[S] + 16 * I * kMmK);
    } else {
      // block I is chunks 2 I, 2 I + 1 past the first: an exclusive or, like
      // the swizzle, since m0 leaves those bits of the chunk index zero
      const int at = (o[0] ^ (I << 4)) + 32 * S * R;
      const uint2 l = __builtin_bit_cast(uint2, mm_read_tr(buf + at));
      const uint2 h = __builtin_bit_cast(uint2, mm_read_tr(buf + at + 4 * R));
      return u32x4_t{l.x, l.y, h.x, h.y};
    }
  }
  static constexpr int kReads = KC ? 1 : 2;       // LDS reads per fragment
};

// -------------------------------------------------------------- tile list

// Group bounds clamped into [0, rows] and non-decreasing, so that no offset
// a caller can pass makes the kernel leave its buffers.
__device__ __forceinline__ void mm_bounds(const MatmulArgs& p, int e, int& lo, int& hi) {
  if (p.offsets == nullptr) {
    lo = 0;
    hi = p.rows;
    return;
  }
  lo = min(max(p.offsets[e], 0), p.rows);
  hi = min(max(p.offsets[e + 1], lo), p.rows);
}

struct MmTile {
  int e;                                          // group
  int split;                                      // contraction slice, or -1: the whole
  int part;                                       // index of the slice's partial tile
  int row0, nrows;                                // first output row (of the group), live rows
  int col0;
  int g0, gn;                                     // group's first row and rows
};

// Row tile rt of RT over cnt rows: whole 32-row blocks, dealt evenly.
__device__ __forceinline__ void mm_row_tile(int cnt, int RT, int rt, int& off, int& n) {
  const int b = ceil_div(cnt, 32);
  const int lo = (int)((long long)b * rt / RT) * 32, hi = min((int)((long long)b * (rt + 1) / RT) * 32, cnt);
  off = lo;
  n = hi - lo;
}

// Tile `t` of an RT x NT grid, in bands of eight row tiles, row tiles fastest:
// the tiles that run side by side on an XCD form a patch that shares both
// operands in its L2.
__device__ __forceinline__ void mm_grid_pos(int t, int RT, int NT, int& rt, int& ct) {
  const int band = t / (8 * NT);
  const int rem = t - band * 8 * NT;
  const int nb = min(8, RT - 8 * band);
  ct = rem / nb;
  rt = 8 * band + rem - ct * nb;
}

// The same value in every lane, kept in scalar registers.
__device__ __forceinline__ void mm_scalar(MmTile& t) {
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.split = __builtin_amdgcn_readfirstlane(t.split);
  t.part = __builtin_amdgcn_readfirstlane(t.part);
  t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
  t.nrows = __builtin_amdgcn_readfirstlane(t.nrows);
  t.col0 = __builtin_amdgcn_readfirstlane(t.col0);
  t.g0 = __builtin_amdgcn_readfirstlane(t.g0);
  t.gn = __builtin_amdgcn_readfirstlane(t.gn);
}

// Row tiles: dealt evenly from 64 rows on, else BM rows at a time.
template <int BM>
__device__ __forceinline__ void mm_row_part(int cnt, int RT, int rt, int& off, int& n) {
  if constexpr (BM >= 64) {
    mm_row_tile(cnt, RT, rt, off, n);
  } else {
    off = rt * BM;
    n = min(cnt - off, BM);
  }
}

// Tile `i` of the list of a call without ragged groups (one group of all rows,
// or the weight gradients' RT x NT tiles of each group).
template <bool WG, int BM, int BN>
__device__ __forceinline__ void mm_plain_tile(const MatmulArgs& p, int i, MmTile& t) {
  const int RT = ceil_div(p.m, BM), NT = ceil_div(p.n, BN), per = RT * NT;
  t.e = 0;
  t.g0 = 0;
  t.gn = p.rows;
  if constexpr (WG) {
    t.e = i / per;
    i -= t.e * per;
    mm_bounds(p, t.e, t.g0, t.gn);
    t.gn -= t.g0;
  }
  int rt, ct;
  mm_grid_pos(i, RT, NT, rt, ct);
  mm_row_part<BM>(p.m, RT, rt, t.row0, t.nrows);
  t.col0 = ct * BN;
}

// Tile number `step` of this block, or false past the end of its list.  Blocks
// go to the XCDs round-robin by index; XCD x takes the x-th eighth of the tile
// list, and its blocks take that run in turn, so that tiles running side by
// side share operands in the XCD's L2.  The last p.tail tiles are cut into
// p.splits slices of the contraction each, and dealt likewise after the whole
// ones.  Ragged groups (never cut): every wave scans the group sizes (four per
// lane), and each round over the grid takes the next tiles of the list, every
// XCD a run of them: an eighth of the whole list may hold only small groups,
// which wait for their weights' bytes, or only large ones (4096 x 1536, 65536
// rows over 128 experts whose loads fall as rank^-1.2: 859 -> 814 us; evenly
// filled 803 -> 797; with a kernel of its own for plain products 779 and 688).
// Dense lists keep the eighths, whose cut slices then meet their operands in L2
// (both linear gradients of 4000 x 5120 x 5120: 427 us against 444).
template <bool WG, int BM, int BN>
__device__ __forceinline__ bool mm_find_tile(const MatmulArgs& p, int lane, int step, MmTile& t) {
  const int x = blockIdx.x & 7;
  const int64_t mine = (int64_t)(blockIdx.x >> 3) + (int64_t)step * (gridDim.x >> 3);
  t.split = -1;
  t.part = 0;
  if (WG || p.offsets == nullptr) {
    const int64_t tiles = (int64_t)ceil_div(p.m, BM) * ceil_div(p.n, BN) * (WG ? p.E : 1);
    const int64_t whole = tiles - p.tail, items = p.tail * p.splits;
    const int64_t w0 = whole * x >> 3, w1 = whole * (x + 1) >> 3;
    // Weight gradients of several groups: every XCD takes its eighth of each
    // group's tiles, since a tile's time goes with its group's rows (16 groups
    // of 32768 rows, 1536 x 4096, fp32: the largest with four times the
    // smallest's 500 us by eighths of the list, 402 so; equal groups 373 and 384).
    const int per = ceil_div(p.m, BM) * ceil_div(p.n, BN);
    if (WG && p.E > 1 && p.tail == 0 && per >= 64) {
      const int lo = (int)((int64_t)per * x >> 3), n = (int)((int64_t)per * (x + 1) >> 3) - lo;
      if (mine >= (int64_t)n * p.E) return false;
      const int g = (int)mine / n;
      mm_plain_tile<WG, BM, BN>(p, g * per + lo + (int)mine - g * n, t);
      return true;
    }
    if (mine < w1 - w0) {
      mm_plain_tile<WG, BM, BN>(p, (int)(w0 + mine), t);
      return true;
    }
    const int64_t i = (items * x >> 3) + mine - (w1 - w0);
    if (i >= (items * (x + 1) >> 3)) return false;
    const int j = (int)(i / p.splits);
    t.split = (int)i - j * p.splits;
    t.part = (int)i;
    mm_plain_tile<WG, BM, BN>(p, (int)whole + j, t);
    return true;
  }
  const int NT = ceil_div(p.n, BN);
  int sum = 0, cnt4[4] = {0, 0, 0, 0}, tl4[4] = {0, 0, 0, 0}, lo4[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * lane + i;
    if (e < p.E) {
      int hi;
      mm_bounds(p, e, lo4[i], hi);
      cnt4[i] = hi - lo4[i];
    }
    tl4[i] = ceil_div(cnt4[i], BM) * NT;
    sum += tl4[i];
  }
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  const int64_t total = __builtin_amdgcn_readlane(inc, 63);
  const int64_t blocks = gridDim.x >> 3, even = (total + 7) >> 3;
  const int64_t run = blocks < even ? blocks : even, in_run = blockIdx.x >> 3;
  const int64_t idx = ((int64_t)step * 8 + x) * run + in_run;
  if (in_run >= run || idx >= total) return false;
  int local = (int)idx;
  // the lane whose inclusive prefix first passes idx owns the group
  const int L = __builtin_ctzll(__ballot(inc > local));
  int before = __builtin_amdgcn_readlane(inc - sum, L);
  int e = 4 * L, found = 0, lo = 0, cnt = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = __builtin_amdgcn_readlane(tl4[i], L);
    if (!found) {
      if (local < before + n) {
        found = 1;
        e = 4 * L + i;
        lo = __builtin_amdgcn_readlane(lo4[i], L);
        cnt = __builtin_amdgcn_readlane(cnt4[i], L);
        local -= before;
      } else {
        before += n;
      }
    }
  }
  t.e = e;
  t.g0 = lo;
  t.gn = cnt;
  const int RT = ceil_div(cnt, BM);
  int rt, ct;
  mm_grid_pos(local, RT, NT, rt, ct);
  mm_row_part<BM>(cnt, RT, rt, t.row0, t.nrows);
  t.col0 = ct * BN;
  return true;
}

// ---------------------------------------------------------------- epilogue

// Eight consecutive columns of one output row: bias, activation, residual,
// stores.  `orow` is the row of out / residual / pre, `col` its first column.
// Results carry the non-temporal hint: no tile reads them again, and L2 stays
// with the operands (8192 x 4096 x 16384 with the pre-activation saved 942 ->
// 929 us, 24576 rows over 160 experts 635 -> 615).
// (At whatever alignment the rows have: unaligned access is on.)
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ void mm_store16(void* p, u32x4_t v) {
  __builtin_nontemporal_store(v, static_cast<u32x4_any_t*>(p));
}

template <bool F16, bool EPI>
__device__ __forceinline__ void mm_finish8(const MatmulArgs& p, float (&v)[8], const float (&bias)[8], int64_t orow,
                                           int col, int64_t out_off) {
  const int n = p.n - col;                        // columns left
  if (EPI && p.bias != nullptr) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += bias[q];
  }
  const bool vec = n >= 8;
  if (EPI && p.pre != nullptr) {
    uint16_t* o = p.pre + orow * p.ldp + col;
    if (vec) {
      mm_store16(o, u32x4_t{mm_pack2<F16>(v[0], v[1]), mm_pack2<F16>(v[2], v[3]), mm_pack2<F16>(v[4], v[5]),
                            mm_pack2<F16>(v[6], v[7])});
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < n) o[q] = mm_store1<F16>(v[q]);
    }
  }
  if (EPI && p.act != kActNone) mm_act(v, p.act);
  if (EPI && p.residual != nullptr) {
    const uint16_t* r = p.residual + orow * p.ldr + col;
    if (vec) {
      float f[8];
      mm_unpack8<F16>(*reinterpret_cast<const u32x4_any_t*>(r), f);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] += f[q];
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < n) v[q] += mm_load1<F16>(r[q]);
    }
  }
  const int64_t at = out_off + orow * p.ldo + col;
  if (p.out_f32) {
    float* o = static_cast<float*>(p.out) + at;
    if (vec) {
      mm_store16(o, __builtin_bit_cast(u32x4_t, f32x4_t{v[0], v[1], v[2], v[3]}));
      mm_store16(o + 4, __builtin_bit_cast(u32x4_t, f32x4_t{v[4], v[5], v[6], v[7]}));
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < n) o[q] = v[q];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out) + at;
    if (vec) {
      mm_store16(o, u32x4_t{mm_pack2<F16>(v[0], v[1]), mm_pack2<F16>(v[2], v[3]), mm_pack2<F16>(v[4], v[5]),
                            mm_pack2<F16>(v[6], v[7])});
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < n) o[q] = mm_store1<F16>(v[q]);
    }
  }
}

template <bool F16>
__device__ __forceinline__ void mm_bias8(const MatmulArgs& p, int col, float (&b)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    b[q] = 0.f;
    if (p.bias != nullptr && col + q < p.n)
      b[q] = p.bias_f32 ? static_cast<const float*>(p.bias)[col + q]
                        : mm_load1<F16>(static_cast<const uint16_t*>(p.bias)[col + q]);
  }
}

// -------------------------------------------------------------- the kernel

// The kernel's arguments, read again from the kernarg segment at each use of
// this function, and the lane index, computed again: what the tile loop could
// otherwise hoist out of itself (arguments, lane offsets) took some 60
// registers for the whole kernel and spilled.
__device__ __forceinline__ MatmulArgs mm_args() {
#ifdef __HIP_DEVICE_COMPILE__
  typedef const __attribute__((address_space(4))) MatmulArgs* ArgsPtr;
  uint64_t a = reinterpret_cast<uint64_t>(__builtin_amdgcn_kernarg_segment_ptr());
  asm volatile("" : "+s"(a));
  return *reinterpret_cast<ArgsPtr>(a);
#else
  return MatmulArgs{};
#endif
}
__device__ __forceinline__ int mm_lane(int lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

// Order of one step's instructions: G rounds of R / G LDS reads, M / G matrix
// instructions and V / G vector loads, so that neither pipe waits for the
// other's whole batch.
template <int R, int M, int V, int G, int I = 0>
__device__ __forceinline__ void mm_order() {
  if constexpr (I < G) {
    constexpr int r = R * (I + 1) / G - R * I / G, m = M * (I + 1) / G - M * I / G, v = V * (I + 1) / G - V * I / G;
    if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(0x100, r, 0);
    if constexpr (m > 0) __builtin_amdgcn_sched_group_barrier(0x008, m, 0);
    if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x020, v, 0);
    mm_order<R, M, V, G, I + 1>();
  }
}

#define MM_WAIT_VM(N) __builtin_amdgcn_s_waitcnt(((N) & 15) | (((N) >> 4) << 14) | 0x0F70)

// BM x BN output tiles: WM x WN waves of (32 FM) x (16 FN).  AKC /
// BKC: how each operand is stored.  A is the operand of the output's rows, B
// that of its columns; the MFMA takes B first, so a lane ends with one output
// row and runs of four consecutive columns.  EPI: bias, activation, residual or
// the saved pre-activation; without any of them a kernel of its own, as the
// epilogue's instructions cost a plain product their fetches (16384 x 1536 ->
// 4096: 195 us with one kernel for both, 170 so).
template <bool F16, bool AKC, bool BKC, int BM, int BN, int WM, int WN, bool ALIGNED, bool EPI>
__global__ __launch_bounds__(64 * WM * WN, BM * BN > 128 * 128 ? 1 : 2) void matmul_tile_kernel(MatmulArgs) {
  constexpr int NW = WM * WN;
  constexpr int FM = BM / (32 * WM);              // a wave's 32-row blocks
  constexpr int FN = BN / (16 * WN);              // and 16-column blocks
  static_assert(FM <= 4 && FN % 4 == 0, "a wave covers whole runs of 64 columns");
  constexpr bool WG = !AKC;                       // weight grad: the contraction runs over rows
  constexpr int STA = BM * kMmK, STB = BN * kMmK;
  // Every buffer an array of its own, so that the compiler knows that loads
  // into one leave reads of another alone.
  __shared__ __align__(16) uint16_t sa0[STA];
  __shared__ __align__(16) uint16_t sa1[STA];
  __shared__ __align__(16) uint16_t sb0[STB];
  __shared__ __align__(16) uint16_t sb1[STB];
  __shared__ __align__(16) uint16_t sb2[STB];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  MmTile t;
  if (!mm_find_tile<WG, BM, BN>(mm_args(), lane, 0, t)) return;
  mm_scalar(t);

  MmOperand<AKC, BM, NW, ALIGNED> la;
  MmOperand<BKC, BN, NW, ALIGNED> lb;
  constexpr int AI = MmOperand<AKC, BM, NW, ALIGNED>::NI, BI = MmOperand<BKC, BN, NW, ALIGNED>::NI;
  constexpr int B2 = (BI + 2) / 3, B3 = (2 * BI + 2) / 3;
  int kend, KT;                                   // the tile's contraction, and its stages
  // a tile's operands, and its first loads: columns of stages 0 and 1, rows of
  // stage 0, in the buffers that the stage loop starts from
  auto start = [&](const MmTile& q) __attribute__((always_inline)) {
    const MatmulArgs p = mm_args();
    const int lane = mm_lane(tid & 63);
    int kbeg = 0;
    kend = WG ? q.gn : p.k;
    if (q.split >= 0) {                           // whole stages to a slice
      const int per = ceil_div(ceil_div(kend, kMmK), p.splits) * kMmK;
      kbeg = min(q.split * per, kend);
      kend = min(kbeg + per, kend) - kbeg;
    }
    KT = max(1, ceil_div(kend, kMmK));
    if constexpr (AKC)
      la.init(p.a + (int64_t)(q.g0 + q.row0) * p.lda + kbeg, p.lda, q.nrows, kbeg, wave, lane);
    else
      la.init(p.a + (int64_t)(q.g0 + kbeg) * p.lda + q.row0, p.lda, p.m - q.row0, q.row0, wave, lane);
    const uint16_t* bp = WG ? p.b + (int64_t)q.g0 * p.ldb : p.b + (int64_t)q.e * p.b_group;
    if constexpr (BKC) lb.init(bp + (int64_t)q.col0 * p.ldb + kbeg, p.ldb, p.n - q.col0, kbeg, wave, lane);
    else lb.init(bp + (int64_t)kbeg * p.ldb + q.col0, p.ldb, p.n - q.col0, q.col0, wave, lane);
    lb.template loads<0, BI>(sb0, 0, kend);
    la.template loads<0, AI>(sa0, 0, kend);
    lb.template loads<0, BI>(sb1, 1, kend);
    if constexpr (!ALIGNED) {
      u32x4_t va[AI], vb[BI];
      la.fetch(va, 0, kend, lane);
      lb.fetch(vb, 0, kend, lane);
      la.put(va, sa0, 0, kend, lane);
      lb.put(vb, sb0, 0, kend, lane);
    }
  };
  start(t);

  MmFrag<AKC, BM> ra;
  MmFrag<BKC, BN> rb;
  ra.init(wm * 32 * FM, lane);
  rb.init(wn * 16 * FN, lane);

  for (int step = 1;; ++step) {
  MmTile tn;
  const bool more = __builtin_amdgcn_readfirstlane(mm_find_tile<WG, BM, BN>(mm_args(), mm_lane(lane), step, tn));
  mm_scalar(tn);

  // NBLK: this wave's 32-row blocks with live rows; the others are neither
  // multiplied nor stored.  Every wave issues its loads and meets every barrier.
  auto body = [&](auto nblk_c) __attribute__((always_inline)) {
    constexpr int NBLK = decltype(nblk_c)::value;
    constexpr int NF = 2 * NBLK;                  // live 16-row blocks
    constexpr int FH = FM;                        // of 2 FM: the first and the second half of a step
    constexpr int N1 = NF < FH ? NF : FH, N2 = NF - N1;
    constexpr int NA = NF > 0 ? NF : 1;
    f32x4_t acc[NA][FN];
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // row fragments of two half steps, column fragments of two steps
    u32x4_t fa[FH], ga[FH], fb[2][FN];

#define MM_FA1(F_, H_, S_, ABUF, I_)                                           \
  if constexpr ((I_) < ((H_) ? N2 : N1)) F_[(I_) < FH ? (I_) : 0] = ra.template get<S_, (H_) * FH + ((I_) < FH ? (I_) : 0)>(ABUF);
#define MM_FA(F_, H_, S_, ABUF)                                                \
  MM_FA1(F_, H_, S_, ABUF, 0) MM_FA1(F_, H_, S_, ABUF, 1) MM_FA1(F_, H_, S_, ABUF, 2) MM_FA1(F_, H_, S_, ABUF, 3)
#define MM_FB1(S_, I_, BBUF)                                                   \
  if constexpr (NF > 0 && (I_) < FN) fb[S_][(I_) < FN ? (I_) : 0] = rb.template get<S_, (I_) < FN ? (I_) : 0>(BBUF);
// half H_ of the column fragments of step S_
#define MM_FB(S_, H_, BBUF)                                                    \
  MM_FB1(S_, (H_) * (FN / 2), BBUF) MM_FB1(S_, (H_) * (FN / 2) + 1, BBUF)      \
  if constexpr (FN > 4) {                                                      \
    MM_FB1(S_, (H_) * (FN / 2) + 2, BBUF) MM_FB1(S_, (H_) * (FN / 2) + 3, BBUF) \
  }
// Products in snake order: from one to the next only one operand changes,
// which costs the matrix pipe less power, and power is what bounds its clock.
#define MM_MMA(F_, H_, S_)                                                     \
  _Pragma("unroll") for (int i = 0; i < ((H_) ? N2 : N1); ++i)                 \
      _Pragma("unroll") for (int jj = 0; jj < FN; ++jj) {                      \
        const int j = (i & 1) ? FN - 1 - jj : jj;                              \
        f32x4_t& c_ = acc[(H_) * FH + i < NA ? (H_) * FH + i : 0][j];          \
        c_ = mm_mfma<F16>(fb[S_][j], F_[i], c_);                               \
      }
// End of one half step (RA_ / RB_ fragments read, M_ rows of products, V_
// loads): nothing moves past it.
#define MM_ORDER(RA_, RB_, M_, V_)                                             \
  if constexpr (NF > 0)                                                        \
    mm_order<(RA_) * decltype(ra)::kReads + (RB_) * decltype(rb)::kReads, (M_) * FN, (V_), 4>();   \
  __builtin_amdgcn_sched_barrier(0);
// Stage KT_: this wave's reads of the last stage and its loads of this one
// are complete (the column operand of the next stage, issued last, may stay in
// flight), the barrier publishes them; then come two 32-wide steps of two
// halves (of the wave's rows), pipelined by one half across the barrier, with
// the loads between their products: the rows of the next stage, into a buffer
// that every wave has finished reading, and the columns of the one after it.
#define MM_STAGE(ABUF, NABUF, BBUF, NBBUF, KT_, FIRST)                         \
  {                                                                            \
    __builtin_amdgcn_s_waitcnt(0xC07F);                                        \
    MM_WAIT_VM(BI);                                                            \
    __builtin_amdgcn_s_barrier();                                              \
    __builtin_amdgcn_sched_barrier(0);                                         \
    la.template loads<0, AI>(NABUF, (KT_) + 1, kend);                          \
    MM_FB(0, 0, BBUF) MM_FA(ga, 0, 0, ABUF) MM_FB(0, 1, BBUF)                  \
    if constexpr (!(FIRST)) { MM_MMA(fa, 1, 1) }                               \
    MM_ORDER(N1, FN, (FIRST) ? 0 : N2, AI)                                     \
    MM_FA(fa, 1, 0, ABUF) MM_FB(1, 0, BBUF)                                    \
    MM_MMA(ga, 0, 0)                                                           \
    lb.template loads<0, B2>(NBBUF, (KT_) + 2, kend);                    \
    MM_ORDER(N2, FN / 2, N1, B2)                                                    \
    MM_FA(ga, 0, 1, ABUF) MM_FB(1, 1, BBUF)                                    \
    MM_MMA(fa, 1, 0)                                                           \
    lb.template loads<B2, B3>(NBBUF, (KT_) + 2, kend);                   \
    MM_ORDER(N1, FN / 2, N2, B3 - B2)                                               \
    MM_FA(fa, 1, 1, ABUF)                                                      \
    MM_MMA(ga, 0, 1)                                                           \
    lb.template loads<B3, BI>(NBBUF, (KT_) + 2, kend);                   \
    MM_ORDER(N2, 0, N1, BI - B3)                                               \
  }
#define MM_A(I) ((I) % 2 == 0 ? sa0 : sa1)
#define MM_B(I) ((I) % 3 == 0 ? sb0 : (I) % 3 == 1 ? sb1 : sb2)
#define MM_U(U, KT_, FIRST) MM_STAGE(MM_A(U), MM_A((U) + 1), MM_B(U), MM_B((U) + 2), KT_, FIRST)

    if constexpr (ALIGNED) {
      MM_U(0, 0, true)
      int kt = 1;
      for (; kt + 5 < KT; kt += 6) {
        MM_U(1, kt, false)
        MM_U(2, kt + 1, false)
        MM_U(3, kt + 2, false)
        MM_U(4, kt + 3, false)
        MM_U(5, kt + 4, false)
        MM_U(6, kt + 5, false)
      }
      if (kt < KT) MM_U(1, kt, false)
      if (kt + 1 < KT) MM_U(2, kt + 1, false)
      if (kt + 2 < KT) MM_U(3, kt + 2, false)
      if (kt + 3 < KT) MM_U(4, kt + 3, false)
      if (kt + 4 < KT) MM_U(5, kt + 4, false)
      MM_MMA(fa, 1, 1)
    } else {
      // One buffer: the next stage is on its way to registers during this
      // one's products, and written when every wave has read this one.
      mm_lds_barrier();
#pragma nounroll
      for (int kt = 0; kt < KT; ++kt) {
        u32x4_t va[AI], vb[BI];
        la.fetch(va, kt + 1, kend, lane);
        lb.fetch(vb, kt + 1, kend, lane);
        MM_FB(0, 0, sb0) MM_FA(ga, 0, 0, sa0) MM_FB(0, 1, sb0)
        MM_FA(fa, 1, 0, sa0) MM_FB(1, 0, sb0)
        MM_MMA(ga, 0, 0)
        MM_FA(ga, 0, 1, sa0) MM_FB(1, 1, sb0)
        MM_MMA(fa, 1, 0)
        MM_FA(fa, 1, 1, sa0)
        MM_MMA(ga, 0, 1)
        MM_MMA(fa, 1, 1)
        mm_lds_barrier();
        la.put(va, sa0, kt + 1, kend, lane);
        lb.put(vb, sb0, kt + 1, kend, lane);
        mm_lds_barrier();
      }
    }
    // Loads past the last stage (zeros) still target the buffers of stages 0
    // and 1 of the next tile and the staging slots: they land first.
    MM_WAIT_VM(0);
    mm_lds_barrier();
    if (more) start(tn);                          // in flight during the epilogue

    // Epilogue: each wave stages 16 rows x 64 columns of fp32 at a time (4 KB of
    // the buffer that the next tile's first loads leave alone) and reads them
    // back as row segments of eight columns, so that loads and stores cover
    // whole 128-byte segments.  Chunk c (four columns) of row r sits at c ^ r:
    // no bank conflicts.
    const MatmulArgs p = mm_args();
    const int lane = mm_lane(tid & 63);
    static_assert(STB * 2 >= NW * 4096, "the waves' staging slots");
    float* blk = reinterpret_cast<float*>(sb2) + wave * 1024;
    const int fr = lane & 15, fg = lane >> 4, ch = lane & 7;
    const int64_t out_off = WG ? (int64_t)t.e * p.out_group : 0;
    const int64_t row_base = (int64_t)(WG ? 0 : t.g0) + t.row0;
#pragma unroll
    for (int h = 0; h < FN / 4; ++h) {
      const int col = t.col0 + wn * 16 * FN + 64 * h + ch * 8;
      float bias[8];
      if constexpr (EPI) mm_bias8<F16>(p, col, bias);
#pragma unroll
      for (int i = 0; i < 2 * FM; ++i) {
        if (i >= NF) break;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<f32x4_t*>(blk + fr * 64 + (((4 * j + fg) ^ fr) << 2)) = acc[i < NA ? i : 0][4 * h + j];
        __builtin_amdgcn_wave_barrier();          // a wave's LDS operations complete in order
        if (t.split >= 0 || p.out_f32) {
          // fp32, nothing to apply: sixteen lanes to a row, so that each store
          // covers whole lines (16 weight gradients of 1536 x 4096, 2048 rows
          // each: 401 us by eight columns a lane, 384 so)
          const int c4 = lane & 15, at = wn * 16 * FN + 64 * h + 4 * c4;
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const int r = 4 * s + fg, row = wm * 32 * FM + 16 * i + r;
            const f32x4_t v = *reinterpret_cast<const f32x4_t*>(blk + r * 64 + ((c4 ^ r) << 2));
            if (row >= t.nrows || t.col0 + at >= p.n) continue;
            if (t.split >= 0) {                   // partial tile [BM][BN], read again by the join
              *reinterpret_cast<f32x4_t*>(p.parts + ((int64_t)t.part * BM + row) * BN + at) = v;
            } else {
              float* o = static_cast<float*>(p.out) + out_off + (row_base + row) * p.ldo + t.col0 + at;
              if (t.col0 + at + 4 <= p.n) {
                mm_store16(o, __builtin_bit_cast(u32x4_t, v));
              } else {
#pragma unroll
                for (int q = 0; q < 3; ++q)
                  if (t.col0 + at + q < p.n) o[q] = v[q];
              }
            }
          }
        } else if (col < p.n) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int r = 8 * s + (lane >> 3);
            const int row = wm * 32 * FM + 16 * i + r;
            const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(blk + r * 64 + (((2 * ch) ^ r) << 2));
            const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(blk + r * 64 + (((2 * ch + 1) ^ r) << 2));
            if (row < t.nrows) {
              float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
              mm_finish8<F16, EPI>(p, v, bias, row_base + row, col, out_off);
            }
          }
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
  };
  const int live = t.nrows - wm * 32 * FM;
  const int nblk = live <= 0 ? 0 : min(FM, ceil_div(live, 32));
  if (!ALIGNED || nblk == FM) {
    body(std::integral_constant<int, FM>{});
  } else if (nblk == 0) {
    body(std::integral_constant<int, 0>{});
  } else if (nblk == 1) {
    body(std::integral_constant<int, 1>{});
  } else if constexpr (FM >= 3) {
    if (nblk == 2) body(std::integral_constant<int, 2>{});
    else if constexpr (FM >= 4) body(std::integral_constant<int, 3>{});
  }
  if (!more) break;
  t = tn;
  }
#undef MM_FA1
#undef MM_FA
#undef MM_FB1
#undef MM_FB
#undef MM_MMA
#undef MM_ORDER
#undef MM_STAGE
#undef MM_A
#undef MM_B
#undef MM_U
}
#undef MM_WAIT_VM

}  // namespace moe
