// Forward products of a few rows (decode): y[r][c] = sum_k x[r][k] W[c][k] for
// at most 16 RB rows of a group at a time, W read once from HBM.
//
// A block of NW waves owns 16 NC output columns; wave w takes every NW-th
// 128-wide chunk of the contraction, so that the block reads 256 NW-byte runs
// of its weight rows.  A chunk (16 NC rows x 256 bytes) goes straight into one
// of two slots of the wave's own LDS, four rows to a load, and comes back as
// MFMA fragments; no wave waits for another until the partial sums are added
// in LDS, in wave order.  The rows of x come as fragments from L2, once per
// block: the wider the block, the fewer of those.
// Bound by the weights' bytes: 6144 -> 16384, one row, bf16: 33.4 us, 6.0 TB/s.
// At tens of rows and smaller weights the fragments of x, which every block
// reads, and the launch weigh as much (37 rows, 4096 -> 4096: 15.5 us).
#include "matmul.h"

namespace moe {

namespace {

constexpr int kStK = 128;                         // contraction per chunk

// NT: the weights are loaded with the non-temporal hint: one group, which reads
// them once (6144 -> 16384, one row: 36.5 -> 33.4 us; among groups some are read
// in several passes, 64 rows over 128 experts of 2048 -> 768 23.8 -> 25.1).
// GATED: the block's columns are pairs, sixteen of W_gate and their sixteen of
// W_up, joined by the activation and the product where the sums are added.
template <bool F16, int RB, int NC, int NW, bool NT, bool GATED>
__global__ __launch_bounds__(64 * NW, RB * NC == 1 ? 4 : NW / 4) void matmul_stream_kernel(MatmulArgs p) {
  constexpr int kOut = GATED ? 8 * NC : 16 * NC;  // output columns of a block
  static_assert(!GATED || NC % 2 == 0, "pairs of columns");
  // an array per slot: loads into one do not hold up reads of the other
  constexpr int kSlot = 16 * NC * kStK;
  __shared__ __align__(16) uint16_t s0[NW * kSlot];
  __shared__ __align__(16) uint16_t s1[NW * kSlot];
  static_assert(RB * NC * 256 * 4 <= kSlot * 2, "a wave's sums fit its slot");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, fg = lane >> 4;
  uint16_t* w0 = s0 + wave * kSlot;
  uint16_t* w1 = s1 + wave * kSlot;
  MmTile t;
  for (int step = 0; mm_find_tile<false, 16 * RB, kOut>(p, lane, step, t); ++step) {
    mm_scalar(t);
    const int chunks = ceil_div(p.k, kStK);
    const int n = wave < chunks ? (chunks - wave + NW - 1) / NW : 0;   // this wave's
    const __amdgpu_buffer_rsrc_t wr = mm_rsrc(p.b + (int64_t)t.e * p.b_group + (int64_t)t.col0 * p.ldb);
    const __amdgpu_buffer_rsrc_t wr2 =
        GATED ? mm_rsrc(p.b2 + (int64_t)t.e * p.b_group + (int64_t)t.col0 * p.ldb) : wr;
    const __amdgpu_buffer_rsrc_t xr = mm_rsrc(p.a + (int64_t)(t.g0 + t.row0) * p.lda);
    // weight rows 4 i + (lane >> 4) of load i, 16-byte piece (lane & 15) ^ (row & 15)
    uint32_t wo[4 * NC];
    int wk[4];
#pragma unroll
    for (int i = 0; i < 4 * NC; ++i) {
      const int r = GATED ? 16 * (i >> 3) + 4 * (i & 3) + fg : 4 * i + fg;    // of its matrix
      wk[i & 3] = (fr ^ (r & 15)) * 8;
      wo[i] = t.col0 + r < p.n ? (uint32_t)r * (uint32_t)(2 * p.ldb) + (uint32_t)(wk[i & 3] * 2) : kMmOut;
    }
    uint32_t xo[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b)
      xo[b] = 16 * b + fr < t.nrows ? (uint32_t)(16 * b + fr) * (uint32_t)(2 * p.lda) + (uint32_t)(fg * 16) : kMmOut;
    f32x4_t acc[NC][RB];
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int b = 0; b < RB; ++b) acc[j][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // chunk c of this wave starts at k = 128 (wave + 8 c); past the last all
    // lanes take zeros
    auto load_w = [&](uint16_t* dst, int c) __attribute__((always_inline)) {
      const int k0 = (wave + NW * c) * kStK;
#pragma unroll
      for (int i = 0; i < 4 * NC; ++i) {
        const uint32_t o = k0 + wk[i & 3] < p.k ? wo[i] : kMmOut;
        const __amdgpu_buffer_rsrc_t w = GATED && (i & 4) ? wr2 : wr;
        if constexpr (NT) mm_dma16_nt(w, o, (uint32_t)(2 * k0), dst + 512 * i);
        else mm_dma16(w, o, (uint32_t)(2 * k0), dst + 512 * i);
      }
    };
    auto load_x = [&](u32x4_t (&x)[RB][4], int c) __attribute__((always_inline)) {
      const int k0 = (wave + NW * c) * kStK;
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          x[b][s] = __builtin_bit_cast(
              u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                           xr, k0 + 32 * s + 8 * fg < p.k ? xo[b] + 64 * s : kMmOut, (uint32_t)(2 * k0), 0));
    };
    auto chunk = [&](const uint16_t* src, const u32x4_t (&x)[RB][4]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        u32x4_t f[4];
#pragma unroll
        for (int s = 0; s < 4; ++s)
          f[s] = *reinterpret_cast<const u32x4_t*>(src + (16 * j + fr) * kStK + (((4 * s + fg) ^ fr) << 3));
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int b = 0; b < RB; ++b) acc[j][b] = mm_mfma<F16>(f[s], x[b][s], acc[j][b]);
      }
    };
    // Two chunks of weights and two of rows under way.  A slot is loaded again
    // once its reads are complete; the wait leaves the younger chunk in flight.
    u32x4_t xa[RB][4], xb[RB][4];
    load_w(w0, 0);
    load_x(xa, 0);
    load_w(w1, 1);
    constexpr int kYounger = 4 * NC + 4 * RB;
    for (int c = 0; c < n; c += 2) {
      load_x(xb, c + 1);
      __builtin_amdgcn_s_waitcnt((kYounger & 15) | ((kYounger >> 4) << 14) | 0x0F70);
      __builtin_amdgcn_sched_barrier(0);
      chunk(w0, xa);
      __builtin_amdgcn_s_waitcnt(0xC07F);
      __builtin_amdgcn_sched_barrier(0);
      load_w(w0, c + 2);
      if (c + 1 >= n) break;
      load_x(xa, c + 2);
      __builtin_amdgcn_s_waitcnt((kYounger & 15) | ((kYounger >> 4) << 14) | 0x0F70);
      __builtin_amdgcn_sched_barrier(0);
      chunk(w1, xb);
      __builtin_amdgcn_s_waitcnt(0xC07F);
      __builtin_amdgcn_sched_barrier(0);
      load_w(w1, c + 3);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);           // loads past the last chunk land
    // partial sums [wave][16 RB rows][16 NC columns] over the slots; column c
    // of row r at c ^ 4 (r & 3), for the banks
    float* part = reinterpret_cast<float*>(w0);
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int j = 0; j < NC; ++j)
        *reinterpret_cast<f32x4_t*>(part + (16 * b + fr) * 16 * NC + 16 * j + 4 * (fg ^ (fr & 3))) = acc[j][b];
    __syncthreads();
    if constexpr (GATED) {
      for (int i = tid; i < RB * NC * 128; i += 64 * NW) {
        const int row = i / kOut, c = i % kOut, col = t.col0 + c;
        const int at = row * 16 * NC + 32 * (c >> 4) + ((c & 15) ^ (4 * (row & 3)));
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          g += reinterpret_cast<const float*>(s0 + w * kSlot)[at];
          u += reinterpret_cast<const float*>(s0 + w * kSlot)[at + 16];
        }
        if (row < t.nrows && col < p.n) gate1<F16>(p, g, u, (int64_t)t.g0 + t.row0 + row, col);
      }
    } else
    for (int i = tid; i < RB * NC * 256; i += 64 * NW) {
      const int row = i / (16 * NC), c = i % (16 * NC), col = t.col0 + (c ^ (4 * (row & 3)));
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v += reinterpret_cast<const float*>(s0 + w * kSlot)[i];
      if (row < t.nrows && col < p.n) finish1<F16>(p, v, (int64_t)t.g0 + t.row0 + row, col);
    }
    __syncthreads();                              // the sums are read before the slots are loaded again
  }
}

template <bool F16, int RB, int NC, int NW, bool NT, bool GATED = false>
hipError_t stream_go(const MatmulArgs& a, hipStream_t st) {
  const long long groups = a.offsets != nullptr ? (a.E < a.rows ? a.E : a.rows) : 1;
  long long grid = ((long long)a.rows / (16 * RB) + groups) * ceil_div(a.n, GATED ? 8 * NC : 16 * NC);
  grid = (grid + 7) / 8 * 8;
  if (grid > (1 << 20)) grid = 1 << 20;
  hipLaunchKernelGGL((matmul_stream_kernel<F16, RB, NC, NW, NT, GATED>), dim3((unsigned)grid), dim3(64 * NW), 0, st, a);
  return hipGetLastError();
}
// Columns per block: sixteen (eight waves) for up to sixteen rows; above, as
// many as leave about 192 blocks, since every block reads all rows of x (32
// rows, us with 16 / 32 / 64 columns: 4096 x 4096 14.6 / 16.8 / 23.7, 16384 ->
// 6144 77.3 / 52.0 / 70.2, 5120 -> 12288 38.2 / 38.2 / 32.9, 6144 -> 16384 47.8
// / 47.7 / 43.3).
template <bool F16, int RB>
hipError_t stream_dense(const MatmulArgs& a, hipStream_t st) {
  if (RB == 1 || a.n < 192 * 32) return stream_go<F16, RB, 1, 8, true>(a, st);
  if (a.n < 192 * 64) return stream_go<F16, RB, 2, 4, true>(a, st);
  return stream_go<F16, RB, 4, 4, true>(a, st);
}
// Gated: sixteen pairs of columns for up to sixteen rows (6144 -> 16384, one row
// 66.3 us, 76.6 with 32; eight rows 68.2 and 79.0), else 32 where they leave about
// 192 blocks (32 rows 88.5 with sixteen, 87.8 so).
template <bool F16, int RB>
hipError_t stream_gated(const MatmulArgs& a, hipStream_t st) {
  if (RB == 1 || a.n < 192 * 32) return stream_go<F16, RB, 2, 4, true, true>(a, st);
  return stream_go<F16, RB, 4, 4, true, true>(a, st);
}
template <bool F16>
hipError_t stream_rows(const MatmulArgs& a, hipStream_t st) {
  if (a.gated) {
    if (a.offsets != nullptr) return stream_go<F16, 1, 2, 4, false, true>(a, st);
    if (a.rows <= 16) return stream_gated<F16, 1>(a, st);
    if (a.rows <= 32) return stream_gated<F16, 2>(a, st);
    return stream_gated<F16, 3>(a, st);
  }
  // groups of a row or two: 32 columns (64 rows over 128 experts of 2048 ->
  // 768 24.2 us, 31.9 with sixteen)
  if (a.offsets != nullptr) return stream_go<F16, 1, 2, 4, false>(a, st);
  if (a.rows <= 16) return stream_dense<F16, 1>(a, st);
  if (a.rows <= 32) return stream_dense<F16, 2>(a, st);
  if (a.rows <= 48) return stream_dense<F16, 3>(a, st);
  return stream_dense<F16, 4>(a, st);
}

}  // namespace

// Dense: up to 64 rows (above, slices of 128 x 128 tiles are as fast: 64 rows of
// 4096 x 4096 22.5 us against 21.9).  Groups: where few experts have a row at
// all, up to half as many rows as experts (8 rows over 128 experts of 2048 ->
// 768 10.0 us against 18.1 by tiles, 64 rows 24.2 against 24.0, 256 rows 52
// against 50, 1024 rows 86 against 85, 4096 rows 143 against 100).  The bound
// is that shape's: 64 experts of it cross a little earlier (32 rows 21.3 us
// against 19.3), wider ones later (rows over 8 experts of 4096 -> 1536: 4 rows
// 13.5 against 30.2, 8 rows 18.3 against the tiles' 31.3 that they take).
// Gated: twice the weights to the rows, so up to twice as many rows as experts
// (256 rows over 128 experts of 2048 -> 768 130 us against 137, 16 rows over 8 of
// 4096 -> 1536 44 against 52), dense up to 48 (4096 -> 4096: 48 rows 20.9 us, 64 rows
// 25.8 against 21.4).
bool matmul_streams(const MatmulArgs& a) {
  if (!a.aligned) return false;
  if (a.gated) return a.offsets != nullptr ? (long long)a.rows <= 2LL * a.E : a.rows <= kMmGatedStreamRows;
  return a.offsets != nullptr ? 2 * (long long)a.rows <= a.E : a.rows <= 64;
}

hipError_t launch_matmul_stream(const MatmulArgs& a, hipStream_t st) {
  return a.f16 ? stream_rows<true>(a, st) : stream_rows<false>(a, st);
}

}  // namespace moe
