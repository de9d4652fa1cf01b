// Internal launchers of the MoE FFN layer's kernels (not part of the C ABI).
// Every launcher enqueues on `st` and returns the launch status; shapes have
// been validated by the caller.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct PermuteArgs;
struct RouteArgs {
  const uint16_t* x;         // [N][M]
  const uint16_t* w_router;  // [M][E]
  const float* bias;         // [E] or null
  int N, M, E, k;
  int32_t* ids;              // [N][k]
  float* weights;            // [N][k]
  // optional, where route_permutes(N): the dispatch and permutation of the
  // routed ids (perm->ids and perm->weights are ids and weights), done by
  // the top-k launch
  const PermuteArgs* perm = nullptr;
};
size_t route_workspace_bytes(int N, int M, int E);
// Batches of at most four tokens: the top-k launch (one block) also permutes.
bool route_permutes(int N);
hipError_t launch_route(const RouteArgs& a, void* ws, hipStream_t st);

// Dispatch + stable permutation.  Tiles of kPermTile assignments.
constexpr int kPermTile = 256;
struct PermuteArgs {
  const int32_t* ids;        // [A] expert of assignment a
  int A, E, k;
  int32_t* counts;           // [E]
  int32_t* offsets;          // [E+1]
  int32_t* s2a;              // [A]
  int32_t* a2s;              // [A]
  int32_t* row_token;        // [A] token of sorted row p (= s2a[p] / k), or null
  const float* weights;      // [A] routing weight per assignment, or null
  float* row_weight;         // [A] weight in sorted order, or null
  int32_t* tile_hist;        // [E][T] workspace
  int32_t* tile_off;         // [E][T] workspace
  int32_t* zero = nullptr;   // n_zero ints set to zero on the way (the expert GEMMs' tile queues)
  int n_zero = 0;
};
// n ints of device memory set to zero (one small launch)
hipError_t launch_zero_words(int32_t* p, int n, hipStream_t st);
hipError_t launch_permute(const PermuteArgs& a, hipStream_t st);

// x_sorted[p] = x[row_token[p]] or x[s2a[p] / k]
hipError_t launch_gather(const uint16_t* x, const int32_t* s2a, int k, int A, int M, uint16_t* xs,
                         hipStream_t st);

// One phase of the grouped SwiGLU.  Rows of group e are
// [offsets[e], offsets[e+1]) (or [0, fixed_rows) with E = 1 if fixed_rows > 0).
struct FfnArgs {
  // phase 1 (gate+up): A rows from `a` ([rows][K]); if a_rows is set, row p
  // of the group reads a[a_rows[p]].  phase 2 (down): A = h, in sorted order
  // (a_rows is ignored).
  const uint16_t* a;
  const int32_t* a_rows;
  const int32_t* offsets;    // [E+1] device, or null with fixed_rows > 0
  int fixed_rows;
  const uint16_t* w0;        // gate [E][H][M] | down [E][M][H]
  const uint16_t* w1;        // up   [E][H][M] | unused
  const float* row_scale;    // phase 2: [rows] fp32 or null
  uint16_t* out;             // phase 1: h [rows][H]; phase 2: y [rows][M]
  int E;                     // groups
  int rows_total;            // upper bound on rows (N*k)
  int K;                     // contraction: M (phase 1) | H (phase 2)
  int ncols;                 // output columns: H (phase 1) | M (phase 2)
  // phase 2: if set, sorted row p is stored as row out_rows[p] of `out` (a
  // token row of the layer output: top-1 routing without shared experts
  // needs no combine)
  const int32_t* out_rows = nullptr;
  // rows of `a` where a_rows is set (0: not known); a launcher sets a_bytes
  // to the bytes of `a` when they fit 32-bit offsets
  int a_nrows = 0;
  uint32_t a_bytes = 0;
  // FP8 weights: if q0 is set, w0/w1 are unused and q0/q1 hold OCP E4M3
  // codes laid out like them; s0/s1 [E][ncols] are the float32 scales of
  // each output channel (weight = value(code) * scale)
  const uint8_t* q0 = nullptr;
  const uint8_t* q1 = nullptr;
  const float* s0 = nullptr;
  const float* s1 = nullptr;
  // eight tile counters of the tile kernel's queues (device, kQueueWords
  // ints), or null for static dealing; queue_zeroed: they are zero when the
  // launch starts (else the launcher clears them first)
  int32_t* queue = nullptr;
  bool queue_zeroed = false;
};
constexpr int kQueueWords = 8;
hipError_t launch_ffn_gateup(const FfnArgs& a, int num_cu, hipStream_t st);
hipError_t launch_ffn_down(const FfnArgs& a, int num_cu, hipStream_t st);
// The routed groups together with the shared experts (shared: E = 1,
// fixed_rows = N): one launch where both take the tile kernel, else two.
hipError_t launch_ffn_gateup_shared(const FfnArgs& routed, const FfnArgs& shared, int num_cu, hipStream_t st);
hipError_t launch_ffn_down_shared(const FfnArgs& routed, const FfnArgs& shared, int num_cu, hipStream_t st);

// Per-row OCP E4M3 quantisation: scale[r] = max_k |w[r][k]| / 448 (1 for a
// zero row), q[r][k] = E4M3 nearest to w[r][k] / scale[r], ties to even,
// saturating.  cols % 8 == 0.
hipError_t launch_quantize_fp8(const uint16_t* w, long long rows, int cols, uint8_t* q, float* scale,
                               hipStream_t st);

// Single-launch layer for decode-sized batches (decode.hip): router, top-k,
// permutation, grouped SwiGLU and combine in one cooperative launch with
// grid-wide barriers.  Weights are bf16 (w_*) or FP8 codes with scales
// (q_*, s_*).  ws holds decode_workspace_bytes(N, M, E) bytes; h and y are
// [N*k][H] and [N*k][M].
constexpr int kDecodeTokens = 8;
constexpr int kDecodeAssign = 64;
constexpr int kDecodeMaxBlocks = 1024;
constexpr int kDecodeMaxExperts = 256;
struct DecodeSync;
struct DecodeArgs {
  const uint16_t* x;         // [N][M]
  const uint16_t* w_router;  // [M][E]
  const float* bias;         // [E] or null
  int N, M, E, k, H;
  const uint16_t* w_gate;
  const uint16_t* w_up;
  const uint16_t* w_down;
  const uint8_t* q_gate;
  const uint8_t* q_up;
  const uint8_t* q_down;
  const float* s_gate;
  const float* s_up;
  const float* s_down;
  int32_t* ids;              // [N][k] out
  float* wts;                // [N][k] out
  uint16_t* out;             // [N][M] out
  uint16_t* h;
  uint16_t* y;
  uint64_t limit;            // longest barrier wait, in wall-clock ticks
  // set by the launcher
  float* part;
  DecodeSync* sync;
  int G, MS;
};
bool decode_fusable(int N, int M, int E, int k, int H, bool f8);
size_t decode_workspace_bytes(int N, int M, int E);
hipError_t launch_decode_layer(DecodeArgs a, void* ws, int num_cu, hipStream_t st);

struct CombineArgs {
  const uint16_t* y;         // [A][M] bf16
  const int32_t* a2s;        // [A]
  const float* weights;      // [N][k] or null
  const uint16_t* shared;    // [N][M] or null
  uint16_t* out;             // [N][M]
  int N, M, k;
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t st);

// ---- matrix products of the linear layer and of the products by expert ----
enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };
// One product (matmul.h states the three forms).  Strides in elements.
struct MatmulArgs {
  const uint16_t* a;         // rows' operand: x | dy | dy
  const uint16_t* b;         // columns' operand: W | W | x
  void* out;
  int64_t lda, ldb, ldo;
  int64_t b_group;           // forward, row grad: elements from one group's W to the next
  int64_t out_group;         // weight grad: elements from one group's output to the next
  const int32_t* offsets;    // [E+1] device, or null: one group of all rows
  int E;
  int rows;                  // rows of the grouped operands
  int m, n, k;               // output rows (of one group), output columns, contraction (weight grad: unused)
  int out_f32;
  // epilogue (null / kActNone: none): out = act(sum + bias) + residual, pre = sum + bias
  const void* bias;
  int bias_f32;
  int act;
  const uint16_t* residual;
  int64_t ldr;
  uint16_t* pre;
  int64_t ldp;
  // the gated projections (GATED in matmul.h)
  int gated;
  const uint16_t* b2;        // forward, row grad: W_up beside W_gate (b), of the same shape
  uint16_t* pre2;            // forward: the up products beside the gates (pre)
  int64_t ldp2;
  void* out2;                // weight grad: W_up's gradient beside W_gate's (out)
  int64_t a_half;            // weight grad: elements from dgate's columns to dup's
  int b2_half;               // weight grad: E counts both gradients of every group of rows
  int a_padded;              // a's last piece of a row may be read whole and is zero past the width
  int b_padded;              // so are b's, and b2's
  int f16;                   // operands are fp16 (else bf16)
  int whole;                 // no contraction slices (no workspace for them)
  // set by launch_matmul: the plan
  int aligned;               // a and b take 16-byte loads
  int big;                   // 256 x 256 tiles (else 128 x 128)
  int tail;                  // tiles at the end of the list that are cut into
  int splits;                // slices of the contraction, whose fp32 partial
  float* parts;              // tiles are here, joined by another launch
};
enum MatmulForm { kMmForward = 0, kMmRowGrad = 1, kMmWeightGrad = 2 };
// Workspace of a call (0: none): partial tiles and copies of operands that
// would not take 16-byte loads.  Of `a` it reads sizes, strides and flags only.
size_t matmul_workspace_bytes(MatmulForm f, const MatmulArgs& a);
hipError_t launch_matmul(MatmulForm f, MatmulArgs a, void* ws, hipStream_t st);
// A copy with padded rows: out[r] = in[r], widened to `pitch` with zeros.
struct PackJob {
  const uint16_t* in;
  uint16_t* out;             // [rows][pitch], 16-byte aligned
  int64_t ld, rows;
  int width, pitch;
};
// The copies of b and b2 that launch_matmul would make, for a launch of the
// caller's: appended to `jobs`, their places from `to` on (null: sizes only),
// and `a` turned to them.  Returns their bytes.
size_t matmul_pack_jobs(MatmulForm f, MatmulArgs& a, void* to, PackJob* jobs, int& n);
// Forward products of a few rows per group (matmul_stream.hip): whether a call
// is one, and its launch.
constexpr int kMmGatedStreamRows = 48;            // of dense gated products
bool matmul_streams(const MatmulArgs& a);
hipError_t launch_matmul_stream(const MatmulArgs& a, hipStream_t st);
// The instances of one form (matmul_*.hip).
hipError_t launch_matmul_forward(const MatmulArgs& a, hipStream_t st);
hipError_t launch_matmul_row_grad(const MatmulArgs& a, hipStream_t st);
hipError_t launch_matmul_weight_grad(const MatmulArgs& a, hipStream_t st);
hipError_t launch_matmul_gated_forward(const MatmulArgs& a, hipStream_t st);
hipError_t launch_matmul_gated_row_grad(const MatmulArgs& a, hipStream_t st);
hipError_t launch_matmul_gated_weight_grad(const MatmulArgs& a, hipStream_t st);

// g = dy * act'(pre) in the operands' type and, if dbias is set, its column
// sums from the unrounded fp32 values.  g null: sums only.
struct ActGradArgs {
  const uint16_t* dy;
  const uint16_t* pre;       // null with kActNone
  uint16_t* g;               // [rows][ldg], or null; 16-byte aligned, ldg % 8 == 0 and >= n, zeros past n
  int64_t ldg;
  void* dbias;               // [n] or null
  int dbias_f32;
  int64_t ldd, ldp;
  int rows, n, act, f16;
};
size_t act_grad_workspace_bytes(int64_t rows, int64_t n);
hipError_t launch_act_grad(const ActGradArgs& a, void* ws, hipStream_t st);

// ---- 4-bit weights (fp4.hip) ----
// Codes [rows][cols / 2] and exponents [rows][cols / 32] of w [rows][cols].
hipError_t launch_quantize_fp4(const uint16_t* w, long long rows, int cols, int f16, uint8_t* codes, uint8_t* exps,
                               hipStream_t st);
struct Fp4Args {
  MatmulArgs mm;             // the product, forward, without b / b2 / ldb / b_group
  const uint8_t* codes[2];   // [E][n][k / 2]; the second of gated products
  const uint8_t* exps[2];    // [E][n][k / 32]
};
// Workspace of a call (0: none): where many rows share the weights, these are
// widened there once, for the products of 16-bit weights.
size_t fp4_workspace_bytes(const Fp4Args& a);
hipError_t launch_fp4(const Fp4Args& a, void* ws, hipStream_t st);

// g = [dgate | dup] of the gated projections, from dh and the saved products.
struct GatedGradArgs {
  const uint16_t* dh;
  const uint16_t* gate;
  const uint16_t* up;
  uint16_t* g;               // [rows][2 half], 16-byte aligned
  int64_t ldd, ldg, ldu;
  const int32_t* offsets;    // rows outside the groups are left alone; null: all rows
  int E, rows, n;
  int half;                  // dup's first column: n to the next multiple of 64
  int act, f16;
  int n_jobs;                // copies made in the same launch
  PackJob jobs[3];
};
hipError_t launch_gated_grad(const GatedGradArgs& a, hipStream_t st);

// ---- layer norm ----
enum : int { kTypeBf16 = 0, kTypeF16 = 1, kTypeF32 = 2 };
constexpr int kNormMaxCols = 16384;
struct NormArgs {
  const void* x;
  const void* dy;            // backward
  const void* gamma;         // [cols] or null (ones)
  const void* beta;          // [cols] or null (zeros)
  void* out;                 // y | dx (backward: may be null)
  float* mean;               // [rows]; forward: out or null; backward: in (null with rms)
  float* rstd;               // [rows]; forward: out or null; backward: in
  void* dgamma;              // [cols] or null
  void* dbeta;               // [cols] or null
  int64_t ldx, ldd, ldo;
  int rows, cols;
  int type;                  // of x, dy, y, dx
  int param_f32;             // gamma, beta, dgamma, dbeta are fp32 (else of `type`)
  int rms;
  float eps;
};
hipError_t launch_norm_forward(const NormArgs& a, hipStream_t st);
size_t norm_backward_workspace_bytes(int64_t rows, int64_t cols);
hipError_t launch_norm_backward(const NormArgs& a, void* ws, hipStream_t st);

// ---- AdamW ----
struct AdamWTensor {
  void* param;
  const void* grad;
  void* m;                   // fp32, or E4M3 codes
  void* v;                   // fp32, or codes of sqrt(v)
  uint8_t* m_exp;            // 8-bit states: an exponent for every 128 values
  uint8_t* v_exp;
  void* copy;                // or null
  int64_t numel;             // > 0
  uint32_t first_chunk;      // set by launch_adamw
  uint8_t param_type, grad_type, copy_type;
};
constexpr int kAdamWTensors = 48;                 // of a launch: its arguments stay below 4 KB
struct AdamWArgs {
  AdamWTensor tensor[kAdamWTensors];
  int count, step, fp8;
  int chunk;                 // set by launch_adamw: values of a block
  float b1, a1, b2, a2;      // beta1, 1 - beta1, beta2, 1 - beta2
  float keep, size, root;    // 1 - lr decay, lr / (1 - beta1^step), 1 / sqrt(1 - beta2^step)
  float eps;
  double lr, decay, beta1, beta2;
  const float* lr_dev;       // or null: lr
  const int32_t* step_dev;   // or null: step
  const float* grad_scale;   // or null: 1
};
static_assert(sizeof(AdamWArgs) <= 4096, "a kernel's arguments");
hipError_t launch_adamw(AdamWArgs& a, hipStream_t st);

}  // namespace moe
