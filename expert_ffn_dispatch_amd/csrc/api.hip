// C ABI of the MoE FFN layer: argument checks, workspace carving and the
// launch sequence.  Every check runs on the host before anything is enqueued.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <mutex>
#include <string>

#include "../../include/moe_ffn.h"
#include "common.h"
#include "kernels.h"

namespace {

thread_local std::string g_err;
thread_local hipEvent_t g_stage_ev[MOE_STAGE_EVENTS];
thread_local bool g_stage_on = false;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_err = buf;
  return code;
}

int ok() {
  g_err.clear();
  return MOE_OK;
}

int device_error(const char* where, hipError_t e) {
  return fail(MOE_ERR_DEVICE, "%s: %s", where, hipGetErrorString(e));
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define REQ_PTR(p)                                                                        \
  do {                                                                                    \
    if ((p) == nullptr) return fail(MOE_ERR_INVALID, "%s: %s is NULL", fn, #p);          \
    if (!aligned(p)) return fail(MOE_ERR_INVALID, "%s: %s is not 16-byte aligned", fn, #p); \
  } while (0)
#define OPT_PTR(p)                                                                        \
  do {                                                                                    \
    if ((p) != nullptr && !aligned(p))                                                    \
      return fail(MOE_ERR_INVALID, "%s: %s is not 16-byte aligned", fn, #p);             \
  } while (0)

constexpr int kMaxE = 256;
constexpr int kMaxK = 16;

// Shape limits shared by every entry point.  `need_k`: top_k must be valid.
int check_dims(const char* fn, const moe_dims* d, bool need_router_shape) {
  if (d == nullptr) return fail(MOE_ERR_INVALID, "%s: dims is NULL", fn);
  if (d->n_tokens < 1 || d->n_tokens > (1 << 20))
    return fail(MOE_ERR_INVALID, "%s: n_tokens=%d outside [1, 2^20]", fn, d->n_tokens);
  if (d->hidden < 64 || d->hidden > 16384 || d->hidden % 64 != 0)
    return fail(MOE_ERR_INVALID, "%s: hidden=%d must be a multiple of 64 in [64, 16384]", fn, d->hidden);
  if (d->n_experts < 1)
    return fail(MOE_ERR_INVALID, "%s: n_experts=%d must be >= 1", fn, d->n_experts);
  if (d->n_experts > kMaxE)
    return fail(MOE_ERR_UNSUPPORTED, "%s: n_experts=%d above the supported %d", fn, d->n_experts, kMaxE);
  if (d->top_k < 1 || d->top_k > d->n_experts || d->top_k > kMaxK)
    return fail(MOE_ERR_INVALID, "%s: top_k=%d must be in [1, min(n_experts, %d)]", fn, d->top_k, kMaxK);
  if ((long long)d->n_tokens * d->top_k > (1 << 24))
    return fail(MOE_ERR_INVALID, "%s: n_tokens*top_k above 2^24", fn);
  if (need_router_shape) {
    if (d->expert_width < 64 || d->expert_width > 65536 || d->expert_width % 64 != 0)
      return fail(MOE_ERR_INVALID, "%s: expert_width=%d must be a multiple of 64 in [64, 65536]", fn,
                  d->expert_width);
    if (d->n_shared < 0) return fail(MOE_ERR_INVALID, "%s: n_shared=%d < 0", fn, d->n_shared);
    if (d->n_shared > 0) {
      const long long sh = (long long)d->n_shared * d->shared_width;
      if (d->shared_width < 1 || sh > 65536 || sh % 64 != 0)
        return fail(MOE_ERR_INVALID,
                    "%s: n_shared*shared_width=%lld must be a positive multiple of 64 <= 65536", fn, sh);
    }
  }
  return MOE_OK;
}

size_t align_up(size_t v) { return (v + MOE_WORKSPACE_ALIGN - 1) & ~size_t(MOE_WORKSPACE_ALIGN - 1); }

struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  template <class T>
  T* take(size_t n) {
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += align_up(n * sizeof(T));
    return p;
  }
};

struct PermuteWs {
  int32_t* tile_hist;
  int32_t* tile_off;
};
PermuteWs carve_permute(Carver& c, int A, int E) {
  const size_t T = (size_t)moe::ceil_div(A, moe::kPermTile);
  PermuteWs w;
  w.tile_hist = c.take<int32_t>((size_t)E * T);
  w.tile_off = c.take<int32_t>((size_t)E * T);
  return w;
}

struct LayerWs {
  void* route;
  int32_t* ids;
  float* wts;
  int32_t* counts;
  int32_t* offsets;
  int32_t* s2a;
  int32_t* a2s;
  int32_t* row_token;
  float* row_weight;
  int32_t* queue;        // tile queues of the routed and shared gate+up and down launches (zeroed by the permutation)
  PermuteWs perm;
  uint16_t* h;
  uint16_t* y;
  uint16_t* hs;
  uint16_t* ys;
  void* decode;          // single-launch decode path (router partials, barrier words)
  bool has_decode;
};
// The single-launch decode path (decode.hip) is switched off: its first run
// ended the calling process with a segmentation fault inside the layer call,
// before any of its kernels had completed, and the fault has not been traced
// to a cause.  Until it is, decode-sized batches run as separate kernels.
constexpr bool kSingleLaunchDecode = false;

// Shapes the single-launch decode path can take (bf16 weights; FP8 weights
// need a subset of them).
bool decode_shape(const moe_dims& d) {
  return kSingleLaunchDecode && d.n_shared == 0 &&
         moe::decode_fusable(d.n_tokens, d.hidden, d.n_experts, d.top_k, d.expert_width, false);
}
LayerWs carve_layer(Carver& c, const moe_dims& d) {
  const size_t N = d.n_tokens, A = (size_t)d.n_tokens * d.top_k, E = d.n_experts;
  const size_t SH = (size_t)d.n_shared * (d.n_shared > 0 ? d.shared_width : 0);
  LayerWs w;
  w.route = c.take<char>(moe::route_workspace_bytes(d.n_tokens, d.hidden, d.n_experts));
  w.ids = c.take<int32_t>(A);
  w.wts = c.take<float>(A);
  w.counts = c.take<int32_t>(E);
  w.offsets = c.take<int32_t>(E + 1);
  w.s2a = c.take<int32_t>(A);
  w.a2s = c.take<int32_t>(A);
  w.row_token = c.take<int32_t>(A);
  w.row_weight = c.take<float>(A);
  w.queue = c.take<int32_t>(4 * moe::kQueueWords);
  w.perm = carve_permute(c, (int)A, (int)E);
  w.h = c.take<uint16_t>(A * d.expert_width);
  w.y = c.take<uint16_t>(A * d.hidden);
  w.hs = SH ? c.take<uint16_t>(N * SH) : nullptr;
  w.ys = SH ? c.take<uint16_t>(N * d.hidden) : nullptr;
  w.has_decode = decode_shape(d);
  w.decode = w.has_decode ? c.take<char>(moe::decode_workspace_bytes(d.n_tokens, d.hidden, d.n_experts)) : nullptr;
  return w;
}

// Ticks of the device's constant-rate clock in half a second: the longest
// wait of a grid barrier in the single-launch decode path.
uint64_t barrier_limit_ticks() {
  static uint64_t cache[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
  if (cache[dev] == 0) {
    int khz = 0;
    if (hipDeviceGetAttribute(&khz, hipDeviceAttributeWallClockRate, dev) != hipSuccess || khz <= 0) return 0;
    cache[dev] = (uint64_t)khz * 500;
  }
  return cache[dev];
}

int num_cus() {
  static int cache[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return -1;
  if (cache[dev] == 0) {
    int v = 0;
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0)
      return -1;
    cache[dev] = v;
  }
  return cache[dev];
}

int check_ws(const char* fn, void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return MOE_OK;
  if (ws == nullptr) return fail(MOE_ERR_WORKSPACE, "%s: workspace is NULL (%zu bytes needed)", fn, need);
  if (reinterpret_cast<uintptr_t>(ws) % MOE_WORKSPACE_ALIGN != 0)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace must be %d-byte aligned", fn, MOE_WORKSPACE_ALIGN);
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", fn, ws_bytes, need);
  return MOE_OK;
}

// Expert weights of one call: bf16 matrices, or FP8 codes with per-channel
// scales (then the bf16 pointers are NULL).
struct ExpertWeights {
  const uint16_t* gate = nullptr;
  const uint16_t* up = nullptr;
  const uint16_t* down = nullptr;
  const uint8_t* qgate = nullptr;
  const uint8_t* qup = nullptr;
  const uint8_t* qdown = nullptr;
  const float* sgate = nullptr;
  const float* sup = nullptr;
  const float* sdown = nullptr;
};

ExpertWeights bf16_weights(const moe_bf16* g, const moe_bf16* u, const moe_bf16* d) {
  ExpertWeights w;
  w.gate = g;
  w.up = u;
  w.down = d;
  return w;
}

ExpertWeights fp8_weights(const moe_fp8_ffn* f) {
  ExpertWeights w;
  if (f == nullptr) return w;
  w.qgate = f->gate;
  w.qup = f->up;
  w.qdown = f->down;
  w.sgate = f->gate_scale;
  w.sup = f->up_scale;
  w.sdown = f->down_scale;
  return w;
}

moe::FfnArgs gateup_args(const ExpertWeights& w) {
  moe::FfnArgs a{};
  a.w0 = w.gate;
  a.w1 = w.up;
  a.q0 = w.qgate;
  a.q1 = w.qup;
  a.s0 = w.sgate;
  a.s1 = w.sup;
  return a;
}

moe::FfnArgs down_args(const ExpertWeights& w) {
  moe::FfnArgs a{};
  a.w0 = w.down;
  a.q0 = w.qdown;
  a.s0 = w.sdown;
  return a;
}

// An FP8 weight set: every pointer present and aligned.
int check_fp8_ffn(const char* fn, const char* which, const moe_fp8_ffn* f) {
  if (f == nullptr) return fail(MOE_ERR_INVALID, "%s: %s is NULL", fn, which);
  const void* ptrs[6] = {f->gate, f->up, f->down, f->gate_scale, f->up_scale, f->down_scale};
  const char* names[6] = {"gate", "up", "down", "gate_scale", "up_scale", "down_scale"};
  for (int i = 0; i < 6; ++i) {
    if (ptrs[i] == nullptr) return fail(MOE_ERR_INVALID, "%s: %s->%s is NULL", fn, which, names[i]);
    if (!aligned(ptrs[i])) return fail(MOE_ERR_INVALID, "%s: %s->%s is not 16-byte aligned", fn, which, names[i]);
  }
  return MOE_OK;
}

// The FP8 kernels walk the contraction in 256-element chunks.
int check_fp8_dims(const char* fn, const moe_dims* d) {
  if (d->hidden % 256 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: FP8 weights need hidden %% 256 == 0 (hidden=%d)", fn, d->hidden);
  if (d->expert_width % 256 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: FP8 weights need expert_width %% 256 == 0 (expert_width=%d)", fn,
                d->expert_width);
  if (d->n_shared > 0 && (d->n_shared * d->shared_width) % 256 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: FP8 weights need n_shared*shared_width %% 256 == 0", fn);
  return MOE_OK;
}

// Both grouped GEMM phases; the arguments have been checked.
int run_grouped_ffn(const char* fn, const moe_dims* dims, const moe_bf16* x_sorted, const int32_t* expert_offsets,
                    const ExpertWeights& wt, const float* row_scale, moe_bf16* y_sorted, void* ws,
                    hipStream_t st) {
  const int ncu = num_cus();
  if (ncu <= 0) return fail(MOE_ERR_DEVICE, "%s: cannot query the device", fn);
  const int A = dims->n_tokens * dims->top_k;
  Carver c(ws);
  uint16_t* h = c.take<uint16_t>((size_t)A * dims->expert_width);
  int32_t* queue = c.take<int32_t>(2 * moe::kQueueWords);
  moe::FfnArgs g = gateup_args(wt);
  g.queue = queue;
  g.a = x_sorted;
  g.offsets = expert_offsets;
  g.out = h;
  g.E = dims->n_experts;
  g.rows_total = A;
  g.K = dims->hidden;
  g.ncols = dims->expert_width;
  if (hipError_t e = moe::launch_ffn_gateup(g, ncu, st)) return device_error(fn, e);
  moe::FfnArgs dn = down_args(wt);
  dn.queue = queue + moe::kQueueWords;
  dn.a = h;
  dn.offsets = expert_offsets;
  dn.row_scale = row_scale;
  dn.out = y_sorted;
  dn.E = dims->n_experts;
  dn.rows_total = A;
  dn.K = dims->expert_width;
  dn.ncols = dims->hidden;
  if (hipError_t e = moe::launch_ffn_down(dn, ncu, st)) return device_error(fn, e);
  return ok();
}

// Argument rules of the layer entry points other than the weights (checked
// by each caller) and the workspace.
int check_layer_args(const char* fn, uint32_t flags, const moe_bf16* x, const moe_bf16* w_router,
                     const float* router_bias, const int32_t* topk_ids, const float* topk_weights,
                     const moe_bf16* out) {
  if (flags & ~uint32_t(MOE_FLAG_IDS_IN)) return fail(MOE_ERR_INVALID, "%s: unknown flags 0x%x", fn, flags);
  const bool ids_in = (flags & MOE_FLAG_IDS_IN) != 0;
  REQ_PTR(x);
  if (ids_in) {
    if (w_router != nullptr || router_bias != nullptr)
      return fail(MOE_ERR_INVALID, "%s: w_router/router_bias must be NULL with MOE_FLAG_IDS_IN", fn);
    REQ_PTR(topk_ids);
    REQ_PTR(topk_weights);
  } else {
    REQ_PTR(w_router);
    OPT_PTR(router_bias);
    OPT_PTR(topk_ids);
    OPT_PTR(topk_weights);
  }
  REQ_PTR(out);
  return MOE_OK;
}

// Optional cross-stream ordering of a layer's expert GEMMs (shared and
// routed): wait for `before` ahead of the first, record `after` behind the
// last.  Used by the micro-batched layer so that one micro-batch's GEMMs run
// at a time while the small kernels around them overlap.
struct GemmOrder {
  hipEvent_t before = nullptr;
  hipEvent_t after = nullptr;
};

// Enqueue the whole layer on `st`; every argument has been checked and `ws`
// holds carve_layer(dims).  `rec`: record the stage events.
// True while `st` records into a graph (or its state cannot be read).
bool capturing(hipStream_t st) {
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(st, &cs) != hipSuccess) return true;
  return cs != hipStreamCaptureStatusNone;
}

int enqueue_layer(const char* fn, const moe_dims* dims, bool ids_in, const moe_bf16* x, const moe_bf16* w_router,
                  const float* router_bias, const ExpertWeights& routed, const ExpertWeights& shared,
                  int32_t* topk_ids, float* topk_weights, moe_bf16* out, void* ws, hipStream_t st, int ncu,
                  bool rec, const GemmOrder& order) {
  Carver c(ws);
  LayerWs w = carve_layer(c, *dims);
  const int N = dims->n_tokens, M = dims->hidden, E = dims->n_experts, k = dims->top_k, H = dims->expert_width;
  const int A = N * k;
  int32_t* ids = topk_ids ? topk_ids : w.ids;
  float* wts = topk_weights ? topk_weights : w.wts;
  auto mark = [&](int i) -> hipError_t { return rec ? hipEventRecord(g_stage_ev[i], st) : hipSuccess; };

  // Decode-sized batches: the whole layer in one launch (not while per-stage
  // events are wanted, not between the micro-batch streams, and not under
  // stream capture, where the kernels below are recorded instead).
  const bool f8 = routed.qgate != nullptr;
  if (!ids_in && !rec && w.has_decode && order.before == nullptr && order.after == nullptr &&
      moe::decode_fusable(N, M, E, k, H, f8) && !capturing(st)) {
    const uint64_t limit = barrier_limit_ticks();
    if (limit == 0) return fail(MOE_ERR_DEVICE, "%s: cannot query the device clock", fn);
    moe::DecodeArgs da{};
    da.x = x;
    da.w_router = w_router;
    da.bias = router_bias;
    da.N = N;
    da.M = M;
    da.E = E;
    da.k = k;
    da.H = H;
    da.w_gate = routed.gate;
    da.w_up = routed.up;
    da.w_down = routed.down;
    da.q_gate = routed.qgate;
    da.q_up = routed.qup;
    da.q_down = routed.qdown;
    da.s_gate = routed.sgate;
    da.s_up = routed.sup;
    da.s_down = routed.sdown;
    da.ids = ids;
    da.wts = wts;
    da.out = out;
    da.h = w.h;
    da.y = w.y;
    da.limit = limit;
    if (hipError_t e = moe::launch_decode_layer(da, w.decode, ncu, st)) return device_error(fn, e);
    return ok();
  }
  if (hipError_t e = mark(0)) return device_error(fn, e);

  moe::PermuteArgs p{ids, A, E, k, w.counts, w.offsets, w.s2a, w.a2s, w.row_token, wts, w.row_weight,
                     w.perm.tile_hist, w.perm.tile_off, w.queue, 4 * moe::kQueueWords};
  // up to four tokens: the route's top-k launch (one block) also permutes
  const bool route_perm = !ids_in && moe::route_permutes(N);
  if (!ids_in) {
    moe::RouteArgs r{x, w_router, router_bias, N, M, E, k, ids, wts};
    if (route_perm) r.perm = &p;
    if (hipError_t e = moe::launch_route(r, w.route, st)) return device_error(fn, e);
  }
  if (hipError_t e = mark(1)) return device_error(fn, e);
  if (!route_perm) {
    if (hipError_t e = moe::launch_permute(p, st)) return device_error(fn, e);
  }
  if (hipError_t e = mark(2)) return device_error(fn, e);
  if (order.before != nullptr) {
    if (hipError_t e = hipStreamWaitEvent(st, order.before, 0)) return device_error(fn, e);
  }

  // Shared experts: one group of all N rows, gate+up then down.  They go
  // into the routed experts' launches (moe::launch_ffn_*_shared), so the
  // "shared" stage between marks 2 and 3 is empty and its time counts in
  // the gate+up and down stages.
  const bool has_shared = dims->n_shared > 0;
  moe::FfnArgs sg{}, sd{};
  if (has_shared) {
    const int SH = dims->n_shared * dims->shared_width;
    sg = gateup_args(shared);
    sg.a = x;
    sg.fixed_rows = N;
    sg.out = w.hs;
    sg.E = 1;
    sg.rows_total = N;
    sg.K = M;
    sg.ncols = SH;
    sd = down_args(shared);
    sd.a = w.hs;
    sd.fixed_rows = N;
    sd.out = w.ys;
    sd.E = 1;
    sd.rows_total = N;
    sd.K = SH;
    sd.ncols = M;
    sg.queue = w.queue + 2 * moe::kQueueWords;
    sd.queue = w.queue + 3 * moe::kQueueWords;
    sg.queue_zeroed = sd.queue_zeroed = true;
  }
  if (hipError_t e = mark(3)) return device_error(fn, e);
  moe::FfnArgs g = gateup_args(routed);
  g.a = x;
  g.a_rows = w.row_token;
  g.a_nrows = N;
  g.offsets = w.offsets;
  g.out = w.h;
  g.E = E;
  g.rows_total = A;
  g.K = M;
  g.ncols = H;
  g.queue = w.queue;
  g.queue_zeroed = true;
  if (hipError_t e = has_shared ? moe::launch_ffn_gateup_shared(g, sg, ncu, st) : moe::launch_ffn_gateup(g, ncu, st))
    return device_error(fn, e);
  if (hipError_t e = mark(4)) return device_error(fn, e);
  // top-1 routing without shared experts: every token has exactly one row,
  // so the down GEMM stores it straight into the output (the combine would
  // only copy it)
  const bool direct = (k == 1 && dims->n_shared == 0);
  moe::FfnArgs dn = down_args(routed);
  dn.a = w.h;
  dn.offsets = w.offsets;
  dn.row_scale = w.row_weight;
  dn.out = direct ? out : w.y;
  dn.E = E;
  dn.rows_total = A;
  dn.K = H;
  dn.ncols = M;
  dn.out_rows = direct ? w.row_token : nullptr;
  dn.queue = w.queue + moe::kQueueWords;
  dn.queue_zeroed = true;
  if (hipError_t e = has_shared ? moe::launch_ffn_down_shared(dn, sd, ncu, st) : moe::launch_ffn_down(dn, ncu, st))
    return device_error(fn, e);
  if (order.after != nullptr) {
    if (hipError_t e = hipEventRecord(order.after, st)) return device_error(fn, e);
  }
  if (hipError_t e = mark(5)) return device_error(fn, e);

  if (!direct) {
    moe::CombineArgs cb{w.y, w.a2s, nullptr, w.ys, out, N, M, k};
    if (hipError_t e = moe::launch_combine(cb, st)) return device_error(fn, e);
  }
  if (hipError_t e = mark(6)) return device_error(fn, e);
  return ok();
}

// The whole layer; the weight pointers have been checked by the caller.
int run_layer(const char* fn, const moe_dims* dims, uint32_t flags, const moe_bf16* x, const moe_bf16* w_router,
              const float* router_bias, const ExpertWeights& routed, const ExpertWeights& shared,
              int32_t* topk_ids, float* topk_weights, moe_bf16* out, void* ws, size_t ws_bytes,
              moe_stream stream) {
  if (int r = check_layer_args(fn, flags, x, w_router, router_bias, topk_ids, topk_weights, out)) return r;
  Carver sz(nullptr);
  carve_layer(sz, *dims);
  if (int r = check_ws(fn, ws, ws_bytes, sz.off)) return r;
  const int ncu = num_cus();
  if (ncu <= 0) return fail(MOE_ERR_DEVICE, "%s: cannot query the device", fn);
  const bool rec = g_stage_on;
  g_stage_on = false;
  return enqueue_layer(fn, dims, (flags & MOE_FLAG_IDS_IN) != 0, x, w_router, router_bias, routed, shared,
                       topk_ids, topk_weights, out, ws, static_cast<hipStream_t>(stream), ncu, rec, GemmOrder{});
}

// ---------------------------------------------------------------------------
// Micro-batched layer: a second stream per calling thread and device, held
// until the process ends (created on first use, default priority), and the
// events that order work across the two streams.

constexpr int kMaxDevices = 64;
constexpr int kMaxMicro = 64;

struct SideStream {
  hipStream_t stream = nullptr;
  hipEvent_t fork = nullptr;       // caller's stream -> side stream
  hipEvent_t join = nullptr;       // side stream -> caller's stream
  hipEvent_t gemm[2] = {nullptr, nullptr};   // end of a micro-batch's GEMMs, per stream
};
thread_local SideStream g_side[kMaxDevices];

int side_stream(const char* fn, SideStream** out) {
  int dev = 0;
  if (hipError_t e = hipGetDevice(&dev)) return device_error(fn, e);
  if (dev < 0 || dev >= kMaxDevices) return fail(MOE_ERR_UNSUPPORTED, "%s: device %d beyond %d", fn, dev, kMaxDevices);
  SideStream& s = g_side[dev];
  if (s.stream == nullptr) {
    SideStream n;
    if (hipError_t e = hipStreamCreateWithFlags(&n.stream, hipStreamNonBlocking)) return device_error(fn, e);
    hipEvent_t* evs[4] = {&n.fork, &n.join, &n.gemm[0], &n.gemm[1]};
    for (hipEvent_t* ev : evs)
      if (hipError_t e = hipEventCreateWithFlags(ev, hipEventDisableTiming)) return device_error(fn, e);
    s = n;
  }
  *out = &s;
  return MOE_OK;
}

// Token range of micro-batch i of n over N tokens (sizes differ by at most one).
void micro_range(int N, int n, int i, int* start, int* count) {
  const int base = N / n, extra = N % n;
  *start = i * base + (i < extra ? i : extra);
  *count = base + (i < extra ? 1 : 0);
}

moe_dims micro_dims(const moe_dims& d, int n_micro) {
  moe_dims m = d;
  m.n_tokens = (d.n_tokens + n_micro - 1) / n_micro;
  return m;
}

size_t pipelined_ws_bytes(const moe_dims& d, int n_micro) {
  const moe_dims m = micro_dims(d, n_micro);
  Carver c(nullptr);
  carve_layer(c, m);
  return n_micro > 1 ? 2 * c.off : c.off;
}

int run_layer_pipelined(const char* fn, const moe_dims* dims, uint32_t flags, int32_t n_micro, const moe_bf16* x,
                        const moe_bf16* w_router, const float* router_bias, const ExpertWeights& routed,
                        const ExpertWeights& shared, int32_t* topk_ids, float* topk_weights, moe_bf16* out,
                        void* ws, size_t ws_bytes, moe_stream stream) {
  if (n_micro < 1 || n_micro > kMaxMicro || n_micro > dims->n_tokens)
    return fail(MOE_ERR_INVALID, "%s: n_micro=%d must be in [1, min(%d, n_tokens)]", fn, n_micro, kMaxMicro);
  if (int r = check_layer_args(fn, flags, x, w_router, router_bias, topk_ids, topk_weights, out)) return r;
  if (int r = check_ws(fn, ws, ws_bytes, pipelined_ws_bytes(*dims, n_micro))) return r;
  const int ncu = num_cus();
  if (ncu <= 0) return fail(MOE_ERR_DEVICE, "%s: cannot query the device", fn);
  g_stage_on = false;
  const bool ids_in = (flags & MOE_FLAG_IDS_IN) != 0;
  hipStream_t main_st = static_cast<hipStream_t>(stream);
  if (n_micro == 1)
    return enqueue_layer(fn, dims, ids_in, x, w_router, router_bias, routed, shared, topk_ids, topk_weights, out,
                         ws, main_st, ncu, false, GemmOrder{});
  SideStream* side = nullptr;
  if (int r = side_stream(fn, &side)) return r;
  const size_t slot = pipelined_ws_bytes(*dims, n_micro) / 2;
  const int M = dims->hidden, k = dims->top_k;
  if (hipError_t e = hipEventRecord(side->fork, main_st)) return device_error(fn, e);
  if (hipError_t e = hipStreamWaitEvent(side->stream, side->fork, 0)) return device_error(fn, e);
  for (int i = 0; i < n_micro; ++i) {
    int t0 = 0, nt = 0;
    micro_range(dims->n_tokens, n_micro, i, &t0, &nt);
    moe_dims d = *dims;
    d.n_tokens = nt;
    hipStream_t st = (i & 1) ? side->stream : main_st;
    GemmOrder order;
    order.before = i > 0 ? side->gemm[(i - 1) & 1] : nullptr;
    order.after = side->gemm[i & 1];
    void* wsi = static_cast<char*>(ws) + (i & 1) * slot;
    if (int r = enqueue_layer(fn, &d, ids_in, x + (size_t)t0 * M, w_router, router_bias, routed, shared,
                              topk_ids ? topk_ids + (size_t)t0 * k : nullptr,
                              topk_weights ? topk_weights + (size_t)t0 * k : nullptr, out + (size_t)t0 * M, wsi,
                              st, ncu, false, order))
      return r;
  }
  if (hipError_t e = hipEventRecord(side->join, side->stream)) return device_error(fn, e);
  if (hipError_t e = hipStreamWaitEvent(main_st, side->join, 0)) return device_error(fn, e);
  return ok();
}

// Workspace of moe_layer_noalloc: one array per GPU, in the code object's
// device memory.  In host code `scratch` names a host-side stand-in, not the
// device array: its device address comes from hipGetSymbolAddress, once per
// device (with that device current), and only that address is used.
static __device__ __align__(256) unsigned char scratch[MOE_NOALLOC_SCRATCH_BYTES];

std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {nullptr};

int scratch_address(const char* fn, void** ptr) {
  int dev = 0;
  if (hipError_t e = hipGetDevice(&dev)) return device_error(fn, e);
  if (dev < 0 || dev >= kMaxDevices) return fail(MOE_ERR_UNSUPPORTED, "%s: device %d beyond %d", fn, dev, kMaxDevices);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch))) return device_error(fn, e);
    if (p == nullptr) return fail(MOE_ERR_DEVICE, "%s: no device address for the scratch array", fn);
    g_scratch_ptr[dev] = p;
  }
  *ptr = g_scratch_ptr[dev];
  return MOE_OK;
}

// ------------- layer norm, linear layers and products by expert -------------

constexpr int kMaxRows = 1 << 24;
constexpr int kMaxWidth = 65536;
constexpr int64_t kMaxLd = 1 << 20;
constexpr int64_t kMaxTiles = 1 << 22;

static_assert(moe::kTypeBf16 == MOE_DTYPE_BF16 && moe::kTypeF16 == MOE_DTYPE_F16 && moe::kTypeF32 == MOE_DTYPE_F32 &&
                  moe::kActNone == MOE_ACT_NONE && moe::kActRelu == MOE_ACT_RELU && moe::kActGelu == MOE_ACT_GELU &&
                  moe::kActGeluTanh == MOE_ACT_GELU_TANH && moe::kActSilu == MOE_ACT_SILU,
              "the ABI's type and activation codes are the kernels'");

size_t elem_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

// A pointer that is there and has its element's alignment.
#define REQ_ELEM(p, dtype)                                                                \
  do {                                                                                    \
    if ((p) == nullptr) return fail(MOE_ERR_INVALID, "%s: %s is NULL", fn, #p);          \
    OPT_ELEM(p, dtype);                                                                   \
  } while (0)
#define OPT_ELEM(p, dtype)                                                                \
  do {                                                                                    \
    if ((reinterpret_cast<uintptr_t>(p) & (elem_bytes(dtype) - 1)) != 0)                  \
      return fail(MOE_ERR_INVALID, "%s: %s is not aligned to its elements", fn, #p);     \
  } while (0)
// Resolves a row stride: 0 is packed; else width..kMaxLd.
#define REQ_LD(ld, width)                                                                 \
  do {                                                                                    \
    if ((ld) == 0) (ld) = (width);                                                        \
    if ((ld) < (width) || (ld) > kMaxLd)                                                  \
      return fail(MOE_ERR_INVALID, "%s: %s=%lld outside [%lld, 2^20]", fn, #ld, (long long)(ld), (long long)(width)); \
  } while (0)

int check_rows(const char* fn, int rows) {
  if (rows < 0 || rows > kMaxRows) return fail(MOE_ERR_INVALID, "%s: rows=%d outside [0, 2^24]", fn, rows);
  return MOE_OK;
}

// `d` is a copy of the caller's dims, whose strides are resolved here.
int check_norm(const char* fn, moe_norm_dims& d) {
  if (int r = check_rows(fn, d.rows)) return r;
  if (d.cols < 1 || d.cols > moe::kNormMaxCols)
    return fail(MOE_ERR_INVALID, "%s: cols=%d outside [1, %d]", fn, d.cols, moe::kNormMaxCols);
  if (d.dtype < MOE_DTYPE_BF16 || d.dtype > MOE_DTYPE_F32)
    return fail(MOE_ERR_INVALID, "%s: unknown dtype %d", fn, d.dtype);
  if (d.param_dtype != d.dtype && d.param_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_INVALID, "%s: param_dtype=%d must be dtype or MOE_DTYPE_F32", fn, d.param_dtype);
  if (d.flags & ~uint32_t(MOE_NORM_RMS)) return fail(MOE_ERR_INVALID, "%s: unknown flags 0x%x", fn, d.flags);
  if (!(d.eps >= 0.f)) return fail(MOE_ERR_INVALID, "%s: eps must be >= 0", fn);
  REQ_LD(d.ld_x, d.cols);
  REQ_LD(d.ld_y, d.cols);
  REQ_LD(d.ld_dy, d.cols);
  REQ_LD(d.ld_dx, d.cols);
  return MOE_OK;
}

moe::NormArgs norm_args(const moe_norm_dims& d) {
  moe::NormArgs a{};
  a.rows = d.rows;
  a.cols = d.cols;
  a.type = d.dtype;
  a.param_f32 = d.param_dtype == MOE_DTYPE_F32;
  a.rms = (d.flags & MOE_NORM_RMS) != 0;
  a.eps = d.eps;
  a.ldx = d.ld_x;
  return a;
}

int check_product(const char* fn, int rows, int n_in, int n_out, int dtype) {
  if (int r = check_rows(fn, rows)) return r;
  if (n_in < 1 || n_in > kMaxWidth)
    return fail(MOE_ERR_INVALID, "%s: in_features=%d outside [1, %d]", fn, n_in, kMaxWidth);
  if (n_out < 1 || n_out > kMaxWidth)
    return fail(MOE_ERR_INVALID, "%s: out_features=%d outside [1, %d]", fn, n_out, kMaxWidth);
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
    return fail(MOE_ERR_INVALID, "%s: dtype=%d must be bf16 or fp16", fn, dtype);
  return MOE_OK;
}

int check_tiles(const char* fn, int64_t groups, int64_t m, int64_t n) {
  const int64_t t = groups * ((m + 127) / 128) * ((n + 127) / 128);
  if (t > kMaxTiles)
    return fail(MOE_ERR_UNSUPPORTED, "%s: %lld output tiles of 128 x 128, above the supported 2^22", fn, (long long)t);
  return MOE_OK;
}

int check_linear(const char* fn, moe_linear_dims& d) {
  if (int r = check_product(fn, d.rows, d.in_features, d.out_features, d.dtype)) return r;
  if (d.act < MOE_ACT_NONE || d.act > MOE_ACT_SILU) return fail(MOE_ERR_INVALID, "%s: unknown act %d", fn, d.act);
  if (d.bias_dtype != d.dtype && d.bias_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_INVALID, "%s: bias_dtype=%d must be dtype or MOE_DTYPE_F32", fn, d.bias_dtype);
  if (d.dw_dtype != d.dtype && d.dw_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_INVALID, "%s: dw_dtype=%d must be dtype or MOE_DTYPE_F32", fn, d.dw_dtype);
  REQ_LD(d.ld_x, d.in_features);
  REQ_LD(d.ld_w, d.in_features);
  REQ_LD(d.ld_dx, d.in_features);
  REQ_LD(d.ld_residual, d.out_features);
  REQ_LD(d.ld_y, d.out_features);
  REQ_LD(d.ld_pre, d.out_features);
  REQ_LD(d.ld_dy, d.out_features);
  if (int r = check_tiles(fn, 1, d.rows, d.out_features)) return r;
  if (int r = check_tiles(fn, 1, d.rows, d.in_features)) return r;
  return MOE_OK;
}

int check_grouped(const char* fn, moe_grouped_dims& d) {
  if (int r = check_product(fn, d.rows, d.in_features, d.out_features, d.dtype)) return r;
  if (d.n_experts < 1) return fail(MOE_ERR_INVALID, "%s: n_experts=%d must be >= 1", fn, d.n_experts);
  if (d.n_experts > kMaxE)
    return fail(MOE_ERR_UNSUPPORTED, "%s: n_experts=%d above the supported %d", fn, d.n_experts, kMaxE);
  if (d.dw_dtype != d.dtype && d.dw_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_INVALID, "%s: dw_dtype=%d must be dtype or MOE_DTYPE_F32", fn, d.dw_dtype);
  REQ_LD(d.ld_x, d.in_features);
  REQ_LD(d.ld_y, d.out_features);
  // a group's last row tile may be short: one more tile per group
  if (int r = check_tiles(fn, 1, d.rows + 128LL * d.n_experts, d.out_features)) return r;
  if (int r = check_tiles(fn, 1, d.rows + 128LL * d.n_experts, d.in_features)) return r;
  return check_tiles(fn, d.n_experts, d.out_features, d.in_features);
}

// dx = dy w over `rows` rows (grouped where offsets is set); padded: of dy's rows
moe::MatmulArgs row_grad_args(const void* dy, int64_t ld_dy, const void* w, int64_t ld_w, void* dx, int64_t ld_dx,
                              int rows, int n_in, int n_out, int dtype, bool padded = false) {
  moe::MatmulArgs a{};
  a.a = static_cast<const uint16_t*>(dy);
  a.lda = ld_dy;
  a.b = static_cast<const uint16_t*>(w);
  a.ldb = ld_w;
  a.out = dx;
  a.ldo = ld_dx;
  a.E = 1;
  a.rows = a.m = rows;
  a.n = n_in;
  a.k = n_out;
  a.f16 = dtype == MOE_DTYPE_F16;
  a.a_padded = padded;
  return a;
}

moe::MatmulArgs weight_grad_args(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, void* dw, int dw_dtype,
                                 int E, int rows, int n_in, int n_out, int dtype, bool padded = false) {
  moe::MatmulArgs a{};
  a.a = static_cast<const uint16_t*>(dy);
  a.lda = ld_dy;
  a.b = static_cast<const uint16_t*>(x);
  a.ldb = ld_x;
  a.out = dw;
  a.ldo = n_in;
  a.out_group = (int64_t)n_out * n_in;
  a.E = E;
  a.rows = rows;
  a.m = n_out;
  a.n = n_in;
  a.out_f32 = dw_dtype == MOE_DTYPE_F32;
  a.f16 = dtype == MOE_DTYPE_F16;
  a.a_padded = padded;
  return a;
}

int64_t pitch8(int64_t width) { return (width + 7) / 8 * 8; }

moe::MatmulArgs linear_args(const moe_linear_dims& d, const void* x, const void* w, void* y) {
  moe::MatmulArgs a{};
  a.a = static_cast<const uint16_t*>(x);
  a.lda = d.ld_x;
  a.b = static_cast<const uint16_t*>(w);
  a.ldb = d.ld_w;
  a.out = y;
  a.ldo = d.ld_y;
  a.E = 1;
  a.rows = a.m = d.rows;
  a.n = d.out_features;
  a.k = d.in_features;
  a.f16 = d.dtype == MOE_DTYPE_F16;
  // A shape for the kernel for a few rows: no workspace.  (Should only the
  // pointers not suit it, the tiles run without slices and copies.)
  a.whole = d.rows <= 64 && d.in_features % 8 == 0 && d.ld_x % 8 == 0 && d.ld_w % 8 == 0;
  return a;
}

struct LinearBackwardWs {
  uint16_t* g;               // [rows][out to the next multiple of 8], with an activation
  float* sums;               // bias gradient's partial sums
  void* products;            // workspace of either product, one after the other
};
LinearBackwardWs carve_linear_backward(Carver& c, const moe_linear_dims& d) {
  const int64_t R = d.rows, O = d.out_features;
  const bool act = d.act != MOE_ACT_NONE;
  const int64_t ld_g = act ? pitch8(O) : d.ld_dy;
  LinearBackwardWs w;
  w.g = act ? c.take<uint16_t>((size_t)(R * pitch8(O))) : nullptr;
  w.sums = c.take<float>(moe::act_grad_workspace_bytes(R, O) / sizeof(float));
  const size_t a = moe::matmul_workspace_bytes(
      moe::kMmRowGrad, row_grad_args(nullptr, ld_g, nullptr, d.ld_w, nullptr, d.ld_dx, d.rows, d.in_features,
                                     d.out_features, d.dtype, act));
  const size_t b = moe::matmul_workspace_bytes(
      moe::kMmWeightGrad, weight_grad_args(nullptr, ld_g, nullptr, d.ld_x, nullptr, d.dw_dtype, 1, d.rows,
                                           d.in_features, d.out_features, d.dtype, act));
  w.products = c.take<char>(a > b ? a : b);
  return w;
}

size_t linear_ws_bytes(const moe_linear_dims& d) {
  return align_up(moe::matmul_workspace_bytes(moe::kMmForward, linear_args(d, nullptr, nullptr, nullptr)));
}
size_t grouped_wgrad_ws_bytes(const moe_grouped_dims& d) {
  return align_up(moe::matmul_workspace_bytes(
      moe::kMmWeightGrad, weight_grad_args(nullptr, d.ld_y, nullptr, d.ld_x, nullptr, d.dw_dtype, d.n_experts, d.rows,
                                           d.in_features, d.out_features, d.dtype)));
}

int check_gated(const char* fn, moe_gated_dims& d, bool grouped) {
  if (int r = check_rows(fn, d.rows)) return r;
  if (d.width < 1 || d.width > kMaxWidth)
    return fail(MOE_ERR_INVALID, "%s: width=%d outside [1, %d]", fn, d.width, kMaxWidth);
  if (int r = check_product(fn, d.rows, d.in_features, d.width, d.dtype)) return r;
  if (d.n_experts < 1) return fail(MOE_ERR_INVALID, "%s: n_experts=%d must be >= 1", fn, d.n_experts);
  if (!grouped && d.n_experts != 1)
    return fail(MOE_ERR_INVALID, "%s: n_experts=%d must be 1 without groups", fn, d.n_experts);
  if (d.n_experts > kMaxE)
    return fail(MOE_ERR_UNSUPPORTED, "%s: n_experts=%d above the supported %d", fn, d.n_experts, kMaxE);
  if (d.act < MOE_ACT_NONE || d.act > MOE_ACT_SILU) return fail(MOE_ERR_INVALID, "%s: unknown act %d", fn, d.act);
  if (d.dw_dtype != d.dtype && d.dw_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_INVALID, "%s: dw_dtype=%d must be dtype or MOE_DTYPE_F32", fn, d.dw_dtype);
  REQ_LD(d.ld_x, d.in_features);
  REQ_LD(d.ld_dx, d.in_features);
  REQ_LD(d.ld_w, d.in_features);
  REQ_LD(d.ld_h, d.width);
  REQ_LD(d.ld_pre, d.width);
  if (grouped && d.ld_w != d.in_features) return fail(MOE_ERR_INVALID, "%s: grouped weights are packed, ld_w=%lld", fn, (long long)d.ld_w);
  // a group's last row tile may be short: one more tile per group
  const int64_t rows = grouped ? d.rows + 128LL * d.n_experts : d.rows;
  if (int r = check_tiles(fn, 1, rows, 2LL * d.width)) return r;
  if (int r = check_tiles(fn, 1, rows, d.in_features)) return r;
  return check_tiles(fn, 2LL * d.n_experts, d.width, d.in_features);
}

// The two halves of the gradient's buffer, in whole stages of a contraction.
int gated_half(const moe_gated_dims& d) { return (d.width + 63) / 64 * 64; }

moe::MatmulArgs gated_args(const moe_gated_dims& d, bool grouped, const void* x, const void* w_gate, const void* w_up,
                           void* h) {
  moe::MatmulArgs a{};
  a.gated = 1;
  a.a = static_cast<const uint16_t*>(x);
  a.lda = d.ld_x;
  a.b = static_cast<const uint16_t*>(w_gate);
  a.b2 = static_cast<const uint16_t*>(w_up);
  a.ldb = d.ld_w;
  a.b_group = (int64_t)d.width * d.in_features;
  a.out = h;
  a.ldo = d.ld_h;
  a.E = d.n_experts;
  a.rows = a.m = d.rows;
  a.n = d.width;
  a.k = d.in_features;
  a.act = d.act;
  a.f16 = d.dtype == MOE_DTYPE_F16;
  a.whole = !grouped && d.rows <= moe::kMmGatedStreamRows && d.in_features % 8 == 0 && d.ld_x % 8 == 0 && d.ld_w % 8 == 0;
  return a;
}
moe::MatmulArgs gated_row_grad_args(const moe_gated_dims& d, const void* g, const void* w_gate, const void* w_up, void* dx) {
  moe::MatmulArgs a = row_grad_args(g, 2LL * gated_half(d), w_gate, d.ld_w, dx, d.ld_dx, d.rows, d.in_features, d.width,
                                    d.dtype, true);
  a.gated = 1;
  a.E = d.n_experts;
  a.b2 = static_cast<const uint16_t*>(w_up);
  a.b_group = (int64_t)d.width * d.in_features;
  return a;
}
moe::MatmulArgs gated_weight_grad_args(const moe_gated_dims& d, const void* g, const void* x, void* dw_gate, void* dw_up) {
  moe::MatmulArgs a = weight_grad_args(g, 2LL * gated_half(d), x, d.ld_x, dw_gate, d.dw_dtype, 2 * d.n_experts, d.rows,
                                       d.in_features, d.width, d.dtype, true);
  a.gated = a.b2_half = 1;
  a.a_half = gated_half(d);
  a.out2 = dw_up;
  return a;
}
size_t gated_ws_bytes(const moe_gated_dims& d) {
  return align_up(moe::matmul_workspace_bytes(moe::kMmForward, gated_args(d, false, nullptr, nullptr, nullptr, nullptr)));
}
struct GatedBackwardWs {
  uint16_t* g;               // [rows][2 half]: dgate | dup
  void* products;            // workspace of either product, one after the other
};
// Also turns both products' arguments to the padded copies in the workspace
// and lists these: the weights' first, then x's.
GatedBackwardWs carve_gated_backward(Carver& c, const moe_gated_dims& d, moe::MatmulArgs& r, moe::MatmulArgs& g,
                                     moe::PackJob* jobs, int& w_jobs, int& x_jobs) {
  GatedBackwardWs w;
  w.g = c.take<uint16_t>((size_t)d.rows * 2 * gated_half(d));
  r.a = g.a = w.g;
  auto take = [&](moe::MatmulForm f, moe::MatmulArgs& p, moe::PackJob* to, int& n) {
    moe::MatmulArgs sized = p;
    n = 0;
    char* at = c.take<char>(moe::matmul_pack_jobs(f, sized, nullptr, to, n));
    n = 0;
    moe::matmul_pack_jobs(f, p, at, to, n);
  };
  take(moe::kMmRowGrad, r, jobs, w_jobs);
  take(moe::kMmWeightGrad, g, jobs + w_jobs, x_jobs);
  const size_t a = moe::matmul_workspace_bytes(moe::kMmRowGrad, r), b = moe::matmul_workspace_bytes(moe::kMmWeightGrad, g);
  w.products = c.take<char>(a > b ? a : b);
  return w;
}

int run_gated(const char* fn, const moe_gated_dims* dims, bool grouped, const void* x, const int32_t* expert_offsets,
              const void* w_gate, const void* w_up, void* h, void* gate, void* up, void* ws, size_t ws_bytes,
              moe_stream stream) {
  if (dims == nullptr) return fail(MOE_ERR_INVALID, "%s: dims is NULL", fn);
  moe_gated_dims d = *dims;
  if (int r = check_gated(fn, d, grouped)) return r;
  if ((gate == nullptr) != (up == nullptr)) return fail(MOE_ERR_INVALID, "%s: gate and up are saved both or not at all", fn);
  if (d.rows == 0) return ok();
  REQ_ELEM(x, d.dtype);
  if (grouped) REQ_ELEM(expert_offsets, MOE_DTYPE_F32);
  REQ_ELEM(w_gate, d.dtype);
  REQ_ELEM(w_up, d.dtype);
  REQ_ELEM(h, d.dtype);
  OPT_ELEM(gate, d.dtype);
  OPT_ELEM(up, d.dtype);
  for (const void* o : {(const void*)h, (const void*)gate, (const void*)up})
    if (o != nullptr && (o == x || o == w_gate || o == w_up)) return fail(MOE_ERR_INVALID, "%s: an output is an input", fn);
  if (h == gate || h == up || (gate != nullptr && gate == up))
    return fail(MOE_ERR_INVALID, "%s: two outputs are one", fn);
  if (!grouped)
    if (int r = check_ws(fn, ws, ws_bytes, gated_ws_bytes(d))) return r;
  moe::MatmulArgs a = gated_args(d, grouped, x, w_gate, w_up, h);
  a.offsets = expert_offsets;
  a.pre = static_cast<uint16_t*>(gate);
  a.pre2 = static_cast<uint16_t*>(up);
  a.ldp = a.ldp2 = d.ld_pre;
  if (hipError_t e = moe::launch_matmul(moe::kMmForward, a, ws, static_cast<hipStream_t>(stream)))
    return device_error(fn, e);
  return ok();
}

// Any address, for a workspace's size: it goes by whether there are offsets.
const int32_t kSomeOffsets = 0;

// Sizes of a backward call's workspace; the grouped form's products are not
// cut, whatever the offsets say: any address stands for them here.
int gated_backward_ws(const char* fn, const moe_gated_dims* dims, bool grouped, size_t* bytes) {
  if (dims == nullptr) return fail(MOE_ERR_INVALID, "%s: dims is NULL", fn);
  moe_gated_dims d = *dims;
  if (int r = check_gated(fn, d, grouped)) return r;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID, "%s: bytes is NULL", fn);
  Carver c(nullptr);
  moe::MatmulArgs r = gated_row_grad_args(d, nullptr, nullptr, nullptr, nullptr);
  moe::MatmulArgs g = gated_weight_grad_args(d, nullptr, nullptr, nullptr, nullptr);
  r.offsets = g.offsets = grouped ? &kSomeOffsets : nullptr;
  moe::PackJob jobs[3];
  int w_jobs, x_jobs;
  carve_gated_backward(c, d, r, g, jobs, w_jobs, x_jobs);
  *bytes = c.off;
  return ok();
}

int run_gated_backward(const char* fn, const moe_gated_dims* dims, bool grouped, const void* dh, const void* x,
                       const int32_t* expert_offsets, const void* w_gate, const void* w_up, const void* gate,
                       const void* up, void* dx, void* dw_gate, void* dw_up, void* ws, size_t ws_bytes,
                       moe_stream stream) {
  size_t need = 0;
  if (int r = gated_backward_ws(fn, dims, grouped, &need)) return r;
  moe_gated_dims d = *dims;
  if (int r = check_gated(fn, d, grouped)) return r;
  if ((dw_gate == nullptr) != (dw_up == nullptr))
    return fail(MOE_ERR_INVALID, "%s: dw_gate and dw_up are wanted both or not at all", fn);
  if (dx == nullptr && dw_gate == nullptr) return ok();
  if (d.rows > 0) {
    REQ_ELEM(dh, d.dtype);
    REQ_ELEM(gate, d.dtype);
    REQ_ELEM(up, d.dtype);
    if (dw_gate != nullptr) REQ_ELEM(x, d.dtype);
    if (dx != nullptr) {
      REQ_ELEM(w_gate, d.dtype);
      REQ_ELEM(w_up, d.dtype);
    }
  }
  if (grouped) REQ_ELEM(expert_offsets, MOE_DTYPE_F32);
  OPT_ELEM(dx, d.dtype);
  OPT_ELEM(dw_gate, d.dw_dtype);
  OPT_ELEM(dw_up, d.dw_dtype);
  for (const void* o : {(const void*)dx, (const void*)dw_gate, (const void*)dw_up})
    if (o != nullptr && (o == dh || o == x || o == w_gate || o == w_up || o == gate || o == up))
      return fail(MOE_ERR_INVALID, "%s: an output is an input", fn);
  if ((dw_gate != nullptr && dw_gate == dw_up) || (dx != nullptr && (dx == dw_gate || dx == dw_up)))
    return fail(MOE_ERR_INVALID, "%s: two outputs are one", fn);
  if (int r = check_ws(fn, ws, ws_bytes, need)) return r;
  Carver c(ws);
  moe::MatmulArgs row_grad = gated_row_grad_args(d, nullptr, w_gate, w_up, dx);
  moe::MatmulArgs weight_grad = gated_weight_grad_args(d, nullptr, x, dw_gate, dw_up);
  row_grad.offsets = weight_grad.offsets = expert_offsets;
  moe::PackJob jobs[3];
  int w_jobs, x_jobs;
  const GatedBackwardWs b = carve_gated_backward(c, d, row_grad, weight_grad, jobs, w_jobs, x_jobs);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (d.rows > 0) {
    moe::GatedGradArgs g{};
    g.dh = static_cast<const uint16_t*>(dh);
    g.gate = static_cast<const uint16_t*>(gate);
    g.up = static_cast<const uint16_t*>(up);
    g.g = b.g;
    g.ldd = d.ld_h;
    g.ldg = g.ldu = d.ld_pre;
    g.offsets = expert_offsets;
    g.E = d.n_experts;
    g.rows = d.rows;
    g.n = d.width;
    g.half = gated_half(d);
    g.act = d.act;
    g.f16 = d.dtype == MOE_DTYPE_F16;
    for (int i = 0; i < w_jobs + x_jobs; ++i)
      if (i < w_jobs ? dx != nullptr : dw_gate != nullptr) g.jobs[g.n_jobs++] = jobs[i];
    if (hipError_t e = moe::launch_gated_grad(g, st)) return device_error(fn, e);
  }
  if (dx != nullptr)
    if (hipError_t e = moe::launch_matmul(moe::kMmRowGrad, row_grad, b.products, st)) return device_error(fn, e);
  if (dw_gate != nullptr)
    if (hipError_t e = moe::launch_matmul(moe::kMmWeightGrad, weight_grad, b.products, st)) return device_error(fn, e);
  return ok();
}

// ------------------------------------------------------- 4-bit weights

int check_fp4_width(const char* fn, int n_in, int64_t ld_w) {
  if (n_in % 32 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: in_features=%d must be a multiple of 32 with 4-bit weights", fn, n_in);
  if (ld_w != n_in) return fail(MOE_ERR_INVALID, "%s: 4-bit weights are packed, ld_w=%lld", fn, (long long)ld_w);
  return MOE_OK;
}
int check_fp4_matrix(const char* fn, const char* which, const moe_fp4_matrix* w) {
  if (w == nullptr) return fail(MOE_ERR_INVALID, "%s: %s is NULL", fn, which);
  if (w->codes == nullptr || w->exps == nullptr) return fail(MOE_ERR_INVALID, "%s: %s has a NULL array", fn, which);
  if (!aligned(w->codes)) return fail(MOE_ERR_INVALID, "%s: %s's codes are not 16-byte aligned", fn, which);
  return MOE_OK;
}
moe::MatmulArgs grouped_args(const moe_grouped_dims& d, const void* x, const int32_t* expert_offsets, const void* w, void* y) {
  moe::MatmulArgs a{};
  a.a = static_cast<const uint16_t*>(x);
  a.lda = d.ld_x;
  a.b = static_cast<const uint16_t*>(w);
  a.ldb = d.in_features;
  a.b_group = (int64_t)d.out_features * d.in_features;
  a.out = y;
  a.ldo = d.ld_y;
  a.offsets = expert_offsets;
  a.E = d.n_experts;
  a.rows = a.m = d.rows;
  a.n = d.out_features;
  a.k = d.in_features;
  a.f16 = d.dtype == MOE_DTYPE_F16;
  return a;
}
moe::Fp4Args fp4_args(moe::MatmulArgs a, const moe_fp4_matrix* w, const moe_fp4_matrix* w2) {
  moe::Fp4Args f{};
  f.mm = a;
  f.mm.whole = 0;
  if (w != nullptr) {
    f.codes[0] = w->codes;
    f.exps[0] = w->exps;
  }
  if (w2 != nullptr) {
    f.codes[1] = w2->codes;
    f.exps[1] = w2->exps;
  }
  return f;
}
int fp4_bytes(const char* fn, const moe::MatmulArgs& a, size_t* bytes) {
  if (bytes == nullptr) return fail(MOE_ERR_INVALID, "%s: bytes is NULL", fn);
  *bytes = align_up(moe::fp4_workspace_bytes(fp4_args(a, nullptr, nullptr)));
  return ok();
}
int run_fp4(const char* fn, const moe::MatmulArgs& a, const moe_fp4_matrix* w, const moe_fp4_matrix* w2, void* ws,
            size_t ws_bytes, moe_stream stream) {
  const moe::Fp4Args f = fp4_args(a, w, w2);
  if (int r = check_ws(fn, ws, ws_bytes, align_up(moe::fp4_workspace_bytes(f)))) return r;
  if (hipError_t e = moe::launch_fp4(f, ws, static_cast<hipStream_t>(stream))) return device_error(fn, e);
  return ok();
}
int run_gated_fp4(const char* fn, const moe_gated_dims* dims, bool grouped, const void* x, const int32_t* expert_offsets,
                  const moe_fp4_matrix* w_gate, const moe_fp4_matrix* w_up, void* h, void* ws, size_t ws_bytes,
                  moe_stream stream) {
  if (dims == nullptr) return fail(MOE_ERR_INVALID, "%s: dims is NULL", fn);
  moe_gated_dims d = *dims;
  if (int r = check_gated(fn, d, grouped)) return r;
  if (int r = check_fp4_width(fn, d.in_features, d.ld_w)) return r;
  if (d.rows == 0) return ok();
  REQ_ELEM(x, d.dtype);
  if (grouped) REQ_ELEM(expert_offsets, MOE_DTYPE_F32);
  if (int r = check_fp4_matrix(fn, "w_gate", w_gate)) return r;
  if (int r = check_fp4_matrix(fn, "w_up", w_up)) return r;
  REQ_ELEM(h, d.dtype);
  if (h == x) return fail(MOE_ERR_INVALID, "%s: h is x", fn);
  moe::MatmulArgs a = gated_args(d, grouped, x, nullptr, nullptr, h);
  a.offsets = expert_offsets;
  return run_fp4(fn, a, w_gate, w_up, ws, ws_bytes, stream);
}
int gated_fp4_bytes(const char* fn, const moe_gated_dims* dims, bool grouped, size_t* bytes) {
  if (dims == nullptr) return fail(MOE_ERR_INVALID, "%s: dims is NULL", fn);
  moe_gated_dims d = *dims;
  if (int r = check_gated(fn, d, grouped)) return r;
  if (int r = check_fp4_width(fn, d.in_features, d.ld_w)) return r;
  moe::MatmulArgs a = gated_args(d, grouped, nullptr, nullptr, nullptr, nullptr);
  a.offsets = grouped ? &kSomeOffsets : nullptr;
  return fp4_bytes(fn, a, bytes);
}

constexpr int64_t kMaxNumel = 1LL << 36;

int check_adamw(const char* fn, const moe_adamw_args* a, const moe_adamw_tensor* tensors, int count) {
  if (a == nullptr) return fail(MOE_ERR_INVALID, "%s: args is NULL", fn);
  if (a->flags & ~uint32_t(MOE_ADAMW_FP8)) return fail(MOE_ERR_INVALID, "%s: unknown flags 0x%x", fn, a->flags);
  if (!isfinite(a->lr) || !isfinite(a->weight_decay)) return fail(MOE_ERR_INVALID, "%s: lr and weight_decay must be finite", fn);
  if (!(a->beta1 >= 0 && a->beta1 < 1) || !(a->beta2 >= 0 && a->beta2 < 1))
    return fail(MOE_ERR_INVALID, "%s: beta1 and beta2 must be in [0, 1)", fn);
  if (!(a->eps >= 0) || !isfinite(a->eps)) return fail(MOE_ERR_INVALID, "%s: eps must be finite and >= 0", fn);
  if (a->step < 1 && a->step_device == nullptr) return fail(MOE_ERR_INVALID, "%s: step=%d must be >= 1", fn, a->step);
  OPT_ELEM(a->lr_device, MOE_DTYPE_F32);
  OPT_ELEM(a->step_device, MOE_DTYPE_F32);
  OPT_ELEM(a->grad_scale, MOE_DTYPE_F32);
  if (count < 0) return fail(MOE_ERR_INVALID, "%s: count=%d", fn, count);
  if (count > 0 && tensors == nullptr) return fail(MOE_ERR_INVALID, "%s: tensors is NULL", fn);
  const bool fp8 = (a->flags & MOE_ADAMW_FP8) != 0;
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (t.numel < 0 || t.numel > kMaxNumel)
      return fail(MOE_ERR_INVALID, "%s: numel=%lld of tensor %d outside [0, 2^36]", fn, (long long)t.numel, i);
    if (t.param_dtype < MOE_DTYPE_BF16 || t.param_dtype > MOE_DTYPE_F32)
      return fail(MOE_ERR_INVALID, "%s: unknown param_dtype %d of tensor %d", fn, t.param_dtype, i);
    if (t.grad_dtype < MOE_DTYPE_BF16 || t.grad_dtype > MOE_DTYPE_F32)
      return fail(MOE_ERR_INVALID, "%s: unknown grad_dtype %d of tensor %d", fn, t.grad_dtype, i);
    if (t.copy != nullptr && t.copy_dtype != MOE_DTYPE_BF16 && t.copy_dtype != MOE_DTYPE_F16)
      return fail(MOE_ERR_INVALID, "%s: copy_dtype=%d of tensor %d must be bf16 or fp16", fn, t.copy_dtype, i);
    if (t.numel == 0 || t.grad == nullptr) continue;
    REQ_ELEM(t.param, t.param_dtype);
    REQ_ELEM(t.grad, t.grad_dtype);
    OPT_ELEM(t.copy, t.copy_dtype);
    if (t.exp_avg == nullptr || t.exp_avg_sq == nullptr)
      return fail(MOE_ERR_INVALID, "%s: tensor %d has no exp_avg or exp_avg_sq", fn, i);
    if (fp8) {
      if (t.exp_avg_exp == nullptr || t.exp_avg_sq_exp == nullptr)
        return fail(MOE_ERR_INVALID, "%s: tensor %d has no exponents of its 8-bit states", fn, i);
    } else {
      REQ_ELEM(t.exp_avg, MOE_DTYPE_F32);
      REQ_ELEM(t.exp_avg_sq, MOE_DTYPE_F32);
    }
    const void* own[] = {t.param, t.exp_avg, t.exp_avg_sq, t.grad, t.copy};
    for (int x = 0; x < 5; ++x)
      for (int y = 0; y < x; ++y)
        if (own[x] != nullptr && own[x] == own[y]) return fail(MOE_ERR_INVALID, "%s: two arrays of tensor %d are one", fn, i);
  }
  return MOE_OK;
}

// A copy of the caller's dims to resolve strides in.
#define COPY_DIMS(type, d)                                                                \
  if (dims == nullptr) return fail(MOE_ERR_INVALID, "%s: dims is NULL", fn);             \
  type d = *dims

}  // namespace

extern "C" {

int moe_abi_version(void) { return MOE_FFN_ABI_VERSION; }

const char* moe_last_error(void) { return g_err.c_str(); }

int moe_set_stage_events(void* const* events, int n) {
  const char* fn = "moe_set_stage_events";
  if (events == nullptr) {
    g_stage_on = false;
    return ok();
  }
  if (n != MOE_STAGE_EVENTS) return fail(MOE_ERR_INVALID, "%s: n=%d, expected %d", fn, n, MOE_STAGE_EVENTS);
  for (int i = 0; i < n; ++i) {
    if (events[i] == nullptr) return fail(MOE_ERR_INVALID, "%s: events[%d] is NULL", fn, i);
    g_stage_ev[i] = static_cast<hipEvent_t>(events[i]);
  }
  g_stage_on = true;
  return ok();
}

int moe_layer_workspace_bytes(const moe_dims* dims, uint32_t flags, size_t* bytes) {
  const char* fn = "moe_layer_workspace_bytes";
  if (int r = check_dims(fn, dims, true)) return r;
  if (flags & ~uint32_t(MOE_FLAG_IDS_IN)) return fail(MOE_ERR_INVALID, "%s: unknown flags 0x%x", fn, flags);
  if (bytes == nullptr) return fail(MOE_ERR_INVALID, "%s: bytes is NULL", fn);
  Carver c(nullptr);
  carve_layer(c, *dims);
  *bytes = c.off;
  return ok();
}

int moe_layer_single_launch(const moe_dims* dims, uint32_t flags, int fp8, int* single) {
  const char* fn = "moe_layer_single_launch";
  if (int r = check_dims(fn, dims, true)) return r;
  if (flags & ~uint32_t(MOE_FLAG_IDS_IN)) return fail(MOE_ERR_INVALID, "%s: unknown flags 0x%x", fn, flags);
  if (single == nullptr) return fail(MOE_ERR_INVALID, "%s: single is NULL", fn);
  *single = ((flags & MOE_FLAG_IDS_IN) == 0 && decode_shape(*dims) &&
             moe::decode_fusable(dims->n_tokens, dims->hidden, dims->n_experts, dims->top_k, dims->expert_width,
                                 fp8 != 0))
                ? 1
                : 0;
  return ok();
}

int moe_route_workspace_bytes(const moe_dims* dims, size_t* bytes) {
  const char* fn = "moe_route_workspace_bytes";
  if (int r = check_dims(fn, dims, false)) return r;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID, "%s: bytes is NULL", fn);
  *bytes = moe::route_workspace_bytes(dims->n_tokens, dims->hidden, dims->n_experts);
  return ok();
}

int moe_permute_workspace_bytes(const moe_dims* dims, size_t* bytes) {
  const char* fn = "moe_permute_workspace_bytes";
  if (int r = check_dims(fn, dims, false)) return r;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID, "%s: bytes is NULL", fn);
  Carver c(nullptr);
  carve_permute(c, dims->n_tokens * dims->top_k, dims->n_experts);
  *bytes = c.off;
  return ok();
}

int moe_grouped_ffn_workspace_bytes(const moe_dims* dims, size_t* bytes) {
  const char* fn = "moe_grouped_ffn_workspace_bytes";
  if (int r = check_dims(fn, dims, true)) return r;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID, "%s: bytes is NULL", fn);
  Carver c(nullptr);
  c.take<uint16_t>((size_t)dims->n_tokens * dims->top_k * dims->expert_width);
  c.take<int32_t>(2 * moe::kQueueWords);
  *bytes = c.off;
  return ok();
}

int moe_route(const moe_dims* dims, const moe_bf16* x, const moe_bf16* w_router,
              const float* router_bias, int32_t* topk_ids, float* topk_weights, void* ws, size_t ws_bytes,
              moe_stream stream) {
  const char* fn = "moe_route";
  if (int r = check_dims(fn, dims, false)) return r;
  REQ_PTR(x);
  REQ_PTR(w_router);
  OPT_PTR(router_bias);
  REQ_PTR(topk_ids);
  REQ_PTR(topk_weights);
  if (int r = check_ws(fn, ws, ws_bytes, moe::route_workspace_bytes(dims->n_tokens, dims->hidden, dims->n_experts)))
    return r;
  moe::RouteArgs a{x, w_router, router_bias, dims->n_tokens, dims->hidden, dims->n_experts, dims->top_k,
                   topk_ids, topk_weights};
  if (hipError_t e = moe::launch_route(a, ws, static_cast<hipStream_t>(stream))) return device_error(fn, e);
  return ok();
}

int moe_permute(const moe_dims* dims, const int32_t* topk_ids, const moe_bf16* x, int32_t* expert_counts,
                int32_t* expert_offsets, int32_t* sorted_to_assign, int32_t* assign_to_sorted,
                moe_bf16* x_sorted, void* ws, size_t ws_bytes, moe_stream stream) {
  const char* fn = "moe_permute";
  if (int r = check_dims(fn, dims, false)) return r;
  REQ_PTR(topk_ids);
  REQ_PTR(expert_counts);
  REQ_PTR(expert_offsets);
  REQ_PTR(sorted_to_assign);
  REQ_PTR(assign_to_sorted);
  OPT_PTR(x_sorted);
  if (x_sorted != nullptr) REQ_PTR(x);
  const int A = dims->n_tokens * dims->top_k;
  Carver sz(nullptr);
  carve_permute(sz, A, dims->n_experts);
  if (int r = check_ws(fn, ws, ws_bytes, sz.off)) return r;
  Carver c(ws);
  PermuteWs w = carve_permute(c, A, dims->n_experts);
  hipStream_t st = static_cast<hipStream_t>(stream);
  moe::PermuteArgs p{topk_ids, A, dims->n_experts, dims->top_k, expert_counts, expert_offsets,
                     sorted_to_assign, assign_to_sorted, nullptr, nullptr, nullptr, w.tile_hist, w.tile_off};
  if (hipError_t e = moe::launch_permute(p, st)) return device_error(fn, e);
  if (x_sorted != nullptr) {
    if (hipError_t e = moe::launch_gather(x, sorted_to_assign, dims->top_k, A, dims->hidden, x_sorted, st))
      return device_error(fn, e);
  }
  return ok();
}

int moe_grouped_ffn(const moe_dims* dims, const moe_bf16* x_sorted, const int32_t* expert_offsets,
                    const moe_bf16* w_gate, const moe_bf16* w_up, const moe_bf16* w_down,
                    const float* row_scale, moe_bf16* y_sorted, void* ws, size_t ws_bytes, moe_stream stream) {
  const char* fn = "moe_grouped_ffn";
  if (int r = check_dims(fn, dims, true)) return r;
  REQ_PTR(x_sorted);
  REQ_PTR(expert_offsets);
  REQ_PTR(w_gate);
  REQ_PTR(w_up);
  REQ_PTR(w_down);
  OPT_PTR(row_scale);
  REQ_PTR(y_sorted);
  size_t need = 0;
  moe_grouped_ffn_workspace_bytes(dims, &need);
  if (int r = check_ws(fn, ws, ws_bytes, need)) return r;
  return run_grouped_ffn(fn, dims, x_sorted, expert_offsets, bf16_weights(w_gate, w_up, w_down), row_scale,
                         y_sorted, ws, static_cast<hipStream_t>(stream));
}

int moe_grouped_ffn_fp8(const moe_dims* dims, const moe_bf16* x_sorted, const int32_t* expert_offsets,
                        const moe_fp8_ffn* experts, const float* row_scale, moe_bf16* y_sorted, void* ws,
                        size_t ws_bytes, moe_stream stream) {
  const char* fn = "moe_grouped_ffn_fp8";
  if (int r = check_dims(fn, dims, true)) return r;
  if (int r = check_fp8_dims(fn, dims)) return r;
  REQ_PTR(x_sorted);
  REQ_PTR(expert_offsets);
  if (int r = check_fp8_ffn(fn, "experts", experts)) return r;
  OPT_PTR(row_scale);
  REQ_PTR(y_sorted);
  size_t need = 0;
  moe_grouped_ffn_workspace_bytes(dims, &need);
  if (int r = check_ws(fn, ws, ws_bytes, need)) return r;
  return run_grouped_ffn(fn, dims, x_sorted, expert_offsets, fp8_weights(experts), row_scale, y_sorted, ws,
                         static_cast<hipStream_t>(stream));
}

int moe_quantize_fp8(const moe_bf16* w, int64_t rows, int32_t cols, moe_fp8* q, float* scale,
                     moe_stream stream) {
  const char* fn = "moe_quantize_fp8";
  if (rows < 1 || rows > (int64_t(1) << 26))
    return fail(MOE_ERR_INVALID, "%s: rows=%lld outside [1, 2^26]", fn, (long long)rows);
  if (cols < 64 || cols > 65536 || cols % 64 != 0)
    return fail(MOE_ERR_INVALID, "%s: cols=%d must be a multiple of 64 in [64, 65536]", fn, cols);
  REQ_PTR(w);
  REQ_PTR(q);
  REQ_PTR(scale);
  if (hipError_t e = moe::launch_quantize_fp8(w, rows, cols, q, scale, static_cast<hipStream_t>(stream)))
    return device_error(fn, e);
  return ok();
}

int moe_combine(const moe_dims* dims, const moe_bf16* y_sorted, const int32_t* assign_to_sorted,
                const float* topk_weights, const moe_bf16* shared_out, moe_bf16* out, moe_stream stream) {
  const char* fn = "moe_combine";
  if (int r = check_dims(fn, dims, false)) return r;
  REQ_PTR(y_sorted);
  REQ_PTR(assign_to_sorted);
  OPT_PTR(topk_weights);
  OPT_PTR(shared_out);
  REQ_PTR(out);
  moe::CombineArgs a{y_sorted, assign_to_sorted, topk_weights, shared_out, out, dims->n_tokens,
                     dims->hidden, dims->top_k};
  if (hipError_t e = moe::launch_combine(a, static_cast<hipStream_t>(stream))) return device_error(fn, e);
  return ok();
}

int moe_layer(const moe_dims* dims, uint32_t flags, const moe_bf16* x, const moe_bf16* w_router,
              const float* router_bias, const moe_bf16* w_gate, const moe_bf16* w_up, const moe_bf16* w_down,
              const moe_bf16* ws_gate, const moe_bf16* ws_up, const moe_bf16* ws_down, int32_t* topk_ids,
              float* topk_weights, moe_bf16* out, void* ws, size_t ws_bytes, moe_stream stream) {
  const char* fn = "moe_layer";
  if (int r = check_dims(fn, dims, true)) return r;
  REQ_PTR(w_gate);
  REQ_PTR(w_up);
  REQ_PTR(w_down);
  if (dims->n_shared > 0) {
    REQ_PTR(ws_gate);
    REQ_PTR(ws_up);
    REQ_PTR(ws_down);
  } else if (ws_gate || ws_up || ws_down) {
    return fail(MOE_ERR_INVALID, "%s: shared-expert weights given with n_shared = 0", fn);
  }
  return run_layer(fn, dims, flags, x, w_router, router_bias, bf16_weights(w_gate, w_up, w_down),
                   bf16_weights(ws_gate, ws_up, ws_down), topk_ids, topk_weights, out, ws, ws_bytes, stream);
}

int moe_layer_noalloc(const moe_dims* dims, uint32_t flags, const moe_bf16* x, const moe_bf16* w_router,
                      const float* router_bias, const moe_bf16* w_gate, const moe_bf16* w_up,
                      const moe_bf16* w_down, const moe_bf16* ws_gate, const moe_bf16* ws_up,
                      const moe_bf16* ws_down, int32_t* topk_ids, float* topk_weights, moe_bf16* out,
                      moe_stream stream) {
  const char* fn = "moe_layer_noalloc";
  if (int r = check_dims(fn, dims, true)) return r;
  REQ_PTR(w_gate);
  REQ_PTR(w_up);
  REQ_PTR(w_down);
  if (dims->n_shared > 0) {
    REQ_PTR(ws_gate);
    REQ_PTR(ws_up);
    REQ_PTR(ws_down);
  } else if (ws_gate || ws_up || ws_down) {
    return fail(MOE_ERR_INVALID, "%s: shared-expert weights given with n_shared = 0", fn);
  }
  if (int r = check_layer_args(fn, flags, x, w_router, router_bias, topk_ids, topk_weights, out)) return r;
  Carver sz(nullptr);
  carve_layer(sz, *dims);
  if (sz.off > MOE_NOALLOC_SCRATCH_BYTES)
    return fail(MOE_ERR_WORKSPACE, "%s: this shape needs %zu bytes of workspace, above the %zu of the library's "
                "scratch array (use moe_layer with a workspace)", fn, sz.off, (size_t)MOE_NOALLOC_SCRATCH_BYTES);
  void* ptr = nullptr;
  if (int r = scratch_address(fn, &ptr)) return r;
  return run_layer(fn, dims, flags, x, w_router, router_bias, bf16_weights(w_gate, w_up, w_down),
                   bf16_weights(ws_gate, ws_up, ws_down), topk_ids, topk_weights, out, ptr,
                   MOE_NOALLOC_SCRATCH_BYTES, stream);
}

int moe_layer_fp8(const moe_dims* dims, uint32_t flags, const moe_bf16* x, const moe_bf16* w_router,
                  const float* router_bias, const moe_fp8_ffn* experts, const moe_fp8_ffn* shared,
                  int32_t* topk_ids, float* topk_weights, moe_bf16* out, void* ws, size_t ws_bytes,
                  moe_stream stream) {
  const char* fn = "moe_layer_fp8";
  if (int r = check_dims(fn, dims, true)) return r;
  if (int r = check_fp8_dims(fn, dims)) return r;
  if (int r = check_fp8_ffn(fn, "experts", experts)) return r;
  if (dims->n_shared > 0) {
    if (int r = check_fp8_ffn(fn, "shared", shared)) return r;
  } else if (shared != nullptr) {
    return fail(MOE_ERR_INVALID, "%s: shared-expert weights given with n_shared = 0", fn);
  }
  return run_layer(fn, dims, flags, x, w_router, router_bias, fp8_weights(experts), fp8_weights(shared),
                   topk_ids, topk_weights, out, ws, ws_bytes, stream);
}

int moe_layer_pipelined_workspace_bytes(const moe_dims* dims, uint32_t flags, int32_t n_micro, size_t* bytes) {
  const char* fn = "moe_layer_pipelined_workspace_bytes";
  if (int r = check_dims(fn, dims, true)) return r;
  if (flags & ~uint32_t(MOE_FLAG_IDS_IN)) return fail(MOE_ERR_INVALID, "%s: unknown flags 0x%x", fn, flags);
  if (n_micro < 1 || n_micro > kMaxMicro || n_micro > dims->n_tokens)
    return fail(MOE_ERR_INVALID, "%s: n_micro=%d must be in [1, min(%d, n_tokens)]", fn, n_micro, kMaxMicro);
  if (bytes == nullptr) return fail(MOE_ERR_INVALID, "%s: bytes is NULL", fn);
  *bytes = pipelined_ws_bytes(*dims, n_micro);
  return ok();
}

int moe_layer_pipelined(const moe_dims* dims, uint32_t flags, int32_t n_micro, const moe_bf16* x,
                        const moe_bf16* w_router, const float* router_bias, const moe_bf16* w_gate,
                        const moe_bf16* w_up, const moe_bf16* w_down, const moe_bf16* ws_gate,
                        const moe_bf16* ws_up, const moe_bf16* ws_down, int32_t* topk_ids, float* topk_weights,
                        moe_bf16* out, void* ws, size_t ws_bytes, moe_stream stream) {
  const char* fn = "moe_layer_pipelined";
  if (int r = check_dims(fn, dims, true)) return r;
  REQ_PTR(w_gate);
  REQ_PTR(w_up);
  REQ_PTR(w_down);
  if (dims->n_shared > 0) {
    REQ_PTR(ws_gate);
    REQ_PTR(ws_up);
    REQ_PTR(ws_down);
  } else if (ws_gate || ws_up || ws_down) {
    return fail(MOE_ERR_INVALID, "%s: shared-expert weights given with n_shared = 0", fn);
  }
  return run_layer_pipelined(fn, dims, flags, n_micro, x, w_router, router_bias, bf16_weights(w_gate, w_up, w_down),
                             bf16_weights(ws_gate, ws_up, ws_down), topk_ids, topk_weights, out, ws, ws_bytes,
                             stream);
}

int moe_layer_norm(const moe_norm_dims* dims, const void* x, const void* gamma, const void* beta, void* y,
                   float* mean, float* rstd, moe_stream stream) {
  const char* fn = "moe_layer_norm";
  COPY_DIMS(moe_norm_dims, d);
  if (int r = check_norm(fn, d)) return r;
  if (d.rows == 0) return ok();
  REQ_ELEM(x, d.dtype);
  OPT_ELEM(gamma, d.param_dtype);
  OPT_ELEM(beta, d.param_dtype);
  REQ_ELEM(y, d.dtype);
  OPT_ELEM(mean, MOE_DTYPE_F32);
  OPT_ELEM(rstd, MOE_DTYPE_F32);
  if (y == x && d.ld_y != d.ld_x) return fail(MOE_ERR_INVALID, "%s: y is x with another row stride", fn);
  moe::NormArgs a = norm_args(d);
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.out = y;
  a.ldo = d.ld_y;
  a.mean = mean;
  a.rstd = rstd;
  if (hipError_t e = moe::launch_norm_forward(a, static_cast<hipStream_t>(stream))) return device_error(fn, e);
  return ok();
}

int moe_layer_norm_backward_workspace_bytes(const moe_norm_dims* dims, size_t* bytes) {
  const char* fn = "moe_layer_norm_backward_workspace_bytes";
  COPY_DIMS(moe_norm_dims, d);
  if (int r = check_norm(fn, d)) return r;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID, "%s: bytes is NULL", fn);
  *bytes = align_up(moe::norm_backward_workspace_bytes(d.rows, d.cols));
  return ok();
}

int moe_layer_norm_backward(const moe_norm_dims* dims, const void* dy, const void* x, const void* gamma,
                            const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta, void* ws,
                            size_t ws_bytes, moe_stream stream) {
  const char* fn = "moe_layer_norm_backward";
  COPY_DIMS(moe_norm_dims, d);
  if (int r = check_norm(fn, d)) return r;
  const bool rms = (d.flags & MOE_NORM_RMS) != 0;
  if (d.rows > 0) {
    REQ_ELEM(dy, d.dtype);
    REQ_ELEM(x, d.dtype);
    if (!rms) REQ_ELEM(mean, MOE_DTYPE_F32);
    REQ_ELEM(rstd, MOE_DTYPE_F32);
  }
  OPT_ELEM(gamma, d.param_dtype);
  OPT_ELEM(dx, d.dtype);
  OPT_ELEM(dgamma, d.param_dtype);
  OPT_ELEM(dbeta, d.param_dtype);
  if (dx != nullptr && ((dx == x && d.ld_dx != d.ld_x) || (dx == dy && d.ld_dx != d.ld_dy)))
    return fail(MOE_ERR_INVALID, "%s: dx is x or dy with another row stride", fn);
  if (dgamma != nullptr || dbeta != nullptr) {
    if (int r = check_ws(fn, ws, ws_bytes, align_up(moe::norm_backward_workspace_bytes(d.rows, d.cols)))) return r;
  } else if (dx == nullptr) {
    return ok();
  }
  moe::NormArgs a = norm_args(d);
  a.x = x;
  a.dy = dy;
  a.ldd = d.ld_dy;
  a.gamma = gamma;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.out = dx;
  a.ldo = d.ld_dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  if (hipError_t e = moe::launch_norm_backward(a, ws, static_cast<hipStream_t>(stream))) return device_error(fn, e);
  return ok();
}

int moe_linear_workspace_bytes(const moe_linear_dims* dims, size_t* bytes) {
  const char* fn = "moe_linear_workspace_bytes";
  COPY_DIMS(moe_linear_dims, d);
  if (int r = check_linear(fn, d)) return r;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID, "%s: bytes is NULL", fn);
  *bytes = linear_ws_bytes(d);
  return ok();
}

int moe_linear(const moe_linear_dims* dims, const void* x, const void* w, const void* bias, const void* residual,
               void* y, void* pre, void* ws, size_t ws_bytes, moe_stream stream) {
  const char* fn = "moe_linear";
  COPY_DIMS(moe_linear_dims, d);
  if (int r = check_linear(fn, d)) return r;
  if (d.rows == 0) return ok();
  REQ_ELEM(x, d.dtype);
  REQ_ELEM(w, d.dtype);
  OPT_ELEM(bias, d.bias_dtype);
  OPT_ELEM(residual, d.dtype);
  REQ_ELEM(y, d.dtype);
  OPT_ELEM(pre, d.dtype);
  if (y == x || y == w || (pre != nullptr && (pre == x || pre == w || pre == y || pre == residual)))
    return fail(MOE_ERR_INVALID, "%s: an output is an input (only residual may be y)", fn);
  if (residual == y && d.ld_residual != d.ld_y)
    return fail(MOE_ERR_INVALID, "%s: residual is y with another row stride", fn);
  if (int r = check_ws(fn, ws, ws_bytes, linear_ws_bytes(d))) return r;
  moe::MatmulArgs a = linear_args(d, x, w, y);
  a.bias = bias;
  a.bias_f32 = d.bias_dtype == MOE_DTYPE_F32;
  a.act = d.act;
  a.residual = static_cast<const uint16_t*>(residual);
  a.ldr = d.ld_residual;
  a.pre = static_cast<uint16_t*>(pre);
  a.ldp = d.ld_pre;
  if (hipError_t e = moe::launch_matmul(moe::kMmForward, a, ws, static_cast<hipStream_t>(stream)))
    return device_error(fn, e);
  return ok();
}

int moe_linear_backward_workspace_bytes(const moe_linear_dims* dims, size_t* bytes) {
  const char* fn = "moe_linear_backward_workspace_bytes";
  COPY_DIMS(moe_linear_dims, d);
  if (int r = check_linear(fn, d)) return r;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID, "%s: bytes is NULL", fn);
  Carver c(nullptr);
  carve_linear_backward(c, d);
  *bytes = c.off;
  return ok();
}

int moe_linear_backward(const moe_linear_dims* dims, const void* dy, const void* x, const void* w, const void* pre,
                        void* dx, void* dw, void* dbias, void* ws, size_t ws_bytes, moe_stream stream) {
  const char* fn = "moe_linear_backward";
  COPY_DIMS(moe_linear_dims, d);
  if (int r = check_linear(fn, d)) return r;
  const bool act = d.act != MOE_ACT_NONE;
  if (!act && pre != nullptr) return fail(MOE_ERR_INVALID, "%s: pre must be NULL with MOE_ACT_NONE", fn);
  if (d.rows > 0) {
    REQ_ELEM(dy, d.dtype);
    if (act) REQ_ELEM(pre, d.dtype);
    if (dw != nullptr) REQ_ELEM(x, d.dtype);
    if (dx != nullptr) REQ_ELEM(w, d.dtype);
  }
  OPT_ELEM(dx, d.dtype);
  OPT_ELEM(dw, d.dw_dtype);
  OPT_ELEM(dbias, d.bias_dtype);
  if ((dx != nullptr && (dx == dy || dx == w || dx == x || dx == pre)) ||
      (dw != nullptr && (dw == w || dw == x || dw == dy || dw == pre)))
    return fail(MOE_ERR_INVALID, "%s: an output is an input", fn);
  if (dx == nullptr && dw == nullptr && dbias == nullptr) return ok();
  Carver sz(nullptr);
  carve_linear_backward(sz, d);
  if (int r = check_ws(fn, ws, ws_bytes, sz.off)) return r;
  Carver c(ws);
  LinearBackwardWs b = carve_linear_backward(c, d);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool products = dx != nullptr || dw != nullptr;
  const void* g = dy;
  int64_t ld_g = d.ld_dy;
  if (dbias != nullptr || (act && products && d.rows > 0)) {
    moe::ActGradArgs a{};
    a.dy = static_cast<const uint16_t*>(dy);
    a.ldd = d.ld_dy;
    a.pre = static_cast<const uint16_t*>(pre);
    a.ldp = d.ld_pre;
    a.g = act && products ? b.g : nullptr;
    a.ldg = pitch8(d.out_features);
    a.dbias = dbias;
    a.dbias_f32 = d.bias_dtype == MOE_DTYPE_F32;
    a.rows = d.rows;
    a.n = d.out_features;
    a.act = d.act;
    a.f16 = d.dtype == MOE_DTYPE_F16;
    if (hipError_t e = moe::launch_act_grad(a, b.sums, st)) return device_error(fn, e);
  }
  if (act) {
    g = b.g;
    ld_g = pitch8(d.out_features);
  }
  if (dx != nullptr) {
    const moe::MatmulArgs a = row_grad_args(g, ld_g, w, d.ld_w, dx, d.ld_dx, d.rows, d.in_features, d.out_features, d.dtype, act);
    if (hipError_t e = moe::launch_matmul(moe::kMmRowGrad, a, b.products, st)) return device_error(fn, e);
  }
  if (dw != nullptr) {
    const moe::MatmulArgs a =
        weight_grad_args(g, ld_g, x, d.ld_x, dw, d.dw_dtype, 1, d.rows, d.in_features, d.out_features, d.dtype, act);
    if (hipError_t e = moe::launch_matmul(moe::kMmWeightGrad, a, b.products, st)) return device_error(fn, e);
  }
  return ok();
}

int moe_grouped_matmul(const moe_grouped_dims* dims, const void* x, const int32_t* expert_offsets, const void* w,
                       void* y, moe_stream stream) {
  const char* fn = "moe_grouped_matmul";
  COPY_DIMS(moe_grouped_dims, d);
  if (int r = check_grouped(fn, d)) return r;
  if (d.rows == 0) return ok();
  REQ_ELEM(x, d.dtype);
  REQ_ELEM(expert_offsets, MOE_DTYPE_F32);
  REQ_ELEM(w, d.dtype);
  REQ_ELEM(y, d.dtype);
  if (y == x || y == w) return fail(MOE_ERR_INVALID, "%s: y is an input", fn);
  const moe::MatmulArgs a = grouped_args(d, x, expert_offsets, w, y);
  if (hipError_t e = moe::launch_matmul(moe::kMmForward, a, nullptr, static_cast<hipStream_t>(stream)))
    return device_error(fn, e);
  return ok();
}

int moe_grouped_matmul_dgrad(const moe_grouped_dims* dims, const void* dy, const int32_t* expert_offsets,
                             const void* w, void* dx, moe_stream stream) {
  const char* fn = "moe_grouped_matmul_dgrad";
  COPY_DIMS(moe_grouped_dims, d);
  if (int r = check_grouped(fn, d)) return r;
  if (d.rows == 0) return ok();
  REQ_ELEM(dy, d.dtype);
  REQ_ELEM(expert_offsets, MOE_DTYPE_F32);
  REQ_ELEM(w, d.dtype);
  REQ_ELEM(dx, d.dtype);
  if (dx == dy || dx == w) return fail(MOE_ERR_INVALID, "%s: dx is an input", fn);
  moe::MatmulArgs a = row_grad_args(dy, d.ld_y, w, d.in_features, dx, d.ld_x, d.rows, d.in_features, d.out_features, d.dtype);
  a.b_group = (int64_t)d.out_features * d.in_features;
  a.offsets = expert_offsets;
  a.E = d.n_experts;
  if (hipError_t e = moe::launch_matmul(moe::kMmRowGrad, a, nullptr, static_cast<hipStream_t>(stream)))
    return device_error(fn, e);
  return ok();
}

int moe_grouped_matmul_wgrad_workspace_bytes(const moe_grouped_dims* dims, size_t* bytes) {
  const char* fn = "moe_grouped_matmul_wgrad_workspace_bytes";
  COPY_DIMS(moe_grouped_dims, d);
  if (int r = check_grouped(fn, d)) return r;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID, "%s: bytes is NULL", fn);
  *bytes = grouped_wgrad_ws_bytes(d);
  return ok();
}

int moe_grouped_matmul_wgrad(const moe_grouped_dims* dims, const void* dy, const void* x,
                             const int32_t* expert_offsets, void* dw, void* ws, size_t ws_bytes, moe_stream stream) {
  const char* fn = "moe_grouped_matmul_wgrad";
  COPY_DIMS(moe_grouped_dims, d);
  if (int r = check_grouped(fn, d)) return r;
  if (d.rows > 0) {
    REQ_ELEM(dy, d.dtype);
    REQ_ELEM(x, d.dtype);
  }
  REQ_ELEM(expert_offsets, MOE_DTYPE_F32);
  REQ_ELEM(dw, d.dw_dtype);
  if (dw == dy || dw == x) return fail(MOE_ERR_INVALID, "%s: dw is an input", fn);
  if (int r = check_ws(fn, ws, ws_bytes, grouped_wgrad_ws_bytes(d))) return r;
  moe::MatmulArgs a = weight_grad_args(dy, d.ld_y, x, d.ld_x, dw, d.dw_dtype, d.n_experts, d.rows, d.in_features,
                                       d.out_features, d.dtype);
  a.offsets = expert_offsets;
  if (hipError_t e = moe::launch_matmul(moe::kMmWeightGrad, a, ws, static_cast<hipStream_t>(stream)))
    return device_error(fn, e);
  return ok();
}

int moe_gated_linear_workspace_bytes(const moe_gated_dims* dims, size_t* bytes) {
  const char* fn = "moe_gated_linear_workspace_bytes";
  COPY_DIMS(moe_gated_dims, d);
  if (int r = check_gated(fn, d, false)) return r;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID, "%s: bytes is NULL", fn);
  *bytes = gated_ws_bytes(d);
  return ok();
}

int moe_gated_linear(const moe_gated_dims* dims, const void* x, const void* w_gate, const void* w_up, void* h,
                     void* gate, void* up, void* ws, size_t ws_bytes, moe_stream stream) {
  return run_gated("moe_gated_linear", dims, false, x, nullptr, w_gate, w_up, h, gate, up, ws, ws_bytes, stream);
}

int moe_grouped_gated(const moe_gated_dims* dims, const void* x, const int32_t* expert_offsets, const void* w_gate,
                      const void* w_up, void* h, void* gate, void* up, moe_stream stream) {
  return run_gated("moe_grouped_gated", dims, true, x, expert_offsets, w_gate, w_up, h, gate, up, nullptr, 0, stream);
}

int moe_gated_linear_backward_workspace_bytes(const moe_gated_dims* dims, size_t* bytes) {
  return gated_backward_ws("moe_gated_linear_backward_workspace_bytes", dims, false, bytes);
}

int moe_gated_linear_backward(const moe_gated_dims* dims, const void* dh, const void* x, const void* w_gate,
                              const void* w_up, const void* gate, const void* up, void* dx, void* dw_gate, void* dw_up,
                              void* ws, size_t ws_bytes, moe_stream stream) {
  return run_gated_backward("moe_gated_linear_backward", dims, false, dh, x, nullptr, w_gate, w_up, gate, up, dx,
                            dw_gate, dw_up, ws, ws_bytes, stream);
}

int moe_grouped_gated_backward_workspace_bytes(const moe_gated_dims* dims, size_t* bytes) {
  return gated_backward_ws("moe_grouped_gated_backward_workspace_bytes", dims, true, bytes);
}

int moe_grouped_gated_backward(const moe_gated_dims* dims, const void* dh, const void* x,
                               const int32_t* expert_offsets, const void* w_gate, const void* w_up, const void* gate,
                               const void* up, void* dx, void* dw_gate, void* dw_up, void* ws, size_t ws_bytes,
                               moe_stream stream) {
  return run_gated_backward("moe_grouped_gated_backward", dims, true, dh, x, expert_offsets, w_gate, w_up, gate, up, dx,
                            dw_gate, dw_up, ws, ws_bytes, stream);
}

int moe_adamw(const moe_adamw_args* args, const moe_adamw_tensor* tensors, int32_t count, moe_stream stream) {
  const char* fn = "moe_adamw";
  if (int r = check_adamw(fn, args, tensors, count)) return r;
  moe::AdamWArgs a{};
  a.fp8 = (args->flags & MOE_ADAMW_FP8) != 0;
  a.step = args->step;
  a.b1 = (float)args->beta1;
  a.a1 = (float)(1.0 - args->beta1);
  a.b2 = (float)args->beta2;
  a.a2 = (float)(1.0 - args->beta2);
  a.eps = (float)args->eps;
  a.lr = args->lr;
  a.decay = args->weight_decay;
  a.beta1 = args->beta1;
  a.beta2 = args->beta2;
  a.keep = (float)(1.0 - args->lr * args->weight_decay);
  a.size = (float)(args->lr / (1.0 - pow(args->beta1, args->step)));
  a.root = (float)(1.0 / sqrt(1.0 - pow(args->beta2, args->step)));
  a.lr_dev = args->lr_device;
  a.step_dev = args->step_device;
  a.grad_scale = args->grad_scale;
  int64_t total = 0;
  auto flush = [&]() {
    const hipError_t e = a.count > 0 ? moe::launch_adamw(a, static_cast<hipStream_t>(stream)) : hipSuccess;
    a.count = 0;
    total = 0;
    return e;
  };
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (t.numel == 0 || t.grad == nullptr) continue;
    if (a.count == moe::kAdamWTensors || total + t.numel > kMaxNumel)
      if (hipError_t e = flush()) return device_error(fn, e);
    a.tensor[a.count++] = moe::AdamWTensor{t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_exp, t.exp_avg_sq_exp, t.copy,
                                           t.numel, 0, (uint8_t)t.param_dtype, (uint8_t)t.grad_dtype, (uint8_t)t.copy_dtype};
    total += t.numel;
  }
  if (hipError_t e = flush()) return device_error(fn, e);
  return ok();
}

int moe_quantize_fp4(const void* w, int32_t dtype, int64_t rows, int32_t cols, uint8_t* codes, uint8_t* exps,
                     moe_stream stream) {
  const char* fn = "moe_quantize_fp4";
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
    return fail(MOE_ERR_INVALID, "%s: dtype=%d must be bf16 or fp16", fn, dtype);
  if (rows < 1 || rows > (1LL << 26)) return fail(MOE_ERR_INVALID, "%s: rows=%lld outside [1, 2^26]", fn, (long long)rows);
  if (cols < 32 || cols > kMaxWidth || cols % 32 != 0)
    return fail(MOE_ERR_INVALID, "%s: cols=%d must be a multiple of 32 in [32, %d]", fn, cols, kMaxWidth);
  REQ_PTR(w);
  REQ_PTR(codes);
  if (exps == nullptr) return fail(MOE_ERR_INVALID, "%s: exps is NULL", fn);
  if (hipError_t e = moe::launch_quantize_fp4(static_cast<const uint16_t*>(w), rows, cols, dtype == MOE_DTYPE_F16, codes, exps,
                                              static_cast<hipStream_t>(stream)))
    return device_error(fn, e);
  return ok();
}

int moe_linear_fp4_workspace_bytes(const moe_linear_dims* dims, size_t* bytes) {
  const char* fn = "moe_linear_fp4_workspace_bytes";
  COPY_DIMS(moe_linear_dims, d);
  if (int r = check_linear(fn, d)) return r;
  if (int r = check_fp4_width(fn, d.in_features, d.ld_w)) return r;
  return fp4_bytes(fn, linear_args(d, nullptr, nullptr, nullptr), bytes);
}

int moe_linear_fp4(const moe_linear_dims* dims, const void* x, const moe_fp4_matrix* w, const void* bias,
                   const void* residual, void* y, void* ws, size_t ws_bytes, moe_stream stream) {
  const char* fn = "moe_linear_fp4";
  COPY_DIMS(moe_linear_dims, d);
  if (int r = check_linear(fn, d)) return r;
  if (int r = check_fp4_width(fn, d.in_features, d.ld_w)) return r;
  if (d.rows == 0) return ok();
  REQ_ELEM(x, d.dtype);
  if (int r = check_fp4_matrix(fn, "w", w)) return r;
  OPT_ELEM(bias, d.bias_dtype);
  OPT_ELEM(residual, d.dtype);
  REQ_ELEM(y, d.dtype);
  if (y == x) return fail(MOE_ERR_INVALID, "%s: y is x", fn);
  if (residual == y && d.ld_residual != d.ld_y)
    return fail(MOE_ERR_INVALID, "%s: residual is y with another row stride", fn);
  moe::MatmulArgs a = linear_args(d, x, nullptr, y);
  a.bias = bias;
  a.bias_f32 = d.bias_dtype == MOE_DTYPE_F32;
  a.act = d.act;
  a.residual = static_cast<const uint16_t*>(residual);
  a.ldr = d.ld_residual;
  return run_fp4(fn, a, w, nullptr, ws, ws_bytes, stream);
}

int moe_grouped_matmul_fp4_workspace_bytes(const moe_grouped_dims* dims, size_t* bytes) {
  const char* fn = "moe_grouped_matmul_fp4_workspace_bytes";
  COPY_DIMS(moe_grouped_dims, d);
  if (int r = check_grouped(fn, d)) return r;
  if (int r = check_fp4_width(fn, d.in_features, d.in_features)) return r;
  return fp4_bytes(fn, grouped_args(d, nullptr, &kSomeOffsets, nullptr, nullptr), bytes);
}

int moe_grouped_matmul_fp4(const moe_grouped_dims* dims, const void* x, const int32_t* expert_offsets,
                           const moe_fp4_matrix* w, void* y, void* ws, size_t ws_bytes, moe_stream stream) {
  const char* fn = "moe_grouped_matmul_fp4";
  COPY_DIMS(moe_grouped_dims, d);
  if (int r = check_grouped(fn, d)) return r;
  if (int r = check_fp4_width(fn, d.in_features, d.in_features)) return r;
  if (d.rows == 0) return ok();
  REQ_ELEM(x, d.dtype);
  REQ_ELEM(expert_offsets, MOE_DTYPE_F32);
  if (int r = check_fp4_matrix(fn, "w", w)) return r;
  REQ_ELEM(y, d.dtype);
  if (y == x) return fail(MOE_ERR_INVALID, "%s: y is x", fn);
  return run_fp4(fn, grouped_args(d, x, expert_offsets, nullptr, y), w, nullptr, ws, ws_bytes, stream);
}

int moe_gated_linear_fp4_workspace_bytes(const moe_gated_dims* dims, size_t* bytes) {
  return gated_fp4_bytes("moe_gated_linear_fp4_workspace_bytes", dims, false, bytes);
}

int moe_gated_linear_fp4(const moe_gated_dims* dims, const void* x, const moe_fp4_matrix* w_gate,
                         const moe_fp4_matrix* w_up, void* h, void* ws, size_t ws_bytes, moe_stream stream) {
  return run_gated_fp4("moe_gated_linear_fp4", dims, false, x, nullptr, w_gate, w_up, h, ws, ws_bytes, stream);
}

int moe_grouped_gated_fp4_workspace_bytes(const moe_gated_dims* dims, size_t* bytes) {
  return gated_fp4_bytes("moe_grouped_gated_fp4_workspace_bytes", dims, true, bytes);
}

int moe_grouped_gated_fp4(const moe_gated_dims* dims, const void* x, const int32_t* expert_offsets,
                          const moe_fp4_matrix* w_gate, const moe_fp4_matrix* w_up, void* h, void* ws, size_t ws_bytes,
                          moe_stream stream) {
  return run_gated_fp4("moe_grouped_gated_fp4", dims, true, x, expert_offsets, w_gate, w_up, h, ws, ws_bytes, stream);
}

}  // extern "C"
