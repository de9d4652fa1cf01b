"""Python binding of the MoE FFN layer's C ABI (include/moe_ffn.h).

Argument marshalling only: every function passes device pointers of torch
tensors and the current HIP stream to the library; all computation happens in
the HIP kernels.  bf16 tensors may be torch.bfloat16 or torch.int16/uint16
views of the same bits.  Output tensors are allocated with torch (device
memory is torch's; the library never allocates).
"""
import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import MoeDims, MOE_FLAG_IDS_IN

_BF16_LIKE = (torch.bfloat16, torch.int16, torch.uint16)


def dims(N: int, M: int, E: int, k: int, H: int = 64, S: int = 0, Hs: int = 0) -> MoeDims:
    return MoeDims(N, M, E, k, H, S, Hs)


def _ptr(t: Optional[torch.Tensor], dtypes=None) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"dtype {t.dtype} not in {dtypes}")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def moe_layer_workspace_bytes(d: MoeDims, flags: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().moe_layer_workspace_bytes(ctypes.byref(d), flags, ctypes.byref(n)))
    return n.value


def moe_layer_single_launch(d: MoeDims, flags: int = 0, fp8: bool = False) -> bool:
    """Whether moe_layer (or moe_layer_fp8) runs these dims as one launch."""
    v = ctypes.c_int(0)
    _lib.check(_lib.load().moe_layer_single_launch(ctypes.byref(d), flags, int(fp8), ctypes.byref(v)))
    return bool(v.value)


def moe_route_workspace_bytes(d: MoeDims) -> int:
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().moe_route_workspace_bytes(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def moe_permute_workspace_bytes(d: MoeDims) -> int:
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().moe_permute_workspace_bytes(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def moe_grouped_ffn_workspace_bytes(d: MoeDims) -> int:
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().moe_grouped_ffn_workspace_bytes(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def moe_route(d: MoeDims, x, w_router, router_bias=None, topk_ids=None, topk_weights=None, ws=None,
              stream=None):
    dev = x.device
    if topk_ids is None:
        topk_ids = torch.empty((d.n_tokens, d.top_k), dtype=torch.int32, device=dev)
    if topk_weights is None:
        topk_weights = torch.empty((d.n_tokens, d.top_k), dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(moe_route_workspace_bytes(d), dev)
    _lib.check(_lib.load().moe_route(ctypes.byref(d), _ptr(x, _BF16_LIKE), _ptr(w_router, _BF16_LIKE),
                                     _ptr(router_bias, (torch.float32,)), _ptr(topk_ids, (torch.int32,)),
                                     _ptr(topk_weights, (torch.float32,)), _ptr(ws), ws.numel(),
                                     _stream(stream)))
    return topk_ids, topk_weights


def moe_permute(d: MoeDims, topk_ids, x=None, want_x_sorted: bool = False, ws=None, stream=None):
    dev = topk_ids.device
    A = d.n_tokens * d.top_k
    counts = torch.empty(d.n_experts, dtype=torch.int32, device=dev)
    offsets = torch.empty(d.n_experts + 1, dtype=torch.int32, device=dev)
    s2a = torch.empty(max(A, 1), dtype=torch.int32, device=dev)[:A]
    a2s = torch.empty(max(A, 1), dtype=torch.int32, device=dev)[:A]
    xs = torch.empty((A, d.hidden), dtype=x.dtype, device=dev) if want_x_sorted else None
    if ws is None:
        ws = workspace(moe_permute_workspace_bytes(d), dev)
    _lib.check(_lib.load().moe_permute(ctypes.byref(d), _ptr(topk_ids, (torch.int32,)),
                                       _ptr(x, _BF16_LIKE) if want_x_sorted else None,
                                       _ptr(counts), _ptr(offsets), _ptr(s2a), _ptr(a2s),
                                       _ptr(xs), _ptr(ws), ws.numel(), _stream(stream)))
    return {"expert_counts": counts, "expert_offsets": offsets, "sorted_to_assign": s2a,
            "assign_to_sorted": a2s, "x_sorted": xs}


def moe_grouped_ffn(d: MoeDims, x_sorted, expert_offsets, w_gate, w_up, w_down, row_scale=None,
                    y_sorted=None, ws=None, stream=None):
    dev = x_sorted.device
    A = d.n_tokens * d.top_k
    if y_sorted is None:
        y_sorted = torch.empty((A, d.hidden), dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = workspace(moe_grouped_ffn_workspace_bytes(d), dev)
    _lib.check(_lib.load().moe_grouped_ffn(ctypes.byref(d), _ptr(x_sorted, _BF16_LIKE),
                                           _ptr(expert_offsets, (torch.int32,)), _ptr(w_gate, _BF16_LIKE),
                                           _ptr(w_up, _BF16_LIKE), _ptr(w_down, _BF16_LIKE),
                                           _ptr(row_scale, (torch.float32,)), _ptr(y_sorted, _BF16_LIKE),
                                           _ptr(ws), ws.numel(), _stream(stream)))
    return y_sorted


def moe_combine(d: MoeDims, y_sorted, assign_to_sorted, topk_weights=None, shared_out=None, out=None,
                stream=None):
    if out is None:
        out = torch.empty((d.n_tokens, d.hidden), dtype=torch.bfloat16, device=y_sorted.device)
    _lib.check(_lib.load().moe_combine(ctypes.byref(d), _ptr(y_sorted, _BF16_LIKE),
                                       _ptr(assign_to_sorted, (torch.int32,)),
                                       _ptr(topk_weights, (torch.float32,)), _ptr(shared_out, _BF16_LIKE),
                                       _ptr(out, _BF16_LIKE), _stream(stream)))
    return out


def moe_layer(d: MoeDims, x, w_gate, w_up, w_down, w_router=None, router_bias=None, ws_gate=None,
              ws_up=None, ws_down=None, topk_ids=None, topk_weights=None, ids_in: bool = False, out=None,
              ws=None, stream=None):
    dev = x.device
    flags = MOE_FLAG_IDS_IN if ids_in else 0
    if out is None:
        out = torch.empty((d.n_tokens, d.hidden), dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = workspace(moe_layer_workspace_bytes(d, flags), dev)
    _lib.check(_lib.load().moe_layer(
        ctypes.byref(d), flags, _ptr(x, _BF16_LIKE), _ptr(w_router, _BF16_LIKE),
        _ptr(router_bias, (torch.float32,)), _ptr(w_gate, _BF16_LIKE), _ptr(w_up, _BF16_LIKE),
        _ptr(w_down, _BF16_LIKE), _ptr(ws_gate, _BF16_LIKE), _ptr(ws_up, _BF16_LIKE),
        _ptr(ws_down, _BF16_LIKE), _ptr(topk_ids, (torch.int32,)), _ptr(topk_weights, (torch.float32,)),
        _ptr(out, _BF16_LIKE), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def moe_layer_noalloc(d: MoeDims, x, w_gate, w_up, w_down, w_router=None, router_bias=None, ws_gate=None,
                      ws_up=None, ws_down=None, topk_ids=None, topk_weights=None, ids_in: bool = False, out=None,
                      stream=None):
    """moe_layer with the library's own workspace array: nothing is
    allocated for the call except `out` when the caller passes none."""
    dev = x.device
    flags = MOE_FLAG_IDS_IN if ids_in else 0
    if out is None:
        out = torch.empty((d.n_tokens, d.hidden), dtype=torch.bfloat16, device=dev)
    _lib.check(_lib.load().moe_layer_noalloc(
        ctypes.byref(d), flags, _ptr(x, _BF16_LIKE), _ptr(w_router, _BF16_LIKE),
        _ptr(router_bias, (torch.float32,)), _ptr(w_gate, _BF16_LIKE), _ptr(w_up, _BF16_LIKE),
        _ptr(w_down, _BF16_LIKE), _ptr(ws_gate, _BF16_LIKE), _ptr(ws_up, _BF16_LIKE),
        _ptr(ws_down, _BF16_LIKE), _ptr(topk_ids, (torch.int32,)), _ptr(topk_weights, (torch.float32,)),
        _ptr(out, _BF16_LIKE), _stream(stream)))
    return out


class Fp8Weights:
    """FP8 (OCP E4M3) expert weights with one float32 scale per output channel:
    codes `gate`/`up` [E][H][M] and `down` [E][M][H] (torch.uint8), scales
    `gate_scale`/`up_scale` [E][H] and `down_scale` [E][M] (torch.float32)."""

    FIELDS = ("gate", "up", "down", "gate_scale", "up_scale", "down_scale")

    def __init__(self, gate, up, down, gate_scale, up_scale, down_scale):
        self.gate, self.up, self.down = gate, up, down
        self.gate_scale, self.up_scale, self.down_scale = gate_scale, up_scale, down_scale

    def c_struct(self) -> _lib.MoeFp8Ffn:
        codes = [_ptr(getattr(self, n), (torch.uint8,)) for n in self.FIELDS[:3]]
        scales = [_ptr(getattr(self, n), (torch.float32,)) for n in self.FIELDS[3:]]
        return _lib.MoeFp8Ffn(*codes, *scales)


def moe_quantize_fp8(w, q=None, scale=None, stream=None):
    """Per-output-channel E4M3 quantisation of a bf16 matrix [..., cols]
    (every leading index is one output channel).  Returns (codes, scales)."""
    rows = w.numel() // w.shape[-1]
    if q is None:
        q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    if scale is None:
        scale = torch.empty(w.shape[:-1], dtype=torch.float32, device=w.device)
    _lib.check(_lib.load().moe_quantize_fp8(_ptr(w, _BF16_LIKE), rows, w.shape[-1], _ptr(q, (torch.uint8,)),
                                            _ptr(scale, (torch.float32,)), _stream(stream)))
    return q, scale


def quantize_ffn_fp8(w_gate, w_up, w_down, stream=None) -> Fp8Weights:
    """FP8 copies of one set of expert weights (three moe_quantize_fp8 calls)."""
    g, sg = moe_quantize_fp8(w_gate, stream=stream)
    u, su = moe_quantize_fp8(w_up, stream=stream)
    d, sd = moe_quantize_fp8(w_down, stream=stream)
    return Fp8Weights(g, u, d, sg, su, sd)


def moe_grouped_ffn_fp8(d: MoeDims, x_sorted, expert_offsets, experts: Fp8Weights, row_scale=None,
                        y_sorted=None, ws=None, stream=None):
    dev = x_sorted.device
    A = d.n_tokens * d.top_k
    if y_sorted is None:
        y_sorted = torch.empty((A, d.hidden), dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = workspace(moe_grouped_ffn_workspace_bytes(d), dev)
    st = experts.c_struct()
    _lib.check(_lib.load().moe_grouped_ffn_fp8(ctypes.byref(d), _ptr(x_sorted, _BF16_LIKE),
                                               _ptr(expert_offsets, (torch.int32,)), ctypes.byref(st),
                                               _ptr(row_scale, (torch.float32,)), _ptr(y_sorted, _BF16_LIKE),
                                               _ptr(ws), ws.numel(), _stream(stream)))
    return y_sorted


def moe_layer_fp8(d: MoeDims, x, experts: Fp8Weights, shared: Optional[Fp8Weights] = None, w_router=None,
                  router_bias=None, topk_ids=None, topk_weights=None, ids_in: bool = False, out=None, ws=None,
                  stream=None):
    dev = x.device
    flags = MOE_FLAG_IDS_IN if ids_in else 0
    if out is None:
        out = torch.empty((d.n_tokens, d.hidden), dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = workspace(moe_layer_workspace_bytes(d, flags), dev)
    ex = experts.c_struct()
    sh = shared.c_struct() if shared is not None else None
    _lib.check(_lib.load().moe_layer_fp8(
        ctypes.byref(d), flags, _ptr(x, _BF16_LIKE), _ptr(w_router, _BF16_LIKE),
        _ptr(router_bias, (torch.float32,)), ctypes.byref(ex), ctypes.byref(sh) if sh is not None else None,
        _ptr(topk_ids, (torch.int32,)), _ptr(topk_weights, (torch.float32,)), _ptr(out, _BF16_LIKE),
        _ptr(ws), ws.numel(), _stream(stream)))
    return out


def moe_layer_pipelined_workspace_bytes(d: MoeDims, n_micro: int, flags: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().moe_layer_pipelined_workspace_bytes(ctypes.byref(d), flags, n_micro, ctypes.byref(n)))
    return n.value


def moe_layer_pipelined(d: MoeDims, n_micro: int, x, w_gate, w_up, w_down, w_router=None, router_bias=None,
                        ws_gate=None, ws_up=None, ws_down=None, topk_ids=None, topk_weights=None,
                        ids_in: bool = False, out=None, ws=None, stream=None):
    dev = x.device
    flags = MOE_FLAG_IDS_IN if ids_in else 0
    if out is None:
        out = torch.empty((d.n_tokens, d.hidden), dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = workspace(moe_layer_pipelined_workspace_bytes(d, n_micro, flags), dev)
    _lib.check(_lib.load().moe_layer_pipelined(
        ctypes.byref(d), flags, n_micro, _ptr(x, _BF16_LIKE), _ptr(w_router, _BF16_LIKE),
        _ptr(router_bias, (torch.float32,)), _ptr(w_gate, _BF16_LIKE), _ptr(w_up, _BF16_LIKE),
        _ptr(w_down, _BF16_LIKE), _ptr(ws_gate, _BF16_LIKE), _ptr(ws_up, _BF16_LIKE),
        _ptr(ws_down, _BF16_LIKE), _ptr(topk_ids, (torch.int32,)), _ptr(topk_weights, (torch.float32,)),
        _ptr(out, _BF16_LIKE), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def moe_set_stage_events(events) -> None:
    """Record the given MOE_STAGE_EVENTS torch.cuda.Event objects at the stage
    boundaries of the next moe_layer call on this thread (None clears).  The
    events must have been recorded once (torch creates them lazily)."""
    lib = _lib.load()
    if events is None:
        _lib.check(lib.moe_set_stage_events(None, 0))
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _lib.check(lib.moe_set_stage_events(arr, len(events)))


# ---------------------- around the expert layer ----------------------------
#
# Layer norm, linear layers and products grouped by expert, with their
# gradients.  Matrices are 2-D tensors whose rows may be strided (the last
# dimension is contiguous); bf16 or fp16, for the layer norm also fp32.
# Outputs and workspaces are allocated for the call's stream, so that the
# allocator reuses them in that stream's order; the call runs on the tensors'
# device, whichever is current.

_DTYPES = {torch.bfloat16: _lib.MOE_DTYPE_BF16, torch.float16: _lib.MOE_DTYPE_F16, torch.float32: _lib.MOE_DTYPE_F32}
_HALVES = (torch.bfloat16, torch.float16)
# the current stream's handle without building a Stream object (1.8 us a call)
_raw_stream = torch._C._cuda_getCurrentRawStream


class _On:
    """Makes the tensors' device and the call's stream current; yields the
    raw stream.  Nothing is switched where both are current already."""

    __slots__ = ("ctx", "raw")

    def __init__(self, device, stream):
        self.ctx = None
        if stream is None:
            index = device.index
            if index != torch.cuda.current_device():
                self.ctx = torch.cuda.device(device)
            self.raw = _raw_stream(index)
            return
        if not hasattr(stream, "cuda_stream"):
            # a raw hipStream_t; 0 is the null stream, torch's default
            stream = torch.cuda.ExternalStream(int(stream), device) if int(stream) else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"stream of {stream.device} for tensors on {device}")
        self.ctx = torch.cuda.stream(stream)
        self.raw = stream.cuda_stream

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.raw

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _mat(t, name, device, dtypes, rows=None, cols=None):
    """(address, row stride in elements) of a matrix, its shape and type checked."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(dtypes)}")
    s = t.shape
    if len(s) != 2 or (rows is not None and s[0] != rows) or (cols is not None and s[1] != cols):
        raise ValueError(f"{name}: shape {tuple(s)}, expected ({'rows' if rows is None else rows}, "
                         f"{'cols' if cols is None else cols})")
    r, c = s
    if r <= 1 and c <= 1 or t.is_contiguous():
        return t.data_ptr(), c
    if c > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: elements of a row must be contiguous (strides {t.stride()})")
    if r <= 1:
        return t.data_ptr(), c
    if t.stride(0) < c:
        raise ValueError(f"{name}: rows overlap (strides {t.stride()})")
    return t.data_ptr(), t.stride(0)


def _vec(t, name, device, dtypes, n):
    """Address of a contiguous vector of n values, or None."""
    if t is None:
        return None
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(dtypes)}")
    s = t.shape
    if len(s) != 1 or s[0] != n or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous vector of {n} values, got shape {tuple(s)}")
    return t.data_ptr()


def _experts(t, name, device, dtypes, shape):
    """Address of a contiguous [E][out][in] tensor."""
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(dtypes)}")
    if t.dim() != 3 or (shape is not None and tuple(t.shape) != shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {'[E][out][in]' if shape is None else shape} tensor, "
                         f"got shape {tuple(t.shape)}")
    return t.data_ptr()


def _is_matrix(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name}: expected a 2-D device tensor")


def _ws_for(query, d, device):
    n = ctypes.c_size_t(0)
    _lib.check(query(ctypes.byref(d), ctypes.byref(n)))
    if n.value == 0:
        return None, None, 0
    t = torch.empty(n.value, dtype=torch.uint8, device=device)
    return t, t.data_ptr(), n.value


def _param_type(dtype, *params):
    """The one type of the given parameters (None: absent)."""
    t = None
    for p in params:
        if p is not None:
            if t is not None and p.dtype != t:
                raise TypeError(f"parameters of different types {t} and {p.dtype}")
            t = p.dtype
    if t is None:
        return dtype
    if t != dtype and t != torch.float32:
        raise TypeError(f"parameters of {t} beside {dtype} data")
    return t


def moe_layer_norm(x, gamma=None, beta=None, eps: float = 1e-5, rms: bool = False, want_stats: bool = False, y=None,
                   stream=None):
    """Layer norm over the rows of x (rms: root-mean-square form).  Returns y,
    or (y, mean, rstd) with want_stats (for moe_layer_norm_backward; mean is
    zero with rms)."""
    _is_matrix(x, "x")
    dev, dt = x.device, x.dtype
    rows, cols = x.shape
    px, ldx = _mat(x, "x", dev, _DTYPES)
    pt = _param_type(dt, gamma, beta)
    with _On(dev, stream) as st:
        if y is None:
            y = torch.empty_like(x)
        py, ldy = _mat(y, "y", dev, (dt,), rows, cols)
        mean = torch.empty(rows, dtype=torch.float32, device=dev) if want_stats else None
        rstd = torch.empty(rows, dtype=torch.float32, device=dev) if want_stats else None
        d = _lib.MoeNormDims(rows, cols, _DTYPES[dt], _DTYPES[pt], _lib.MOE_NORM_RMS if rms else 0, eps, ldx, ldy, 0, 0)
        _lib.check(_lib.load().moe_layer_norm(
            ctypes.byref(d), px, _vec(gamma, "gamma", dev, (pt,), cols), _vec(beta, "beta", dev, (pt,), cols), py,
            mean.data_ptr() if want_stats else None, rstd.data_ptr() if want_stats else None, st))
    return (y, mean, rstd) if want_stats else y


def moe_layer_norm_backward(dy, x, gamma, mean, rstd, rms: bool = False, want_dx: bool = True,
                            want_params: bool = True, param_dtype=None, dx=None, stream=None):
    """Gradients of moe_layer_norm: (dx, dgamma, dbeta), None where not wanted.
    mean (may be None with rms) and rstd are the forward pass's.  dgamma and
    dbeta have gamma's type (param_dtype where gamma is None; x's by default)."""
    _is_matrix(x, "x")
    dev, dt = x.device, x.dtype
    rows, cols = x.shape
    px, ldx = _mat(x, "x", dev, _DTYPES)
    pd, ldd = _mat(dy, "dy", dev, (dt,), rows, cols)
    pt = _param_type(dt, gamma) if gamma is not None or param_dtype is None else param_dtype
    if pt not in (dt, torch.float32):
        raise TypeError(f"param_dtype {pt} beside {dt} data")
    f32 = (torch.float32,)
    if mean is None and not rms:
        raise ValueError("mean: required without rms")
    if rstd is None:
        raise ValueError("rstd: required")
    lib = _lib.load()
    with _On(dev, stream) as st:
        if dx is None and want_dx:
            dx = torch.empty_like(x)
        po, ldo = _mat(dx, "dx", dev, (dt,), rows, cols) if dx is not None else (None, 0)
        dgamma = torch.empty(cols, dtype=pt, device=dev) if want_params else None
        dbeta = torch.empty(cols, dtype=pt, device=dev) if want_params else None
        d = _lib.MoeNormDims(rows, cols, _DTYPES[dt], _DTYPES[pt], _lib.MOE_NORM_RMS if rms else 0, 0.0, ldx, 0, ldd, ldo)
        ws, pw, nw = _ws_for(lib.moe_layer_norm_backward_workspace_bytes, d, dev) if want_params else (None, None, 0)
        _lib.check(lib.moe_layer_norm_backward(
            ctypes.byref(d), pd, px, _vec(gamma, "gamma", dev, (pt,), cols),
            None if rms else _vec(mean, "mean", dev, f32, rows), _vec(rstd, "rstd", dev, f32, rows), po,
            dgamma.data_ptr() if want_params else None, dbeta.data_ptr() if want_params else None, pw, nw, st))
    return dx, dgamma, dbeta


def _act(act: str) -> int:
    if act not in _lib.MOE_ACTS:
        raise ValueError(f"act {act!r} not in {tuple(_lib.MOE_ACTS)}")
    return _lib.MOE_ACTS[act]


def moe_linear(x, w, bias=None, residual=None, act: str = "none", want_pre: bool = False, y=None, pre=None,
               stream=None):
    """act(x w^T + bias) + residual for x [rows][in] and w [out][in].  Returns
    y, or (y, pre) with want_pre (or a given pre): the sum before the
    activation, for moe_linear_backward."""
    _is_matrix(x, "x")
    dev, dt = x.device, x.dtype
    rows, n_in = x.shape
    px, ldx = _mat(x, "x", dev, _HALVES)
    pw, ldw = _mat(w, "w", dev, (dt,), None, n_in)
    n_out = w.shape[0]
    bt = _param_type(dt, bias)
    pr, ldr = _mat(residual, "residual", dev, (dt,), rows, n_out) if residual is not None else (None, 0)
    code = _act(act)
    lib = _lib.load()
    with _On(dev, stream) as st:
        if y is None:
            y = torch.empty((rows, n_out), dtype=dt, device=dev)
        py, ldy = _mat(y, "y", dev, (dt,), rows, n_out)
        if pre is None and want_pre:
            pre = torch.empty((rows, n_out), dtype=dt, device=dev)
        pp, ldp = _mat(pre, "pre", dev, (dt,), rows, n_out) if pre is not None else (None, 0)
        d = _lib.MoeLinearDims(rows, n_in, n_out, _DTYPES[dt], code, _DTYPES[bt], _DTYPES[dt], ldx, ldw, ldr, ldy, ldp, 0, 0)
        ws, pws, nws = _ws_for(lib.moe_linear_workspace_bytes, d, dev)
        _lib.check(lib.moe_linear(ctypes.byref(d), px, pw, _vec(bias, "bias", dev, (bt,), n_out), pr, py, pp, pws, nws, st))
    return (y, pre) if pre is not None else y


def moe_linear_backward(dy, x, w, pre=None, act: str = "none", want_dx: bool = True, want_dw: bool = True,
                        want_dbias: bool = False, bias_dtype=None, dw_dtype=None, dx=None, stream=None):
    """Gradients of moe_linear: (dx, dw, dbias), None where not wanted.  pre is
    what the forward pass returned (None with act "none"); the residual's
    gradient is dy itself.  dw has w's type unless dw_dtype is torch.float32."""
    _is_matrix(dy, "dy")
    dev, dt = dy.device, dy.dtype
    rows, n_out = dy.shape
    pd, ldd = _mat(dy, "dy", dev, _HALVES)
    px, ldx = _mat(x, "x", dev, (dt,), rows, None)
    n_in = x.shape[1]
    pw, ldw = _mat(w, "w", dev, (dt,), n_out, n_in)
    code = _act(act)
    if (pre is None) != (act == "none"):
        raise ValueError("pre: required with an activation, None without")
    pp, ldp = _mat(pre, "pre", dev, (dt,), rows, n_out) if pre is not None else (None, 0)
    bt, wt = bias_dtype or dt, dw_dtype or dt
    for t in (bt, wt):
        if t not in (dt, torch.float32):
            raise TypeError(f"gradients of {t} beside {dt} data")
    lib = _lib.load()
    with _On(dev, stream) as st:
        if dx is None and want_dx:
            dx = torch.empty((rows, n_in), dtype=dt, device=dev)
        po, ldo = _mat(dx, "dx", dev, (dt,), rows, n_in) if dx is not None else (None, 0)
        dw = torch.empty((n_out, n_in), dtype=wt, device=dev) if want_dw else None
        dbias = torch.empty(n_out, dtype=bt, device=dev) if want_dbias else None
        d = _lib.MoeLinearDims(rows, n_in, n_out, _DTYPES[dt], code, _DTYPES[bt], _DTYPES[wt], ldx, ldw, 0, 0, ldp, ldd, ldo)
        ws, pws, nws = _ws_for(lib.moe_linear_backward_workspace_bytes, d, dev)
        _lib.check(lib.moe_linear_backward(ctypes.byref(d), pd, px, pw, pp, po, dw.data_ptr() if want_dw else None,
                                           dbias.data_ptr() if want_dbias else None, pws, nws, st))
    return dx, dw, dbias


def moe_grouped_matmul(x, expert_offsets, w, y=None, stream=None):
    """x[r] w[e]^T for the rows r of every expert e (moe_permute's offsets);
    x [rows][in], w [E][out][in].  Rows outside every group are left as they are."""
    _is_matrix(x, "x")
    dev, dt = x.device, x.dtype
    rows, n_in = x.shape
    px, ldx = _mat(x, "x", dev, _HALVES)
    pw = _experts(w, "w", dev, (dt,), None)
    E, n_out = w.shape[0], w.shape[1]
    if w.shape[2] != n_in:
        raise ValueError(f"w: shape {tuple(w.shape)} beside rows of {n_in}")
    po = _vec(expert_offsets, "expert_offsets", dev, (torch.int32,), E + 1)
    with _On(dev, stream) as st:
        if y is None:
            y = torch.empty((rows, n_out), dtype=dt, device=dev)
        py, ldy = _mat(y, "y", dev, (dt,), rows, n_out)
        d = _lib.MoeGroupedDims(rows, E, n_in, n_out, _DTYPES[dt], _DTYPES[dt], ldx, ldy)
        _lib.check(_lib.load().moe_grouped_matmul(ctypes.byref(d), px, po, pw, py, st))
    return y


def moe_grouped_matmul_dgrad(dy, expert_offsets, w, dx=None, stream=None):
    """The rows' gradient of moe_grouped_matmul: dy[r] w[e]."""
    _is_matrix(dy, "dy")
    dev, dt = dy.device, dy.dtype
    rows, n_out = dy.shape
    pd, ldd = _mat(dy, "dy", dev, _HALVES)
    pw = _experts(w, "w", dev, (dt,), None)
    E, n_in = w.shape[0], w.shape[2]
    if w.shape[1] != n_out:
        raise ValueError(f"w: shape {tuple(w.shape)} beside gradients of {n_out}")
    po = _vec(expert_offsets, "expert_offsets", dev, (torch.int32,), E + 1)
    with _On(dev, stream) as st:
        if dx is None:
            dx = torch.empty((rows, n_in), dtype=dt, device=dev)
        px, ldx = _mat(dx, "dx", dev, (dt,), rows, n_in)
        d = _lib.MoeGroupedDims(rows, E, n_in, n_out, _DTYPES[dt], _DTYPES[dt], ldx, ldd)
        _lib.check(_lib.load().moe_grouped_matmul_dgrad(ctypes.byref(d), pd, po, pw, px, st))
    return dx


def moe_grouped_matmul_wgrad(dy, x, expert_offsets, dtype=None, dw=None, stream=None):
    """The weights' gradient of moe_grouped_matmul: dw[e] = sum of dy[r]^T x[r]
    over e's rows, [E][out][in] in x's type or torch.float32."""
    _is_matrix(x, "x")
    dev, dt = x.device, x.dtype
    rows, n_in = x.shape
    px, ldx = _mat(x, "x", dev, _HALVES)
    pd, ldd = _mat(dy, "dy", dev, (dt,), rows, None)
    n_out = dy.shape[1]
    if expert_offsets is None or expert_offsets.dim() != 1 or expert_offsets.numel() < 2:
        raise ValueError("expert_offsets: expected [E+1]")
    E = expert_offsets.numel() - 1
    po = _vec(expert_offsets, "expert_offsets", dev, (torch.int32,), E + 1)
    wt = dtype or (dw.dtype if dw is not None else dt)
    if wt not in (dt, torch.float32):
        raise TypeError(f"gradients of {wt} beside {dt} data")
    lib = _lib.load()
    with _On(dev, stream) as st:
        if dw is None:
            dw = torch.empty((E, n_out, n_in), dtype=wt, device=dev)
        pw = _experts(dw, "dw", dev, (wt,), (E, n_out, n_in))
        d = _lib.MoeGroupedDims(rows, E, n_in, n_out, _DTYPES[dt], _DTYPES[wt], ldx, ldd)
        ws, pws, nws = _ws_for(lib.moe_grouped_matmul_wgrad_workspace_bytes, d, dev)
        _lib.check(lib.moe_grouped_matmul_wgrad(ctypes.byref(d), pd, px, po, pw, pws, nws, st))
    return dw
