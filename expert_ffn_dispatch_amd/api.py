"""Python binding of the MoE FFN layer's C ABI (include/moe_ffn.h).

Argument marshalling only: every function passes device pointers of torch
tensors and the current HIP stream to the library; all computation happens in
the HIP kernels.  bf16 tensors may be torch.bfloat16 or torch.int16/uint16
views of the same bits.  Output tensors are allocated with torch (device
memory is torch's; the library never allocates).
"""
import array
import ctypes
from typing import NamedTuple, Optional

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


def _gated(x, w_gate, w_up, offsets, act, want_pre, h, gate, up, stream):
    _is_matrix(x, "x")
    dev, dt = x.device, x.dtype
    rows, n_in = x.shape
    px, ldx = _mat(x, "x", dev, _HALVES)
    code = _act(act)
    if offsets is None:
        E, po = 1, None
        pg, ldw = _mat(w_gate, "w_gate", dev, (dt,), None, n_in)
        width = w_gate.shape[0]
        pu, ldu = _mat(w_up, "w_up", dev, (dt,), width, n_in)
        if ldu != ldw:
            raise ValueError(f"w_gate and w_up: row strides {ldw} and {ldu} differ")
    else:
        pg, ldw = _experts(w_gate, "w_gate", dev, (dt,), None), 0
        E, width = w_gate.shape[0], w_gate.shape[1]
        if w_gate.shape[2] != n_in:
            raise ValueError(f"w_gate: shape {tuple(w_gate.shape)} beside rows of {n_in}")
        pu = _experts(w_up, "w_up", dev, (dt,), (E, width, n_in))
        po = _vec(offsets, "expert_offsets", dev, (torch.int32,), E + 1)
    if (gate is None) != (up is None):
        raise ValueError("gate and up: both or neither")
    lib = _lib.load()
    with _On(dev, stream) as st:
        if h is None:
            h = torch.empty((rows, width), dtype=dt, device=dev)
        ph, ldh = _mat(h, "h", dev, (dt,), rows, width)
        if gate is None and want_pre:
            gate, up = (torch.empty((rows, width), dtype=dt, device=dev) for _ in range(2))
        pa, pb, ldp = _pair(gate, up, dev, dt, rows, width)
        d = _lib.MoeGatedDims(rows, E, n_in, width, _DTYPES[dt], code, _DTYPES[dt], ldx, 0, ldw, ldh, ldp)
        if offsets is None:
            ws, pws, nws = _ws_for(lib.moe_gated_linear_workspace_bytes, d, dev)
            _lib.check(lib.moe_gated_linear(ctypes.byref(d), px, pg, pu, ph, pa, pb, pws, nws, st))
        else:
            _lib.check(lib.moe_grouped_gated(ctypes.byref(d), px, po, pg, pu, ph, pa, pb, st))
    return (h, gate, up) if gate is not None else h


def _pair(gate, up, dev, dt, rows, width):
    """Addresses and the one row stride of the saved products (None: absent)."""
    if gate is None:
        return None, None, 0
    pa, lda = _mat(gate, "gate", dev, (dt,), rows, width)
    pb, ldb = _mat(up, "up", dev, (dt,), rows, width)
    if lda != ldb:
        raise ValueError(f"gate and up: row strides {lda} and {ldb} differ")
    return pa, pb, lda


def moe_gated_linear(x, w_gate, w_up, act: str = "silu", want_pre: bool = False, h=None, gate=None, up=None,
                     stream=None):
    """act(x w_gate^T) * (x w_up^T) for x [rows][in] and w_gate, w_up
    [width][in].  Returns h, or (h, gate, up) with want_pre (or given gate and
    up): both products, for moe_gated_linear_backward."""
    return _gated(x, w_gate, w_up, None, act, want_pre, h, gate, up, stream)


def moe_grouped_gated(x, expert_offsets, w_gate, w_up, act: str = "silu", want_pre: bool = False, h=None, gate=None,
                      up=None, stream=None):
    """moe_gated_linear by expert (moe_permute's offsets): w_gate, w_up
    [E][width][in].  Rows outside every group are left as they are."""
    if expert_offsets is None:
        raise ValueError("expert_offsets: expected [E+1]")
    return _gated(x, w_gate, w_up, expert_offsets, act, want_pre, h, gate, up, stream)


def _gated_backward(dh, x, w_gate, w_up, gate, up, offsets, act, want_dx, want_dw, dw_dtype, dx, stream):
    _is_matrix(dh, "dh")
    dev, dt = dh.device, dh.dtype
    rows, width = dh.shape
    pd, ldh = _mat(dh, "dh", dev, _HALVES)
    px, ldx = _mat(x, "x", dev, (dt,), rows, None)
    n_in = x.shape[1]
    code = _act(act)
    if gate is None or up is None:
        raise ValueError("gate and up: required")
    pa, pb, ldp = _pair(gate, up, dev, dt, rows, width)
    if offsets is None:
        E, po, lead = 1, None, ()
        pg, ldw = _mat(w_gate, "w_gate", dev, (dt,), width, n_in)
        pu, ldu = _mat(w_up, "w_up", dev, (dt,), width, n_in)
        if ldu != ldw:
            raise ValueError(f"w_gate and w_up: row strides {ldw} and {ldu} differ")
    else:
        pg, ldw = _experts(w_gate, "w_gate", dev, (dt,), None), 0
        E = w_gate.shape[0]
        if tuple(w_gate.shape[1:]) != (width, n_in):
            raise ValueError(f"w_gate: shape {tuple(w_gate.shape)} beside gradients of {width} and rows of {n_in}")
        pu = _experts(w_up, "w_up", dev, (dt,), (E, width, n_in))
        po, lead = _vec(offsets, "expert_offsets", dev, (torch.int32,), E + 1), (E,)
    wt = dw_dtype or dt
    if wt not in (dt, torch.float32):
        raise TypeError(f"gradients of {wt} beside {dt} data")
    lib = _lib.load()
    with _On(dev, stream) as st:
        if dx is None and want_dx:
            dx = torch.empty((rows, n_in), dtype=dt, device=dev)
        pdx, lddx = _mat(dx, "dx", dev, (dt,), rows, n_in) if dx is not None else (None, 0)
        dwg, dwu = ((torch.empty((*lead, width, n_in), dtype=wt, device=dev) for _ in range(2)) if want_dw
                    else (None, None))
        pwg, pwu = (dwg.data_ptr(), dwu.data_ptr()) if want_dw else (None, None)
        d = _lib.MoeGatedDims(rows, E, n_in, width, _DTYPES[dt], code, _DTYPES[wt], ldx, lddx, ldw, ldh, ldp)
        if offsets is None:
            ws, pws, nws = _ws_for(lib.moe_gated_linear_backward_workspace_bytes, d, dev)
            _lib.check(lib.moe_gated_linear_backward(ctypes.byref(d), pd, px, pg, pu, pa, pb, pdx, pwg, pwu, pws, nws, st))
        else:
            ws, pws, nws = _ws_for(lib.moe_grouped_gated_backward_workspace_bytes, d, dev)
            _lib.check(lib.moe_grouped_gated_backward(ctypes.byref(d), pd, px, po, pg, pu, pa, pb, pdx, pwg, pwu, pws,
                                                      nws, st))
    return dx, dwg, dwu


def moe_gated_linear_backward(dh, x, w_gate, w_up, gate, up, act: str = "silu", want_dx: bool = True,
                              want_dw: bool = True, dw_dtype=None, dx=None, stream=None):
    """Gradients of moe_gated_linear: (dx, dw_gate, dw_up), None where not
    wanted.  gate and up are what the forward pass returned.  The weights'
    gradients have dh's type unless dw_dtype is torch.float32."""
    return _gated_backward(dh, x, w_gate, w_up, gate, up, None, act, want_dx, want_dw, dw_dtype, dx, stream)


def moe_grouped_gated_backward(dh, x, expert_offsets, w_gate, w_up, gate, up, act: str = "silu",
                               want_dx: bool = True, want_dw: bool = True, dw_dtype=None, dx=None, stream=None):
    """Gradients of moe_grouped_gated: (dx, dw_gate, dw_up), zero for the
    weights of an expert without rows."""
    if expert_offsets is None:
        raise ValueError("expert_offsets: expected [E+1]")
    return _gated_backward(dh, x, w_gate, w_up, gate, up, expert_offsets, act, want_dx, want_dw, dw_dtype, dx, stream)


class Fp8Moment(NamedTuple):
    """An 8-bit optimiser state: E4M3 codes [numel] (torch.float8_e4m3fn) and
    one exponent (torch.uint8) for every 128 of them; value = code *
    2^(exponent - 127).  All bytes zero is a state of zeros."""
    codes: torch.Tensor
    exps: torch.Tensor

    @classmethod
    def zeros(cls, param):
        n = param.numel()
        return cls(torch.zeros(n, dtype=torch.uint8, device=param.device).view(torch.float8_e4m3fn),
                   torch.zeros(-(-n // _lib.MOE_ADAMW_BLOCK), dtype=torch.uint8, device=param.device))

    def values(self):
        """The state in fp32 (for the second moment: its square root)."""
        n = self.codes.numel()
        scale = torch.where(self.exps == 255, float("nan"), torch.exp2(self.exps.double() - 127)).float()
        return self.codes.view(-1).float() * scale.repeat_interleave(_lib.MOE_ADAMW_BLOCK)[:n]


_TABLE_WORDS = ctypes.sizeof(_lib.MoeAdamWTensor) // 8
_data_ptr = torch.Tensor.data_ptr


def _same_order(a, b):
    """Whether contiguous values of the two shapes lie in the same order: one shape (but for ones), or one of them flat."""
    if a == b:
        return True
    p, q = ([n for n in s if n != 1] for s in (a, b))
    return a.numel() == b.numel() and (p == q or len(p) <= 1 or len(q) <= 1)


class AdamWTensors:
    """The tensors that moe_adamw updates, looked over once: params (bf16, fp16
    or fp32), their first and second moments (fp32 tensors, or Fp8Moment, all of
    one kind) and, where given, copies (bf16 or fp16, None for a parameter
    without one) that receive the new parameters.  All of the parameter's shape,
    or one of the two flat; contiguous, on one device, without overlaps.  The
    object keeps the memory of all, and is refused once any of them lies
    elsewhere.  One call at a time uses it."""

    def __init__(self, params, exp_avg, exp_avg_sq, copies=None):
        params, exp_avg, exp_avg_sq = list(params), list(exp_avg), list(exp_avg_sq)
        copies = [None] * len(params) if copies is None else list(copies)
        if not len(params) == len(exp_avg) == len(exp_avg_sq) == len(copies):
            raise ValueError("params, exp_avg, exp_avg_sq and copies: different lengths")
        self.fp8 = bool(params) and isinstance(exp_avg[0], Fp8Moment)
        self.device = params[0].device if params else None
        self._shapes = [p.shape for p in params]
        self.count = len(params)
        self._table = (_lib.MoeAdamWTensor * max(1, self.count))()
        self._words = memoryview(self._table).cast("B").cast("Q")
        self._kept = []                         # every tensor's memory, whatever becomes of the caller's object
        self._tensors, self._at = [], []        # every tensor, and where it was
        device, spans = self.device, []

        def place(i, entry, field, t, n, dtypes):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device:
                raise ValueError(f"{field} {i}: expected a tensor on {device}")
            if t.dtype not in dtypes:
                raise TypeError(f"{field} {i}: dtype {t.dtype} not in {tuple(dtypes)}")
            if t.numel() != n or not t.is_contiguous():
                raise ValueError(f"{field} {i}: expected {n} contiguous values, got shape {tuple(t.shape)}")
            if not field.endswith("_exp") and not _same_order(t.shape, self._shapes[i]):
                raise ValueError(f"{field} {i}: shape {tuple(t.shape)} beside a parameter of {tuple(self._shapes[i])}")
            at = t.data_ptr()
            setattr(entry, field, at)
            self._kept.append(t.untyped_storage())
            self._tensors.append(t)
            self._at.append(at)
            if n:
                spans.append((at, at + n * t.element_size(), field, i))

        fp8, codes = self.fp8, (torch.float8_e4m3fn,)
        for i, (p, m, v, c) in enumerate(zip(params, exp_avg, exp_avg_sq, copies)):
            n, e = p.numel(), self._table[i]
            place(i, e, "param", p, n, _DTYPES)
            for t, field in ((m, "exp_avg"), (v, "exp_avg_sq")):
                if isinstance(t, Fp8Moment) != fp8:
                    raise TypeError(f"{field} {i}: 8-bit and 32-bit states in one list")
                if fp8:
                    place(i, e, field, t.codes, n, codes)
                    place(i, e, field + "_exp", t.exps, -(-n // _lib.MOE_ADAMW_BLOCK), (torch.uint8,))
                else:
                    place(i, e, field, t, n, (torch.float32,))
            if c is not None:
                place(i, e, "copy", c, n, _HALVES)
                e.copy_dtype = _DTYPES[c.dtype]
            e.numel = n
            e.param_dtype = _DTYPES[p.dtype]
        spans.sort()
        for a, b in zip(spans, spans[1:]):
            if b[0] < a[1]:
                raise ValueError(f"{a[2]} {a[3]} and {b[2]} {b[3]} overlap")
        self._devices = [p.get_device() for p in params]
        self._grad_types = self._grad_shapes = None

    def _entries(self, grads):
        """The table with this step's gradients.  (List by list: 37 tensors one by
        one took 22 us, of a step of 9.)"""
        if list(map(_data_ptr, self._tensors)) != self._at:       # t.data = ..., or a storage of another size
            raise ValueError("the memory of a parameter, state or copy has moved since the list was made")
        if len(grads) != self.count:
            raise ValueError(f"grads: {len(grads)} for {self.count} parameters")
        if any(g is None for g in grads):
            return self._some(grads)
        shapes = [g.shape for g in grads]
        if (shapes != self._grad_shapes or [g.get_device() for g in grads] != self._devices
                or not all([g.is_contiguous() for g in grads])):
            self._refuse(grads)
            self._grad_shapes = shapes
        types = [g.dtype for g in grads]
        if types != self._grad_types:
            self._types(types)
        self._words[1::_TABLE_WORDS] = array.array("Q", [g.data_ptr() for g in grads])
        return self._table

    def _types(self, types):
        self._grad_types = None
        for i, t in enumerate(types):
            if t not in _DTYPES:
                raise TypeError(f"grad {i}: dtype {t} not in {tuple(_DTYPES)}")
            self._table[i].grad_dtype = _DTYPES[t]
        self._grad_types = types

    def _refuse(self, grads):
        for i, (g, s, d) in enumerate(zip(grads, self._shapes, self._devices)):
            if g is not None and (not _same_order(g.shape, s) or g.get_device() != d or not g.is_contiguous()):
                raise ValueError(f"grad {i}: expected contiguous values of shape {tuple(s)} on {self.device}, got shape "
                                 f"{tuple(g.shape)} on {g.device}")

    def _some(self, grads):
        """With parameters that have no gradient."""
        there = [(i, g) for i, g in enumerate(grads) if g is not None]
        self._refuse(grads)
        for i, g in there:
            if g.dtype not in _DTYPES:
                raise TypeError(f"grad {i}: dtype {g.dtype} not in {tuple(_DTYPES)}")
        self._grad_types = None
        for i, g in enumerate(grads):
            self._table[i].grad = None if g is None else g.data_ptr()
            if g is not None:
                self._table[i].grad_dtype = _DTYPES[g.dtype]
        return self._table


def _scalar(t, name, dtype, device):
    """(value, None) of a number, (0, address) of a one-element device tensor."""
    if not isinstance(t, torch.Tensor):
        return t, None
    if t.device != device or t.dtype != dtype or t.numel() != 1:
        raise ValueError(f"{name}: expected a number or one {dtype} on {device}")
    return 0, t.data_ptr()


def moe_adamw(tensors: AdamWTensors, grads, step, lr, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
              weight_decay: float = 0.01, grad_scale=None, stream=None):
    """One AdamW step in place over all tensors; grads: one for each (bf16, fp16
    or fp32, of its shape or flat; None leaves its parameter as it is).  step
    (from 1) and lr: numbers, or one-element device tensors (int32, fp32), which
    a captured call reads at every replay.  grad_scale: a one-element fp32 device tensor that the
    gradients are multiplied by, or None."""
    dev = tensors.device
    if dev is None:
        return
    step, p_step = _scalar(step, "step", torch.int32, dev)
    lr, p_lr = _scalar(lr, "lr", torch.float32, dev)
    p_scale = None
    if grad_scale is not None:
        if not isinstance(grad_scale, torch.Tensor):
            raise TypeError("grad_scale: expected a one-element fp32 device tensor")
        p_scale = _scalar(grad_scale, "grad_scale", torch.float32, dev)[1]
    table = tensors._entries(grads)
    a = _lib.MoeAdamWArgs(lr, beta1, beta2, eps, weight_decay, step, _lib.MOE_ADAMW_FP8 if tensors.fp8 else 0, p_lr,
                          p_step, p_scale)
    with _On(dev, stream) as st:
        _lib.check(_lib.load().moe_adamw(ctypes.byref(a), table, tensors.count, st))


class Fp4Weights(NamedTuple):
    """4-bit weights [..][out][in]: E2M1 codes [..][out][in / 2], two to a byte
    (the first in the low half), and one exponent [..][out][in / 32] for every
    32 of a row, both torch.uint8; weight = code * 2^(exponent - 127)."""
    codes: torch.Tensor
    exps: torch.Tensor

    def values(self):
        """The weights in fp32."""
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=self.codes.device)
        w = table[torch.stack([self.codes & 15, self.codes >> 4], -1).int()]
        scale = (self.exps.int() << 23).view(torch.float32)
        return (w.view(*self.exps.shape, 32) * scale[..., None]).view(*self.exps.shape[:-1], -1)


def moe_quantize_fp4(w, stream=None) -> Fp4Weights:
    """4-bit codes and exponents of contiguous bf16 or fp16 weights
    [..][out][in], in % 32 == 0."""
    if not isinstance(w, torch.Tensor) or not w.is_cuda or w.dim() < 2 or not w.is_contiguous():
        raise ValueError("w: expected a contiguous device tensor [..][out][in]")
    if w.dtype not in _HALVES:
        raise TypeError(f"w: dtype {w.dtype} not in {tuple(_HALVES)}")
    cols = w.shape[-1]
    rows = w.numel() // cols if cols else 0
    with _On(w.device, stream) as st:
        codes = torch.empty((*w.shape[:-1], cols // 2), dtype=torch.uint8, device=w.device)
        exps = torch.empty((*w.shape[:-1], cols // 32), dtype=torch.uint8, device=w.device)
        _lib.check(_lib.load().moe_quantize_fp4(w.data_ptr(), _DTYPES[w.dtype], rows, cols, codes.data_ptr(),
                                                exps.data_ptr(), st))
    return Fp4Weights(codes, exps)


def _fp4(w, name, device, n_in, lead=None):
    """The C descriptor of 4-bit weights with `lead` dimensions in front of the
    contraction's n_in (None: any two or three)."""
    if not isinstance(w, Fp4Weights):
        raise TypeError(f"{name}: expected Fp4Weights, got {type(w).__name__}")
    codes, exps = w
    lead = codes.shape[:-1] if lead is None else lead
    for t, what, per in ((codes, "codes", 2), (exps, "exponents", 32)):
        if t.device != device or t.dtype != torch.uint8:
            raise ValueError(f"{name}: {what} must be torch.uint8 on {device}, got {t.dtype} on {t.device}")
        s = t.shape
        if n_in % 32 or len(s) < 2 or s[:-1] != lead or s[-1] != n_in // per or not t.is_contiguous():
            raise ValueError(f"{name}: {what} of shape {tuple(s)}, expected a contiguous "
                             f"{(*lead, f'{n_in} / {per}')} with a multiple of 32 inputs")
    return _lib.MoeFp4Matrix(codes.data_ptr(), exps.data_ptr())


def moe_linear_fp4(x, w: Fp4Weights, bias=None, residual=None, act: str = "none", y=None, stream=None):
    """moe_linear with 4-bit weights [out][in]."""
    _is_matrix(x, "x")
    dev, dt = x.device, x.dtype
    rows, n_in = x.shape
    px, ldx = _mat(x, "x", dev, _HALVES)
    m = _fp4(w, "w", dev, n_in)
    if w.codes.dim() != 2:
        raise ValueError(f"w: codes of shape {tuple(w.codes.shape)}, expected [out][in / 2]")
    n_out = w.codes.shape[0]
    bt = _param_type(dt, bias)
    pr, ldr = _mat(residual, "residual", dev, (dt,), rows, n_out) if residual is not None else (None, 0)
    code = _act(act)
    lib = _lib.load()
    with _On(dev, stream) as st:
        if y is None:
            y = torch.empty((rows, n_out), dtype=dt, device=dev)
        py, ldy = _mat(y, "y", dev, (dt,), rows, n_out)
        d = _lib.MoeLinearDims(rows, n_in, n_out, _DTYPES[dt], code, _DTYPES[bt], _DTYPES[dt], ldx, 0, ldr, ldy, 0, 0, 0)
        ws, pws, nws = _ws_for(lib.moe_linear_fp4_workspace_bytes, d, dev)
        _lib.check(lib.moe_linear_fp4(ctypes.byref(d), px, ctypes.byref(m), _vec(bias, "bias", dev, (bt,), n_out), pr, py,
                                      pws, nws, st))
    return y


def moe_grouped_matmul_fp4(x, expert_offsets, w: Fp4Weights, y=None, stream=None):
    """moe_grouped_matmul with 4-bit weights [E][out][in]."""
    _is_matrix(x, "x")
    dev, dt = x.device, x.dtype
    rows, n_in = x.shape
    px, ldx = _mat(x, "x", dev, _HALVES)
    m = _fp4(w, "w", dev, n_in)
    if w.codes.dim() != 3:
        raise ValueError(f"w: codes of shape {tuple(w.codes.shape)}, expected [E][out][in / 2]")
    E, n_out = w.codes.shape[:2]
    if expert_offsets is None:
        raise ValueError("expert_offsets: expected [E+1]")
    po = _vec(expert_offsets, "expert_offsets", dev, (torch.int32,), E + 1)
    lib = _lib.load()
    with _On(dev, stream) as st:
        if y is None:
            y = torch.empty((rows, n_out), dtype=dt, device=dev)
        py, ldy = _mat(y, "y", dev, (dt,), rows, n_out)
        d = _lib.MoeGroupedDims(rows, E, n_in, n_out, _DTYPES[dt], _DTYPES[dt], ldx, ldy)
        ws, pws, nws = _ws_for(lib.moe_grouped_matmul_fp4_workspace_bytes, d, dev)
        _lib.check(lib.moe_grouped_matmul_fp4(ctypes.byref(d), px, po, ctypes.byref(m), py, pws, nws, st))
    return y


def _gated_fp4(x, w_gate, w_up, offsets, act, h, stream):
    _is_matrix(x, "x")
    dev, dt = x.device, x.dtype
    rows, n_in = x.shape
    px, ldx = _mat(x, "x", dev, _HALVES)
    code = _act(act)
    g = _fp4(w_gate, "w_gate", dev, n_in)
    shape = w_gate.codes.shape[:-1]
    if len(shape) != (1 if offsets is None else 2):
        raise ValueError(f"w_gate: codes of shape {tuple(w_gate.codes.shape)}")
    u = _fp4(w_up, "w_up", dev, n_in, shape)
    E, width = shape if offsets is not None else (1, shape[0])
    po = _vec(offsets, "expert_offsets", dev, (torch.int32,), E + 1)
    lib = _lib.load()
    with _On(dev, stream) as st:
        if h is None:
            h = torch.empty((rows, width), dtype=dt, device=dev)
        ph, ldh = _mat(h, "h", dev, (dt,), rows, width)
        d = _lib.MoeGatedDims(rows, E, n_in, width, _DTYPES[dt], code, _DTYPES[dt], ldx, 0, 0, ldh, 0)
        if offsets is None:
            ws, pws, nws = _ws_for(lib.moe_gated_linear_fp4_workspace_bytes, d, dev)
            _lib.check(lib.moe_gated_linear_fp4(ctypes.byref(d), px, ctypes.byref(g), ctypes.byref(u), ph, pws, nws, st))
        else:
            ws, pws, nws = _ws_for(lib.moe_grouped_gated_fp4_workspace_bytes, d, dev)
            _lib.check(lib.moe_grouped_gated_fp4(ctypes.byref(d), px, po, ctypes.byref(g), ctypes.byref(u), ph, pws, nws, st))
    return h


def moe_gated_linear_fp4(x, w_gate: Fp4Weights, w_up: Fp4Weights, act: str = "silu", h=None, stream=None):
    """moe_gated_linear with 4-bit weights [width][in]."""
    return _gated_fp4(x, w_gate, w_up, None, act, h, stream)


def moe_grouped_gated_fp4(x, expert_offsets, w_gate: Fp4Weights, w_up: Fp4Weights, act: str = "silu", h=None,
                          stream=None):
    """moe_grouped_gated with 4-bit weights [E][width][in]."""
    if expert_offsets is None:
        raise ValueError("expert_offsets: expected [E+1]")
    return _gated_fp4(x, w_gate, w_up, expert_offsets, act, h, stream)
