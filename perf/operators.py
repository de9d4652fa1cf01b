"""Cases, plain forms and calls of the operators around the expert layer: layer norm, linear layers with a
fused epilogue, and matrix products grouped by expert, each with its gradients.

Sizes are those of the workloads in datagen/configs.py (hidden sizes 2048, 4096, 5120 and 6144, expert widths
768, 1536 and 16384, 8 to 160 experts, 1 to 65536 rows) and numbers between them.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-5


# ------------------------------------------------------------------ cases

def norm_case(name, op, rows, cols, dtype="bf16", params="same", rms=False):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "params": params, "rms": rms}


def linear_case(name, op, rows, n_in, n_out, act, bias, residual, dtype="bf16", params="same", save=False):
    return {"name": name, "op": op, "rows": rows, "n_in": n_in, "n_out": n_out, "act": act, "bias": bias,
            "residual": residual, "dtype": dtype, "params": params, "save": save}


def grouped_case(name, op, rows, experts, n_in, n_out, dtype="bf16", grad="same", skew=1.2):
    return {"name": name, "op": op, "rows": rows, "experts": experts, "n_in": n_in, "n_out": n_out, "dtype": dtype,
            "grad": grad, "skew": skew}


def listed():
    return [
        # one token before the router of a 2048-wide layer: a decode step, all latency
        norm_case("norm_token", "norm_forward", 1, 2048),
        # a prompt of 8192 tokens before the 4096-wide layer
        norm_case("norm_prompt", "norm_forward", 8192, 4096),
        # the training step's gradient for 4096 tokens of the 5120-wide layer, weights kept in 32 bits
        norm_case("norm_grad", "norm_backward", 4096, 5120, params="f32"),
        # a ragged micro-batch of odd width in fp16, root-mean-square form
        norm_case("norm_grad_odd", "norm_backward", 777, 1111, dtype="f16", rms=True),
        # the first projection of a 6144 x 16384 feed-forward block, one token: weight reads
        linear_case("linear_token", "linear_forward", 1, 6144, 16384, "silu", True, False),
        # a decode batch through a square projection that closes a residual branch
        linear_case("linear_batch", "linear_forward", 37, 4096, 4096, "none", True, True, dtype="f16"),
        # a prompt of 8192 tokens through a feed-forward projection that saves what its gradient needs
        linear_case("linear_prompt", "linear_forward", 8192, 4096, 16384, "gelu_tanh", True, False, save=True),
        # its training step's gradient at 4000 tokens of the 5120-wide model
        linear_case("linear_grad", "linear_backward", 4000, 5120, 5120, "gelu", True, False),
        # eight tokens, top 8 of 128 experts: a few rows for some experts, none for most
        grouped_case("grouped_decode", "grouped_forward", 64, 128, 2048, 768),
        # 8192 tokens, top 8 of 128 experts, the hottest with about four times the mean load
        grouped_case("grouped_prompt", "grouped_forward", 65536, 128, 4096, 1536),
        # gradient of the rows, 4096 tokens, top 6 of 160 experts
        grouped_case("grouped_rows_grad", "grouped_dgrad", 24576, 160, 5120, 1536, skew=0.5),
        # gradient of 16 experts' weights in 32 bits, for 32768 rows
        grouped_case("grouped_weight_grad", "grouped_wgrad", 32768, 16, 4096, 1536, grad="f32", skew=0.5),
    ]


def _size(rng, low, high):
    """A whole number between the two, even over its logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def _width(rng, low, high):
    """A matrix's width: mostly a multiple of 64 or 8, one time in five any number."""
    n, kind = _size(rng, low, high), rng.random()
    step = 64 if kind < 0.5 else 8 if kind < 0.8 else 1
    return max(step, n // step * step)


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "linear_forward", "linear_backward", "grouped_forward",
                     "grouped_dgrad", "grouped_wgrad"])
    if op.startswith("norm"):
        c = norm_case("", op, _size(rng, 1, 16384), _size(rng, 64, 16384), rng.choice(["bf16", "bf16", "f16", "f32"]),
                      rng.choice(["same", "f32"]), rng.random() < 0.4)
        c["rows"] = min(c["rows"], (1 << 25) // c["cols"])
    elif op.startswith("linear"):
        n_in, n_out = _width(rng, 64, 8192), _width(rng, 64, 8192)
        c = linear_case("", op, _size(rng, 1, 8192), n_in, n_out, rng.choice(ACTS), rng.random() < 0.7,
                        rng.random() < 0.5, rng.choice(["bf16", "bf16", "f16"]), rng.choice(["same", "f32"]),
                        rng.random() < 0.5)
        c["rows"] = max(1, min(c["rows"], 200_000_000_000 // (n_in * n_out)))
    else:
        n_in, n_out = _width(rng, 128, 5120), _width(rng, 128, 5120)
        experts = _size(rng, 1, 160)
        experts = max(1, min(experts, 1_000_000_000 // (n_in * n_out)))
        c = grouped_case("", op, _size(rng, 1, 32768), experts, n_in, n_out, rng.choice(["bf16", "bf16", "f16"]),
                         rng.choice(["same", "f32"]), rng.choice([0.0, 0.5, 1.2]))
        c["rows"] = max(1, min(c["rows"], 200_000_000_000 // (n_in * n_out)))
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs

def _randn(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype).mul_(scale)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"].startswith("norm"):
        rows, cols = case["rows"], case["cols"]
        pt = torch.float32 if case["params"] == "f32" else dt
        # a residual stream: a mean of its own in each row, a few wide channels
        x = torch.randn((rows, cols), generator=gen, device=DEV)
        x.mul_(1 + 9 * (torch.rand(cols, generator=gen, device=DEV) < 0.01)).mul_(0.5)
        x.add_(0.3 * torch.randn((rows, 1), generator=gen, device=DEV))
        s["x"] = x.to(dt)
        s["gamma"] = (1 + 0.2 * torch.randn(cols, generator=gen, device=DEV)).to(pt)
        s["beta"] = (0.1 * torch.randn(cols, generator=gen, device=DEV)).to(pt)
        if case["op"] == "norm_backward":
            # what the forward pass kept: each row's mean and reciprocal deviation
            f = s["x"].float()
            mean = torch.zeros(rows, device=DEV) if case["rms"] else f.mean(1)
            s["mean"], s["rstd"] = mean, torch.rsqrt((f - mean[:, None]).square().mean(1) + EPS)
            s["dy"] = _randn(gen, (rows, cols), dt)
        return s
    if case["op"].startswith("linear"):
        rows, n_in, n_out = case["rows"], case["n_in"], case["n_out"]
        pt = torch.float32 if case["params"] == "f32" else dt
        s["x"] = _randn(gen, (rows, n_in), dt)
        s["w"] = _randn(gen, (n_out, n_in), dt, n_in ** -0.5)
        s["bias"] = _randn(gen, (n_out,), torch.float32, 0.2).to(pt) if case["bias"] else None
        if case["op"] == "linear_forward":
            s["residual"] = _randn(gen, (rows, n_out), dt) if case["residual"] else None
        else:
            s["dy"] = _randn(gen, (rows, n_out), dt)
            # the pre-activation that the forward pass saved
            s["pre"] = _randn(gen, (rows, n_out), dt) if case["act"] != "none" else None
        return s
    rows, E, n_in, n_out = case["rows"], case["experts"], case["n_in"], case["n_out"]
    r = np.random.RandomState(seed % (1 << 32))
    share = (np.arange(1, E + 1) ** -float(case["skew"]))[r.permutation(E)]
    counts = r.multinomial(rows, share / share.sum())
    ends = np.concatenate([[0], np.cumsum(counts)])
    s["offsets"] = torch.from_numpy(ends.astype(np.int32)).to(DEV)
    s["spans"] = [(int(a), int(b)) for a, b in zip(ends[:-1], ends[1:])]
    if case["op"] != "grouped_dgrad":
        s["x"] = _randn(gen, (rows, n_in), dt)
    if case["op"] != "grouped_forward":
        s["dy"] = _randn(gen, (rows, n_out), dt)
    if case["op"] != "grouped_wgrad":
        s["w"] = _randn(gen, (E, n_out, n_in), dt, n_in ** -0.5)
    return s


# ------------------------------------------------------------ plain forms

def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    dt = DTYPES[case["dtype"]]
    if op == "norm_forward":
        x = s["x"].float()
        c = x if case["rms"] else x - x.mean(1, keepdim=True)
        y = c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
        return (y * s["gamma"].float() + s["beta"].float()).to(dt)
    if op == "norm_backward":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        n = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["gamma"].float()
        dx = g - n * (g * n).mean(1, keepdim=True)
        if not case["rms"]:
            dx = dx - g.mean(1, keepdim=True)
        pt = s["gamma"].dtype
        return {"dx": (dx * rstd).to(dt), "dgamma": (dy * n).sum(0).to(pt), "dbeta": dy.sum(0).to(pt)}
    if op == "linear_forward":
        z = s["x"].float() @ s["w"].float().T
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dt), "pre": z.to(dt)} if case["save"] else y.to(dt)
    if op == "linear_backward":
        g = s["dy"].float()
        if s["pre"] is not None:
            g = g * _act_grad(s["pre"].float(), case["act"])
        out = {"dx": (g @ s["w"].float()).to(dt), "dw": (g.T @ s["x"].float()).to(dt)}
        if s["bias"] is not None:
            out["dbias"] = g.sum(0).to(s["bias"].dtype)
        return out
    # one product per expert that has rows
    if op == "grouped_forward":
        return torch.cat([s["x"][a:b].float() @ s["w"][e].float().T for e, (a, b) in enumerate(s["spans"]) if b > a]).to(dt)
    if op == "grouped_dgrad":
        return torch.cat([s["dy"][a:b].float() @ s["w"][e].float() for e, (a, b) in enumerate(s["spans"]) if b > a]).to(dt)
    gt = torch.float32 if case["grad"] == "f32" else dt
    return torch.stack([(s["dy"][a:b].float().T @ s["x"][a:b].float()).to(gt) for a, b in s["spans"]])


# -------------------------------------------------- the framework's calls

def _own(s):
    import expert_ffn_dispatch_amd as moe
    case, op = s["case"], s["case"]["op"]
    if op == "norm_forward":
        return moe.moe_layer_norm(s["x"], s["gamma"], s["beta"], eps=EPS, rms=case["rms"])
    if op == "norm_backward":
        dx, dgamma, dbeta = moe.moe_layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"],
                                                        rms=case["rms"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "linear_forward":
        if case["save"]:
            y, pre = moe.moe_linear(s["x"], s["w"], s["bias"], s["residual"], act=case["act"], want_pre=True)
            return {"y": y, "pre": pre}
        return moe.moe_linear(s["x"], s["w"], s["bias"], s["residual"], act=case["act"])
    if op == "linear_backward":
        bias = s["bias"]
        dx, dw, dbias = moe.moe_linear_backward(s["dy"], s["x"], s["w"], s["pre"], act=case["act"],
                                                want_dbias=bias is not None,
                                                bias_dtype=None if bias is None else bias.dtype)
        out = {"dx": dx, "dw": dw}
        if bias is not None:
            out["dbias"] = dbias
        return out
    if op == "grouped_forward":
        return moe.moe_grouped_matmul(s["x"], s["offsets"], s["w"])
    if op == "grouped_dgrad":
        return moe.moe_grouped_matmul_dgrad(s["dy"], s["offsets"], s["w"])
    gt = torch.float32 if case["grad"] == "f32" else DTYPES[case["dtype"]]
    return moe.moe_grouped_matmul_wgrad(s["dy"], s["x"], s["offsets"], dtype=gt)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------ work and exact values

def work(case):
    b = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("norm"):
        n, cols = case["rows"] * case["cols"], case["cols"]
        p = 4 if case["params"] == "f32" else b
        if case["op"] == "norm_forward":
            return {"bytes": 2 * n * b + 2 * cols * p, "flops": 8 * n}
        return {"bytes": 3 * n * b + 3 * cols * p + 8 * case["rows"], "flops": 14 * n}
    n_in, n_out, rows = case["n_in"], case["n_out"], case["rows"]
    if case["op"] == "linear_forward":
        outs = 1 + case["residual"] + case["save"]
        return {"bytes": b * (rows * n_in + n_in * n_out + rows * n_out * outs), "flops": 2 * rows * n_in * n_out}
    if case["op"] == "linear_backward":
        ins = 1 + (case["act"] != "none")
        return {"bytes": b * (2 * rows * n_in + 2 * n_in * n_out + rows * n_out * ins), "flops": 4 * rows * n_in * n_out}
    used = min(case["experts"], rows)
    if case["op"] == "grouped_wgrad":
        g = 4 if case["grad"] == "f32" else b
        return {"bytes": b * rows * (n_in + n_out) + g * case["experts"] * n_in * n_out, "flops": 2 * rows * n_in * n_out}
    return {"bytes": b * (rows * (n_in + n_out) + used * n_in * n_out), "flops": 2 * rows * n_in * n_out}


def exact(case, seed):
    """run()'s outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and k not in ("offsets", "w")}
    op = case["op"]
    if op == "norm_forward":
        dev = d["x"] - (0 if case["rms"] else d["x"].sum(1, keepdim=True) / case["cols"])
        second = dev.pow(2).sum(1, keepdim=True) / case["cols"]
        return dev / (second + EPS).sqrt() * d["gamma"] + d["beta"]
    if op == "norm_backward":
        xhat = (d["x"] - d["mean"].unsqueeze(1)) * d["rstd"].unsqueeze(1)
        t = d["dy"] * d["gamma"]
        inner = torch.linalg.vecdot(t, xhat).unsqueeze(1) / case["cols"]
        shift = 0 if case["rms"] else t.sum(1, keepdim=True) / case["cols"]
        return {"dx": d["rstd"].unsqueeze(1) * (t - shift - xhat * inner), "dgamma": (d["dy"] * xhat).sum(0),
                "dbeta": d["dy"].sum(0)}
    if op.startswith("linear"):
        w = s["w"].double()
        z = torch.addmm(d["bias"], d["x"], w.t()) if op == "linear_forward" and s["bias"] is not None else None
        if op == "linear_forward":
            z = torch.mm(d["x"], w.t()) if z is None else z
            a = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0),
                 "gelu": lambda v: v * torch.special.ndtr(v),
                 "gelu_tanh": lambda v: v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3)),
                 "silu": lambda v: v * torch.sigmoid(v)}[case["act"]](z)
            y = a if s["residual"] is None else a + d["residual"]
            return {"y": y, "pre": z} if case["save"] else y
        g = d["dy"]
        if case["act"] != "none":
            p = d["pre"]
            if case["act"] == "relu":
                g = torch.where(p > 0, g, torch.zeros_like(g))
            elif case["act"] == "gelu":
                g = g * (torch.special.ndtr(p) + p / math.sqrt(2 * math.pi) * torch.exp(-p * p / 2))
            else:
                # v * sigmoid(u(v)): sigmoid + v sigmoid (1 - sigmoid) u'
                k = math.sqrt(8 / math.pi)
                u, du = (p, 1.0) if case["act"] == "silu" else (k * (p + 0.044715 * p ** 3), k * (1 + 0.134145 * p ** 2))
                sg = torch.sigmoid(u)
                g = g * (sg + p * sg * torch.sigmoid(-u) * du)
        out = {"dx": torch.mm(g, w), "dw": torch.mm(g.t(), d["x"])}
        if case["bias"]:
            out["dbias"] = g.sum(0)
        return out
    if op == "grouped_wgrad":
        out = torch.zeros((case["experts"], case["n_out"], case["n_in"]), dtype=torch.float64, device=DEV)
        for e, (a, b) in enumerate(s["spans"]):
            torch.mm(d["dy"][a:b].t(), d["x"][a:b], out=out[e])
        return out
    src = d["x"] if op == "grouped_forward" else d["dy"]
    out = torch.empty((case["rows"], case["n_out"] if op == "grouped_forward" else case["n_in"]), dtype=torch.float64, device=DEV)
    for e, (a, b) in enumerate(s["spans"]):
        if b > a:
            w = s["w"][e].double()
            out[a:b] = torch.mm(src[a:b], w.t() if op == "grouped_forward" else w)
    return out
