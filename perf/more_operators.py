"""Cases, plain forms and calls of what trains and serves the experts: the gated feed-forward projections with
their gradients, the AdamW step that takes those gradients, and products with 4-bit weights.

Sizes are those of the workloads in datagen/configs.py (hidden sizes 2048, 4096, 5120 and 6144, expert widths 768,
1536 and 16384, 8 to 160 experts, 1 to 65536 rows) and numbers between them.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
BETA1, BETA2, EPS, DECAY, LR = 0.9, 0.95, 1e-8, 0.1, 3e-4
BLOCK = 128                     # values of an 8-bit state that share an exponent
GROUP = 32                      # 4-bit weights that share an exponent
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def gated_case(name, op, rows, experts, n_in, width, act="silu", dtype="bf16", save=False, skew=0.5):
    """experts 0: one dense pair of projections."""
    return {"name": name, "op": op, "rows": rows, "experts": experts, "n_in": n_in, "width": width, "act": act,
            "dtype": dtype, "save": save, "skew": skew}


def adamw_case(name, tensors, numel, ragged, states, params="f32", grads="bf16", copy="bf16", step=10):
    """copy: the type of the weights that the next forward pass reads ("": the parameters themselves)."""
    return {"name": name, "op": "adamw", "tensors": tensors, "numel": numel, "ragged": ragged, "states": states,
            "params": params, "grads": grads, "copy": copy, "step": step}


def fp4_case(name, rows, experts, n_in, n_out, act="none", bias=False, residual=False, gated=False, dtype="bf16",
             skew=0.5):
    return {"name": name, "op": "fp4", "rows": rows, "experts": experts, "n_in": n_in, "n_out": n_out, "act": act,
            "bias": bias, "residual": residual, "gated": gated, "dtype": dtype, "skew": skew}


def listed():
    return [
        # one token through a 6144-wide block's gated projections of 16384: two weight matrices are read
        gated_case("gated_token", "gated_forward", 1, 0, 6144, 16384),
        # 8192 tokens, top 8 of 128 experts, the hottest with about four times the mean load, in a training step
        # that saves what the gradient needs
        gated_case("gated_prompt", "gated_forward", 65536, 128, 4096, 1536, save=True, skew=1.2),
        # a ragged micro-batch of odd widths in fp16 through a dense block
        gated_case("gated_grad_odd", "gated_backward", 777, 0, 1111, 2222, act="gelu_tanh", dtype="f16"),
        # gradients of 16 local experts of 1536, 32768 rows
        gated_case("gated_grad", "gated_backward", 32768, 16, 4096, 1536),
        # the vectors of a small model (norm weights): one step is all latency
        adamw_case("adamw_vectors", 12, 2048, False, "f32", grads="f32", copy=""),
        # 16 experts of 4096 x 1536, three matrices each: 32-bit masters, bf16 gradients, bf16 working copies
        adamw_case("adamw_experts", 48, 4096 * 1536, False, "f32"),
        # tensors of odd sizes, bf16 parameters updated in place, 8-bit states
        adamw_case("adamw8_ragged", 37, 50021, True, "fp8", params="bf16", copy=""),
        # the same experts with 8-bit states: what bounds the step is what is left
        adamw_case("adamw8_experts", 48, 4096 * 1536, False, "fp8"),
        # one token through a projection of 6144 -> 16384 with 4-bit weights: weight reads
        fp4_case("fp4_token", 1, 0, 6144, 16384, act="silu", bias=True),
        # a prompt of 2000 tokens through a square projection that closes a residual branch, fp16
        fp4_case("fp4_prompt", 2000, 0, 5120, 5120, residual=True, dtype="f16"),
        # eight tokens, top 8 of 128 experts: a few rows for some experts, none for the others
        fp4_case("fp4_experts_decode", 64, 128, 2048, 768),
        # 512 tokens, top 8 of 128 experts, both gated projections
        fp4_case("fp4_experts_gated", 4096, 128, 2048, 768, act="silu", gated=True),
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
    op = rng.choice(["gated_forward", "gated_backward", "adamw", "adamw8", "fp4", "fp4"])
    if op.startswith("gated"):
        n_in, width = _width(rng, 64, 6144), _width(rng, 64, 6144)
        experts = 0 if rng.random() < 0.5 else max(1, min(_size(rng, 1, 160), 500_000_000 // (n_in * width)))
        c = gated_case("", op, _size(rng, 1, 32768), experts, n_in, width, rng.choice(ACTS),
                       rng.choice(["bf16", "bf16", "f16"]), op == "gated_forward" and rng.random() < 0.5,
                       rng.choice([0.0, 0.5, 1.2]))
        c["rows"] = max(1, min(c["rows"], 150_000_000_000 // (n_in * width)))
    elif op.startswith("adamw"):
        tensors = _size(rng, 1, 60)
        numel = _size(rng, 64, 200_000_000 // tensors)
        params = rng.choice(["f32", "f32", "bf16", "f16"])
        c = adamw_case("", tensors, numel, rng.random() < 0.5, "f32" if op == "adamw" else "fp8", params,
                       rng.choice(["bf16", "f16", "f32"]),
                       rng.choice(["", "bf16", "f16"]) if params == "f32" else "", rng.randint(1, 1000))
    else:
        # a contraction of whole groups, any number of outputs
        n_in, n_out = max(GROUP, _size(rng, 64, 8192) // GROUP * GROUP), _width(rng, 64, 8192)
        experts = 0 if rng.random() < 0.5 else max(1, min(_size(rng, 1, 160), 500_000_000 // (n_in * n_out)))
        gated = rng.random() < 0.4
        dense = experts == 0 and not gated
        c = fp4_case("", _size(rng, 1, 8192), experts, n_in, n_out, rng.choice(ACTS) if dense or gated else "none",
                     dense and rng.random() < 0.5, dense and rng.random() < 0.5, gated,
                     rng.choice(["bf16", "bf16", "f16"]), rng.choice([0.0, 0.5, 1.2]))
        c["rows"] = max(1, min(c["rows"], 100_000_000_000 // (n_in * n_out)))
    del c["name"]
    return c


def _numels(case):
    n = case["numel"]
    return [max(1, n * (3 + i * 7 % 11) // 9 + i) if case["ragged"] else n for i in range(case["tensors"])]


# ----------------------------------------------------------------- inputs

def _randn(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype).mul_(scale)


def _spans(case, seed):
    """Rows dealt to the experts by a power of their rank, in an order of the seed's: offsets, and spans."""
    rows, E = case["rows"], case["experts"]
    if E == 0:
        return None, [(0, rows)]
    r = np.random.RandomState(seed % (1 << 32))
    share = (np.arange(1, E + 1) ** -float(case["skew"]))[r.permutation(E)]
    ends = np.concatenate([[0], np.cumsum(r.multinomial(rows, share / share.sum()))])
    return torch.from_numpy(ends.astype(np.int32)).to(DEV), [(int(a), int(b)) for a, b in zip(ends[:-1], ends[1:])]


def _fp4_weights(gen, shape):
    """Normal weights in 4 bits: codes (two to a byte, the first in the low half) and an exponent for each group."""
    w = torch.randn((*shape[:-1], shape[-1] // GROUP, GROUP), generator=gen, device=DEV).mul_(shape[-1] ** -0.5)
    e = torch.floor(torch.log2(w.abs().amax(-1, keepdim=True).clamp_min(1e-30))) - 2
    w.mul_(torch.exp2(-e))
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.zeros(w.shape, dtype=torch.uint8, device=DEV)
    for m in mid:
        code += w.abs() > m
    code += (w < 0).to(torch.uint8) * 8
    code = code.reshape(shape)
    return code[..., 0::2] | code[..., 1::2] << 4, (e.squeeze(-1) + 127).to(torch.uint8)


def _flat(numels):
    """Tensors in one buffer, each at a multiple of 128 values: where they start, and the buffer's length."""
    starts, at = [], 0
    for n in numels:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    return starts, at


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "adamw":
        numels = _numels(case)
        starts, total = _flat(numels)
        s["starts"], s["numels"] = starts, numels
        spans = list(zip(starts, numels))
        # one buffer of each kind, as a program that trains keeps it, with zeros between the tensors
        live = torch.zeros(total, dtype=torch.bool, device=DEV)
        for a, n in spans:
            live[a:a + n] = True

        def buffer(dtype, scale):
            return torch.randn(total, generator=gen, device=DEV).mul_(scale).mul_(live).to(dtype)

        s["param"] = buffer(DTYPES[case["params"]], 0.02)
        s["grad"] = buffer(DTYPES[case["grads"]], 1e-3 * 64)
        s["copy"] = s["param"].to(DTYPES[case["copy"]]) if case["copy"] else None
        s["grad_scale"] = torch.tensor([1 / 64], device=DEV)          # a loss scale, or the clipping of a norm
        m = buffer(torch.float32, 3e-4)
        v = buffer(torch.float32, 1e-3).square_()
        if case["states"] == "fp8":
            s["m"], s["m_exp"] = _encode(m, None)
            s["v"], s["v_exp"] = _encode(v.sqrt(), None)
        else:
            s["m"], s["v"] = m, v
        if own:                                                       # the list of tensors, looked over once
            import expert_ffn_dispatch_amd as moe
            view = lambda t: [t[a:a + n] for a, n in spans]           # noqa: E731
            if case["states"] == "fp8":
                exps = lambda t: [t[a // BLOCK:a // BLOCK - (-n // BLOCK)] for a, n in spans]  # noqa: E731
                m = [moe.Fp8Moment(c, e) for c, e in zip(view(s["m"]), exps(s["m_exp"]))]
                v = [moe.Fp8Moment(c, e) for c, e in zip(view(s["v"]), exps(s["v_exp"]))]
            else:
                m, v = view(s["m"]), view(s["v"])
            s["plan"] = moe.AdamWTensors(view(s["param"]), m, v, copies=view(s["copy"]) if case["copy"] else None)
            s["grads"] = view(s["grad"])
        return s
    dt = DTYPES[case["dtype"]]
    rows, E, n_in = case["rows"], case["experts"], case["n_in"]
    lead = (E,) if E else ()
    s["offsets"], s["spans"] = _spans(case, seed)
    s["x"] = _randn(gen, (rows, n_in), dt)
    if case["op"] == "fp4":
        n_out = case["n_out"]
        s["w"] = [_fp4_weights(gen, (*lead, n_out, n_in)) for _ in range(1 + case["gated"])]
        s["bias"] = _randn(gen, (n_out,), dt, 0.2) if case["bias"] else None
        s["residual"] = _randn(gen, (rows, n_out), dt) if case["residual"] else None
        return s
    width = case["width"]
    s["w_gate"] = _randn(gen, (*lead, width, n_in), dt, n_in ** -0.5)
    s["w_up"] = _randn(gen, (*lead, width, n_in), dt, n_in ** -0.5)
    if case["op"] == "gated_backward":
        s["dh"] = _randn(gen, (rows, width), dt)
        # what the forward pass saved
        s["gate"], s["up"] = _randn(gen, (rows, width), dt), _randn(gen, (rows, width), dt)
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
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _decode(code, exp):
    """Values of 8-bit states: E4M3 codes times two to the block's exponent."""
    scale = (exp.to(torch.int32) << 23).view(torch.float32)
    return (code.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _encode(x, draws):
    """Blocks of 128 values as E4M3 codes and an exponent: the least power of two that brings the largest to 448 or
    below.  draws: whole numbers below 2^16, the part of a step (in 1 / 65536) from which a value rounds up; None:
    to nearest."""
    top = x.abs().view(-1, BLOCK).amax(1)
    exp = (((top.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=1)
    f = (x.view(-1, BLOCK) * ((254 - exp) << 23).view(torch.float32)[:, None]).view(-1)
    mag = f.abs()
    small = mag < 2.0 ** -6                                           # one step below the smallest exponent
    bits = torch.where(small, mag + 2.0 ** -6, mag).view(torch.int32)
    code = ((bits + (0x80000 if draws is None else draws << 4)) >> 20) - 960 - 8 * small.to(torch.int32)
    code = code.clamp(max=126) | (f.signbit().to(torch.int32) << 7)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), exp.to(torch.uint8)


def _draws(s):
    """For each value a number below 2^32 from its place in its tensor and the step."""
    at = torch.arange(len(s["param"]), device=DEV)
    first = torch.repeat_interleave(torch.tensor(s["starts"], device=DEV),
                                    torch.tensor([-(-n // BLOCK) * BLOCK for n in s["numels"]], device=DEV),
                                    output_size=len(s["param"]))
    mask = 0xFFFFFFFF
    z = ((at - first) + s["case"]["step"] * 0x9E3779B9) & mask
    z = ((z ^ (z >> 16)) * 0x6C8E9CF5) & mask
    z = ((z ^ (z >> 15)) * 0x2B7E1517) & mask
    return z ^ (z >> 16)


def _plain_adamw(s):
    case = s["case"]
    eight = case["states"] == "fp8"
    c1, c2 = 1 - BETA1 ** case["step"], 1 - BETA2 ** case["step"]
    m = _decode(s["m"], s["m_exp"]) if eight else s["m"]
    v = _decode(s["v"], s["v_exp"]).square() if eight else s["v"]
    g = s["grad"].float() * s["grad_scale"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    root = torch.sqrt(v)
    p = s["param"].float() * (1 - LR * DECAY) - (m / (root * (1 / math.sqrt(c2)) + EPS)) * (LR / c1)
    s["param"].copy_(p)
    out = {"param": s["param"]}
    if s["copy"] is not None:
        s["copy"].copy_(p)
        out["copy"] = s["copy"]
    if eight:
        z = _draws(s)
        code, exp = _encode(m, (z & 0xFFFF).to(torch.int32))
        s["m"].copy_(code), s["m_exp"].copy_(exp)
        code, exp = _encode(root, (z >> 16).to(torch.int32))
        # no divisor that was there is lost to rounding
        code = torch.where(root > 0, code.view(torch.uint8).clamp(min=1), code.view(torch.uint8))
        s["v"].copy_(code.view(torch.float8_e4m3fn)), s["v_exp"].copy_(exp)
        return {**out, "m": s["m"], "m_exp": s["m_exp"], "v": s["v"], "v_exp": s["v_exp"]}
    s["m"].copy_(m), s["v"].copy_(v)
    return {**out, "m": s["m"], "v": s["v"]}


def _fp4_values(codes, exps):
    table = torch.tensor(FP4 + tuple(-v for v in FP4), device=DEV)
    w = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1)
    w = w.view(*exps.shape, GROUP) * (exps.to(torch.int32) << 23).view(torch.float32)[..., None]
    return w.view(*codes.shape[:-1], -1)


def _by_expert(f, s, *operands):
    """f of each expert's rows of the operands (and the weights' index), one after the other."""
    if s["offsets"] is None:
        return f(..., *operands)
    parts = [f(e, *(t[a:b] for t in operands)) for e, (a, b) in enumerate(s["spans"]) if b > a]
    return tuple(torch.cat(p) for p in zip(*parts)) if isinstance(parts[0], tuple) else torch.cat(parts)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "adamw":
        return _plain_adamw(s)
    dt, act = DTYPES[case["dtype"]], case["act"]
    if op == "fp4":
        def product(e, x):
            z = [x.float() @ _fp4_values(c[e], x4[e]).T for c, x4 in s["w"]]
            if case["gated"]:
                return (_act(z[0], act) * z[1]).to(dt)
            z = z[0] if s["bias"] is None else z[0] + s["bias"].float()
            y = _act(z, act)
            return (y if s["residual"] is None else y + s["residual"].float()).to(dt)
        return _by_expert(product, s, s["x"])
    if op == "gated_forward":
        def forward(e, x):
            gate, up = x.float() @ s["w_gate"][e].float().T, x.float() @ s["w_up"][e].float().T
            h = (_act(gate, act) * up).to(dt)
            return (h, gate.to(dt), up.to(dt)) if case["save"] else h
        out = _by_expert(forward, s, s["x"])
        return dict(zip(("h", "gate", "up"), out)) if case["save"] else out
    z, dh = s["gate"].float(), s["dh"].float()
    dgate, dup = dh * s["up"].float() * _act_grad(z, act), dh * _act(z, act)
    x = s["x"].float()
    out = {"dx": _by_expert(lambda e, g, u: g @ s["w_gate"][e].float() + u @ s["w_up"][e].float(), s, dgate, dup).to(dt)}
    for name, g in (("dw_gate", dgate), ("dw_up", dup)):
        dw = [(g[a:b].T @ x[a:b]).to(dt) for a, b in s["spans"]]
        out[name] = dw[0] if s["offsets"] is None else torch.stack(dw)
    return out


# -------------------------------------------------- the framework's calls

def _own(s):
    import expert_ffn_dispatch_amd as moe
    case, op = s["case"], s["case"]["op"]
    if op == "adamw":
        moe.moe_adamw(s["plan"], s["grads"], step=case["step"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS,
                      weight_decay=DECAY, grad_scale=s["grad_scale"])
        names = ("param", "copy", "m", "m_exp", "v", "v_exp")
        return {k: s[k] for k in names if s.get(k) is not None}
    act, offsets = case["act"], s["offsets"]
    if op == "fp4":
        w = [moe.Fp4Weights(c, e) for c, e in s["w"]]
        if offsets is None:
            if case["gated"]:
                return moe.moe_gated_linear_fp4(s["x"], w[0], w[1], act=act)
            return moe.moe_linear_fp4(s["x"], w[0], s["bias"], s["residual"], act=act)
        if case["gated"]:
            return moe.moe_grouped_gated_fp4(s["x"], offsets, w[0], w[1], act=act)
        return moe.moe_grouped_matmul_fp4(s["x"], offsets, w[0])
    if op == "gated_forward":
        if offsets is None:
            out = moe.moe_gated_linear(s["x"], s["w_gate"], s["w_up"], act=act, want_pre=case["save"])
        else:
            out = moe.moe_grouped_gated(s["x"], offsets, s["w_gate"], s["w_up"], act=act, want_pre=case["save"])
        return dict(zip(("h", "gate", "up"), out)) if case["save"] else out
    if offsets is None:
        out = moe.moe_gated_linear_backward(s["dh"], s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"], act=act)
    else:
        out = moe.moe_grouped_gated_backward(s["dh"], s["x"], offsets, s["w_gate"], s["w_up"], s["gate"], s["up"],
                                             act=act)
    return dict(zip(("dx", "dw_gate", "dw_up"), out))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------ work and exact values

def work(case):
    if case["op"] == "adamw":
        n = sum(_numels(case))
        size = lambda t: 4 if case[t] == "f32" else 2                 # noqa: E731
        states = 4 * (1 + 1 / BLOCK) if case["states"] == "fp8" else 16
        return {"bytes": n * (2 * size("params") + size("grads") + states + (size("copy") if case["copy"] else 0)),
                "flops": 14 * n}
    rows, E, n_in = case["rows"], case["experts"], case["n_in"]
    used = min(E, rows) if E else 1
    if case["op"] == "fp4":
        n_out, mats = case["n_out"], 1 + case["gated"]
        return {"bytes": 2 * rows * (n_in + n_out * (1 + case["residual"])) + mats * used * n_out * n_in * 17 / 32,
                "flops": 2 * mats * rows * n_in * n_out}
    width = case["width"]
    if case["op"] == "gated_forward":
        return {"bytes": 2 * rows * (n_in + width * (3 if case["save"] else 1)) + 4 * used * n_in * width,
                "flops": 4 * rows * n_in * width}
    return {"bytes": 2 * rows * (2 * n_in + 3 * width) + 4 * (used + max(E, 1)) * n_in * width,
            "flops": 8 * rows * n_in * width}


def _exact_act(z, act):
    """The activation and its slope, in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z / math.sqrt(2 * math.pi) * torch.exp(-z * z / 2)
    # v sigmoid(u(v)), and sigmoid + v sigmoid (1 - sigmoid) u'
    k = math.sqrt(8 / math.pi)
    u, du = (z, 1.0) if act == "silu" else (k * (z + 0.044715 * z ** 3), k * (1 + 0.134145 * z ** 2))
    sg = torch.sigmoid(u)
    return z * sg, sg + z * sg * torch.sigmoid(-u) * du


def exact(case, seed):
    """run()'s outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "adamw":
        def moments(name):
            if case["states"] != "fp8":
                return s[name].double()
            two = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=DEV), s[name + "_exp"].double() - 127)
            d = (s[name].double().view(-1, BLOCK) * two[:, None]).flatten()
            return d if name == "m" else d ** 2
        t, g = case["step"], s["grad"].double() / 64
        m = torch.lerp(g, moments("m"), BETA1)
        v = torch.lerp(g ** 2, moments("v"), BETA2)
        p = s["param"].double()
        p = p - LR * (DECAY * p + m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)) ** 0.5 + EPS))
        out = {"param": p, "copy": p if case["copy"] else None}
        if case["states"] == "fp8":                                   # codes of rounded states: no value of their own
            return {**out, "m": None, "m_exp": None, "v": None, "v_exp": None}
        return {**out, "m": m, "v": v}
    rows, dense = case["rows"], s["offsets"] is None
    pick = lambda w, e: w if dense else w[e]                          # noqa: E731
    spans = [(e, a, b) for e, (a, b) in enumerate(s["spans"]) if b > a]
    if case["op"] == "fp4":
        table = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12], dtype=torch.float64, device=DEV)
        y = torch.empty((rows, case["n_out"]), dtype=torch.float64, device=DEV)
        for e, a, b in spans:
            z = []
            for codes, exps in s["w"]:
                c = pick(codes, e).long()
                half = torch.ldexp(torch.ones_like(exps, dtype=torch.float64)[e if not dense else ...],
                                   pick(exps, e).long() - 128).repeat_interleave(GROUP, -1)
                w = torch.empty(half.shape, dtype=torch.float64, device=DEV)
                w[:, 0::2], w[:, 1::2] = table[c % 16], table[c // 16]
                z.append(torch.mm(s["x"][a:b].double(), (w * half).t()))
            if case["gated"]:
                y[a:b] = _exact_act(z[0], case["act"])[0] * z[1]
            else:
                y[a:b] = _exact_act(z[0] + (s["bias"].double() if case["bias"] else 0), case["act"])[0]
        return y + s["residual"].double() if case["residual"] else y
    width, n_in = case["width"], case["n_in"]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=DEV)  # noqa: E731
    if case["op"] == "gated_forward":
        gate, up = new(rows, width), new(rows, width)
        for e, a, b in spans:
            xd = s["x"][a:b].double()
            gate[a:b], up[a:b] = torch.mm(xd, pick(s["w_gate"], e).double().t()), torch.mm(xd, pick(s["w_up"], e).double().t())
        h = _exact_act(gate, case["act"])[0] * up
        return {"h": h, "gate": gate, "up": up} if case["save"] else h
    value, slope = _exact_act(s["gate"].double(), case["act"])
    grads = {"dw_gate": s["dh"].double() * s["up"].double() * slope, "dw_up": s["dh"].double() * value}
    out = {"dx": new(rows, n_in)}
    for name, g in grads.items():
        out[name] = new(*(() if dense else (case["experts"],)), width, n_in)
        w = s["w" + name[2:]]
        for e, a, b in spans:
            out["dx"][a:b].addmm_(g[a:b], pick(w, e).double())
            torch.mm(g[a:b].t(), s["x"][a:b].double(), out=pick(out[name], e))
    return out
