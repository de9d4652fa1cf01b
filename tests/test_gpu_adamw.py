"""The AdamW step against the formulas in 64 bits, its 8-bit states against
their definition in whole numbers, and over many steps.

fp32 arithmetic: m and v are three and four roundings of 2^-24 of their terms'
sizes.  The step m / (sqrt(v) / sqrt(c2) + eps) lr / c1 is off by at most 12
such roundings (square root and reciprocal within 1 ulp of 2^-23, the others
2^-24), relative to its size where m is; p then is rounded by u of its type."""
import math

import pytest
import torch

import expert_ffn_dispatch_amd as moe
from test_gpu_operators import BF, DEV, F32, HF, check, gen, tiny, u

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def ref_step(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay, scale=1.0):
    """New p, m, v in 64 bits and the error that fp32 arithmetic may leave in each."""
    p, g, m, v = (t.double() for t in (p, g, m, v))
    g = g * scale
    m1, v1 = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    em = 4 * E * (beta1 * m.abs() + (1 - beta1) * g.abs())
    ev = 5 * E * v1
    den = v1.sqrt() / math.sqrt(1 - beta2 ** step) + eps
    size = lr / (1 - beta1 ** step)
    p1 = p * (1 - lr * weight_decay) - size * m1 / den
    ep = size / den * (1.01 * em + 12 * E * m1.abs()) + 3 * E * p.abs() + E * p1.abs()
    return p1, m1, v1, ep + 1e-44, em + 1e-44, ev + 1e-44


def make(g, numels, pt, gt, ct, shift=0):
    """Tensors of a list, each `shift` elements into a buffer of its own."""
    def t(n, dtype, scale=1.0):
        return (torch.randn(n + shift, generator=g, device=DEV) * scale).to(dtype)[shift:]
    out = []
    for n in numels:
        m, v = t(n, F32, 0.1), t(n, F32, 0.2).square()
        zero = torch.rand(n, generator=g, device=DEV) < 0.05
        m[zero], v[zero] = 0, 0
        gr = t(n, gt)
        gr[torch.rand(n, generator=g, device=DEV) < 0.05] = 0
        out.append(dict(p=t(n, pt), g=gr, m=m, v=v, c=None if ct is None else t(n, ct)))
    return out


def check_param(got, p, ep, what):
    """A parameter rounded to its type.  A value from max (1 + eps / 4) on (half a step past the largest) is infinity in
    that type: a zero gradient over a near-zero v takes a step that fp16 does not hold."""
    t = got.dtype
    top = float(torch.finfo(t).max)
    tol = u(t) * p.abs() + 1.01 * ep + tiny(t)
    over = p.abs() >= top * (1 + torch.finfo(t).eps / 4) if t == HF else torch.zeros_like(p, dtype=torch.bool)
    assert torch.equal(got[over].double(), torch.copysign(torch.full_like(p[over], math.inf), p[over])), what
    check(got[~over], p[~over], tol[~over], what)


NUMELS = [[1], [3, 4, 5], [2048, 2047, 2049, 8192, 8193], [0, 7, 0, 100001], list(range(1, 101)), [20_000_003]]


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("pt,gt,ct", [(F32, BF, BF), (F32, F32, None), (BF, BF, None), (HF, F32, None), (F32, HF, HF), (BF, F32, HF)])
@pytest.mark.parametrize("numels", NUMELS, ids=[f"{len(n)}x{sum(n)}" for n in NUMELS])
def test_step(numels, pt, gt, ct, shift):
    g = gen(sum(numels) + shift)
    ts = make(g, numels, pt, gt, ct, shift)
    scale = torch.tensor([0.5], device=DEV)
    want = [ref_step(t["p"], t["g"], t["m"], t["v"], 3, scale=0.5, **HYPER) for t in ts]
    plan = moe.AdamWTensors(*([t[k] for t in ts] for k in ("p", "m", "v")), copies=[t["c"] for t in ts])
    assert moe.moe_adamw(plan, [t["g"] for t in ts], step=3, grad_scale=scale, **HYPER) is None
    for t, (p, m, v, ep, em, ev) in zip(ts, want):
        check(t["m"], m, em, "m")
        check(t["v"], v, ev, "v")
        check_param(t["p"], p, ep, "param")
        if ct is not None:
            check_param(t["c"], p, ep, "copy")


def test_mixed_types_in_one_list_and_missing_gradients():
    g = gen(2)
    kinds = [(F32, BF, BF), (BF, F32, None), (HF, HF, None), (F32, F32, None)]
    ts = [t for k in kinds for t in make(g, [1000, 33], *k)]
    want = [ref_step(t["p"], t["g"], t["m"], t["v"], 1, **HYPER) for t in ts]
    before = {k: ts[2][k].clone() for k in ("p", "m", "v")}
    plan = moe.AdamWTensors(*([t[k] for t in ts] for k in ("p", "m", "v")), copies=[t["c"] for t in ts])
    moe.moe_adamw(plan, [None if i == 2 else t["g"] for i, t in enumerate(ts)], step=1, **HYPER)
    for i, (t, (p, m, v, ep, em, ev)) in enumerate(zip(ts, want)):
        if i == 2:
            assert all(torch.equal(t[k], before[k]) for k in before)
            continue
        check(t["m"], m, em, "m")
        check_param(t["p"], p, ep, "param")
    moe.moe_adamw(plan, [None] * len(ts), step=1, **HYPER)
    moe.moe_adamw(moe.AdamWTensors([], [], []), [], step=1, lr=1.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_no_eps_and_tiny_gradients(fp8):
    """Without eps the step is lr for the first gradient of any size whose square has bits: here second moments down to
    2^-128, 21 bits below which fp32 rounds (ref_step counts relative roundings: 2^-22 more of v, half that of its root)."""
    n = 2000
    e = torch.randint(-60, 20, (n,), generator=gen(3), device=DEV)
    grad = torch.ldexp(1 + torch.rand(n, generator=gen(4), device=DEV), e) * torch.where(e % 2 == 0, 1.0, -1.0)
    p = torch.ones(n, device=DEV)
    m, v = ([moe.Fp8Moment.zeros(p)] if fp8 else [torch.zeros_like(p)] for _ in range(2))
    want, _, _, ep, _, _ = ref_step(p, grad, torch.zeros_like(p), torch.zeros_like(p), 1, 1e-2, 0.9, 1 - 2.0 ** -8, 0.0, 0.0)
    moe.moe_adamw(moe.AdamWTensors([p], m, v), [grad], step=1, lr=1e-2, beta2=1 - 2.0 ** -8, eps=0.0, weight_decay=0.0)
    check(p, want, ep + 1e-2 * 2.0 ** -22, "param")


# ------------------------------------------------------------- 8-bit states

def draws(n, step):
    mask = 0xFFFFFFFF
    z = (torch.arange(n, device=DEV) + step * 0x9E3779B9) & mask
    z = ((z ^ (z >> 16)) * 0x6C8E9CF5) & mask
    z = ((z ^ (z >> 15)) * 0x2B7E1517) & mask
    z = z ^ (z >> 16)
    return z & 0xFFFF, z >> 16


def encode(x, u16):
    """Codes and exponents by the definition, in 64-bit whole numbers and fractions."""
    n = x.numel()
    pad = -(-n // 128) * 128 - n
    xb = torch.nn.functional.pad(x.double(), (0, pad)).view(-1, 128)
    top = xb.abs().amax(1)
    exp = torch.ceil(torch.log2(top.clamp_min(1e-300) / 448)).clamp(min=-126)
    exp = torch.where(top <= 448 * torch.exp2(exp - 1), exp - 1, exp)          # log2's last bit
    exp = torch.where(top > 448 * torch.exp2(exp), exp + 1, exp).clamp(min=-126)
    f = (xb * torch.exp2(-exp)[:, None]).view(-1)[:n].abs()
    low = torch.floor(torch.log2(f.clamp_min(2.0 ** -6)))
    unit = torch.exp2(low - 3)
    k = torch.floor(f / unit)
    # the part of a step, in the 16 bits that fp32 has below the code and above its own last four (of f plus 2^-6, where
    # the codes are subnormal: 2^-20 of a step)
    part = torch.floor((f / unit - k) * 65536 + u16.double() / 1.0 + 1e-9)
    value = (k + (part >= 65536)) * unit
    return torch.copysign(value, x.double()), (exp + 127).to(torch.uint8)


def values(moment):
    return moment.codes.view(torch.float8_e4m3fn).double(), moment.exps


def fp8_list(g, numels, pt, gt, ct, shift=0):
    ts = make(g, numels, pt, gt, ct, shift)
    for t in ts:
        n = t["p"].numel()
        for k in ("m", "v"):
            x = t[k] if k == "m" else t[k].sqrt()
            val, exp = encode(x, torch.full((n,), 32768, device=DEV))
            code = torch.empty(n + shift, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)[shift:]
            code.copy_(val.float().to(torch.float8_e4m3fn))
            t[k + "8"] = moe.Fp8Moment(code, exp)
    return ts


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("pt,gt,ct", [(F32, BF, BF), (BF, BF, None), (HF, F32, None), (F32, HF, HF)])
@pytest.mark.parametrize("numels", NUMELS[:5] + [[127, 128, 129], [3_000_001]], ids=lambda n: f"{len(n)}x{sum(n)}")
def test_step_with_8_bit_states(numels, pt, gt, ct, shift):
    g = gen(sum(numels) + 7)
    ts = fp8_list(g, numels, pt, gt, ct, shift)
    step = 5
    want = []
    for t in ts:
        m, r = t["m8"].values().double(), t["v8"].values().double()
        want.append(ref_step(t["p"], t["g"], m, r * r, step, **HYPER))
    plan = moe.AdamWTensors(*([t[k] for t in ts] for k in ("p", "m8", "v8")), copies=[t["c"] for t in ts])
    moe.moe_adamw(plan, [t["g"] for t in ts], step=step, **HYPER)
    for t, (p, m, v, ep, em, ev) in zip(ts, want):
        check_param(t["p"], p, ep, "param")
        if ct is not None:
            check_param(t["c"], p, ep, "copy")
        n = p.numel()
        lo, hi = draws(n, step)
        for name, x, bits in (("m8", m, lo), ("v8", v.sqrt(), hi)):
            code, exp = values(t[name])
            rv, re = encode(x, bits)
            if name == "v8":
                rv = torch.where((x > 0) & (rv == 0), 2.0 ** -9, rv)
            # the kernel's fp32 x is within 2^-21 of this one, so a code may fall on the other side of its border for
            # values that are 2^-21 * 16 steps from it (once in 2^-16 or so); an exponent where the largest value is
            # at 448 2^k to within 2^-21
            scale = torch.exp2(exp.double() - 127).repeat_interleave(128)[:n]
            off = (code * scale - x.abs().copysign(x)).abs()
            stepsize = torch.maximum(code.abs(), torch.tensor(2.0 ** -6, device=DEV)) / 8 * scale
            assert (off <= 1.0001 * stepsize).all(), f"{name}: further than a step"
            assert (exp != re).sum().item() <= 1 + exp.numel() * 1e-4, f"{name}: exponents"
            same = (exp == re).repeat_interleave(128)[:n]
            assert ((code != rv) & same).sum().item() <= 2 + n * 2e-4, f"{name}: codes"


def test_8_bit_averages_follow_their_gradients():
    """Constant gradients, for which a step is far below half a code: m and v reach what 32-bit states reach, on average
    within the spread of the rounding (a code is off by at most 1/8 at a time, averaged over 1000 values and 1 / (1 -
    beta) steps)."""
    n, beta1, beta2 = 128 * 64, 0.9, 0.99
    p = torch.zeros(n, device=DEV)
    m, v = moe.Fp8Moment.zeros(p), moe.Fp8Moment.zeros(p)
    plan = moe.AdamWTensors([p], [m], [v])
    sizes = torch.logspace(-3, 0, 8, device=DEV)
    g = sizes.repeat(n // 8)
    for t in range(1, 801):
        moe.moe_adamw(plan, [g], step=t, lr=0.0, beta1=beta1, beta2=beta2)
    for k in range(8):
        mean = m.values()[k::8].double().mean().item()
        square = v.values()[k::8].double().square().mean().item()
        assert abs(mean / sizes[k].item() - 1) < 0.02, (k, mean)
        assert abs(square / sizes[k].item() ** 2 - 1) < 0.04, (k, square)


def test_8_bit_edges():
    """Zeros stay zeros; a tiny second moment keeps a code; a value that is not finite takes its block alone; rows past
    the end are left alone."""
    n = 128 * 3 + 5
    p = torch.ones(n, device=DEV)
    m, v = moe.Fp8Moment.zeros(p), moe.Fp8Moment.zeros(p)
    g = torch.zeros(n, device=DEV)
    plan = moe.AdamWTensors([p], [m], [v])
    moe.moe_adamw(plan, [g], step=1, lr=0.5, weight_decay=0.0)
    assert (p == 1).all() and not m.values().any() and not v.values().any()
    g[0], g[1] = 1.0, 1e-9                         # in one block, far below the smallest code of it
    moe.moe_adamw(plan, [g], step=1, lr=0.5, weight_decay=0.0)
    assert v.codes.view(torch.uint8)[1] == 1 and torch.isfinite(p).all()
    assert abs(p[0].item() - 0.5) < 1e-5           # the first step's size is lr
    g[200] = float("inf")
    g[380] = float("nan")
    moe.moe_adamw(plan, [g], step=2, lr=0.5, weight_decay=0.0)
    bad = torch.zeros(n, dtype=torch.bool, device=DEV)
    bad[128:256] = bad[256:384] = True
    for t in (m, v):
        assert torch.equal(torch.isnan(t.values()), bad) and t.exps[1] == t.exps[2] == 255
    only = torch.zeros(n, dtype=torch.bool, device=DEV)
    only[200] = only[380] = True
    assert torch.equal(~torch.isfinite(p), only)


@pytest.mark.parametrize("fp8", [False, True])
def test_extremes(fp8):
    """Gradients from the smallest to the largest: no state or parameter that should be finite is not."""
    g = torch.logspace(-44, 18, 128 * 4, device=DEV)
    p = torch.zeros_like(g)
    m, v = (moe.Fp8Moment.zeros(p), moe.Fp8Moment.zeros(p)) if fp8 else (torch.zeros_like(p), torch.zeros_like(p))
    plan = moe.AdamWTensors([p], [m], [v])
    for t in (1, 2):
        moe.moe_adamw(plan, [g], step=t, lr=1e-3, eps=1e-8, weight_decay=0.0)
    assert torch.isfinite(p).all() and (p <= 0).all()
    big = g > 1e-4
    tol = 1e-3 if not fp8 else 1.0                  # rounded states: see above for theirs
    assert ((p[big] / -2e-3 - 1).abs() < tol).all()


# ----------------------------------------- streams, graphs, repetition, use

def _two(g, fp8):
    ts = fp8_list(g, [5000, 300], F32, BF, BF)
    plan = moe.AdamWTensors(*([t[k] for t in ts] for k in (("p", "m8", "v8") if fp8 else ("p", "m", "v"))),
                            copies=[t["c"] for t in ts])
    return ts, plan


def _state(ts, fp8):
    out = [t[k] for t in ts for k in ("p", "c")]
    out += [x for t in ts for k in ("m8", "v8") for x in t[k]] if fp8 else [t[k] for t in ts for k in ("m", "v")]
    return [x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in out]


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_and_replayed(fp8):
    """Step and learning rate on the device: every replay is the eager step of that number, in turn with eager ones."""
    ts, plan = _two(gen(3), fp8)
    tw, twin = _two(gen(3), fp8)
    step, lr = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, device=DEV)
    grads, tgrads = [t["g"] for t in ts], [t["g"] for t in tw]
    scale = torch.ones(1, device=DEV)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        moe.moe_adamw(plan, grads, step=step, lr=lr, grad_scale=scale)
    assert torch.equal(ts[0]["p"], tw[0]["p"])
    for k in range(1, 5):
        g = gen(50 + k)
        for a, b in zip(grads, tgrads):
            a.copy_(torch.randn(a.shape, generator=g, device=DEV))
            b.copy_(a)
        step.fill_(k)
        lr.fill_(1e-3 * k)
        scale.fill_(0.5 ** k)
        if k == 3:
            moe.moe_adamw(plan, grads, step=step, lr=lr, grad_scale=scale)
        else:
            gr.replay()
        moe.moe_adamw(twin, tgrads, step=k, lr=float(lr.item()), grad_scale=scale)
        torch.cuda.synchronize()
        for a, b in zip(_state(ts, fp8), _state(tw, fp8)):
            # 1 - beta^k by squaring against the host's power: the last bit of a factor
            if a.dtype == torch.uint8:
                assert torch.equal(a, b)
            else:
                assert ((a.double() - b.double()).abs() <= 2 * u(a.dtype) * b.double().abs() + 8 * E * 1e-2).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_repeatable_and_on_another_stream(fp8):
    side = torch.cuda.Stream()
    got = []
    for stream in (None, side, side.cuda_stream):
        ts, plan = _two(gen(5), fp8)
        torch.cuda.synchronize()
        for k in (1, 2):
            moe.moe_adamw(plan, [t["g"] for t in ts], step=k, lr=1e-3, stream=stream)
        torch.cuda.synchronize()
        got.append([t.clone() for t in _state(ts, fp8)])
    for a, b, c in zip(*got):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_a_tensor_split_or_whole_is_the_same():
    """32-bit states: one tensor, or its parts in a list of more than one launch."""
    g = gen(6)
    n = 128 * 130
    t, = make(g, [n], F32, F32, None)
    parts = {k: t[k].clone() for k in ("p", "m", "v")}
    moe.moe_adamw(moe.AdamWTensors([t["p"]], [t["m"]], [t["v"]]), [t["g"]], step=2, lr=1e-2)
    cut = {k: list(v.split(128)) for k, v in parts.items()}
    moe.moe_adamw(moe.AdamWTensors(cut["p"], cut["m"], cut["v"]), list(t["g"].split(128)), step=2, lr=1e-2)
    for k in parts:
        assert torch.equal(parts[k], t[k])


@pytest.mark.parametrize("fp8", [False, True])
def test_more_values_than_a_grid_of_one_turn_blocks(fp8):
    """1.1e9 values: a block takes two turns.  The last values and some between are those of a short list of the same."""
    n, k = (1 << 30) + 50_000_001, 4096
    p, g = torch.zeros(n, dtype=BF, device=DEV), torch.zeros(n, dtype=BF, device=DEV)
    m, v = (moe.Fp8Moment.zeros(p), moe.Fp8Moment.zeros(p)) if fp8 else (torch.zeros(n, device=DEV), torch.zeros(n, device=DEV))
    rng = gen(3)
    spots = [0, 1 << 20, (1 << 30) - 2048, (n - k) // 128 * 128]
    values = [torch.randn(k, generator=rng, device=DEV).to(BF) for _ in spots]
    for a, x in zip(spots, values):
        g[a:a + k] = x
    moe.moe_adamw(moe.AdamWTensors([p], [m], [v]), [g], step=1, lr=1e-2, weight_decay=0.0)
    for a, x in zip(spots, values):
        want, _, _, ep, _, _ = ref_step(torch.zeros_like(x), x, torch.zeros_like(x), torch.zeros_like(x), 1, 1e-2, 0.9, 0.999, 1e-8, 0.0)
        check_param(p[a:a + k], want, ep, f"at {a}")
    assert not p[spots[0] + k:spots[1]].any() and not p[spots[2] + k:spots[3]].any()


def test_refusals():
    n = 256
    f = lambda dt=F32, k=n: torch.zeros(k, dtype=dt, device=DEV)  # noqa: E731
    p, m, v = f(), f(), f()
    new = moe.AdamWTensors
    plan = new([p], [m], [v])
    for bad, err in [(lambda: new([p], [m], [m]), ValueError), (lambda: new([p, p], [m, f()], [v, f()]), ValueError),
                     (lambda: new([p], [m], []), ValueError), (lambda: new([p], [f(BF)], [v]), TypeError),
                     (lambda: new([p], [f(k=255)], [v]), ValueError), (lambda: new([p.cpu()], [m], [v]), ValueError),
                     (lambda: new([p.view(16, 16).t()], [m], [v]), ValueError),
                     (lambda: new([p], [m], [v], copies=[f()]), TypeError), (lambda: new([p], [m], [v], copies=[]), ValueError),
                     (lambda: new([p], [moe.Fp8Moment.zeros(p)], [v]), TypeError),
                     (lambda: new([p], [m], [v], copies=[p.view(BF)[:n]]), ValueError),
                     (lambda: moe.moe_adamw(plan, [], 1, 0.1), ValueError), (lambda: moe.moe_adamw(plan, [f(k=3)], 1, 0.1), ValueError),
                     (lambda: moe.moe_adamw(plan, [f(torch.float64)], 1, 0.1), TypeError),
                     (lambda: moe.moe_adamw(plan, [f().cpu()], 1, 0.1), ValueError),
                     (lambda: moe.moe_adamw(plan, [f()], 0, 0.1), moe.MoeError),
                     (lambda: moe.moe_adamw(plan, [p], 1, 0.1), moe.MoeError),
                     (lambda: moe.moe_adamw(plan, [f()], 1, float("nan")), moe.MoeError),
                     (lambda: moe.moe_adamw(plan, [f()], 1, 0.1, beta1=1.0), moe.MoeError),
                     (lambda: moe.moe_adamw(plan, [f()], torch.ones(1, device=DEV), 0.1), ValueError),
                     (lambda: moe.moe_adamw(plan, [f()], 1, 0.1, grad_scale=0.5), TypeError)]:
        with pytest.raises(err):
            bad()
    p.data = f()
    with pytest.raises(ValueError, match="moved"):
        moe.moe_adamw(plan, [f()], 1, 0.1)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", ["p", "m", "v", "c"])
@pytest.mark.parametrize("how", ["data", "freed"])
def test_memory_that_is_no_longer_the_lists(how, what, fp8):
    """A parameter, state or copy that was given other memory, or whose memory was freed: refused before anything is written."""
    for part in range(2 if fp8 and what in "mv" else 1):     # codes, exponents
        ts, plan = _two(gen(3), fp8)
        x = ts[1][what + "8"][part] if fp8 and what in "mv" else ts[1][what]
        before, size = [y.clone() for y in _state(ts, fp8)], x.untyped_storage().nbytes()
        old, saved = x.data, x.clone()
        if how == "data":
            x.data = saved
        else:
            x.untyped_storage().resize_(0)
        with pytest.raises(ValueError, match="moved"):
            moe.moe_adamw(plan, [t["g"] for t in ts], step=1, lr=0.1)
        if how == "data":
            x.data = old
        else:
            x.untyped_storage().resize_(size)
            x.copy_(saved)
        for a, b in zip(_state(ts, fp8), before):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        if how == "data":                           # its own memory again
            moe.moe_adamw(plan, [t["g"] for t in ts], step=1, lr=0.1)
            assert not torch.equal(ts[1]["p"], before[2])


def test_shapes():
    """States, copies and gradients have their parameter's shape, or are flat (or the parameter is): never another order."""
    f = lambda *s, dt=F32: torch.randn(s, generator=gen(sum(s)), device=DEV).to(dt)  # noqa: E731
    new = moe.AdamWTensors
    for kw in (dict(m=f(24, 16)), dict(v=f(24, 16)), dict(c=f(24, 16, dt=BF)), dict(m=f(2, 8, 24))):
        a = {**dict(p=f(16, 24), m=f(16, 24), v=f(16, 24), c=f(16, 24, dt=BF)), **kw}
        with pytest.raises(ValueError, match="shape"):
            new([a["p"]], [a["m"]], [a["v"]], copies=[a["c"]])
    p, m, v, p2 = f(16, 24), torch.zeros(16, 24, device=DEV), torch.zeros(16 * 24, device=DEV), f(16 * 24)
    plan = new([p, p2], [m, torch.zeros_like(p2)], [v, torch.zeros_like(p2)])
    for bad in ([f(24, 16), f(16 * 24)], [f(4, 4, 24), f(16 * 24)], [f(24, 16), None]):
        with pytest.raises(ValueError, match="shape"):
            moe.moe_adamw(plan, bad, 1, 0.1)
    assert not m.any() and not v.any()
    for grads in ([f(16, 24), f(16 * 24)], [f(16 * 24), f(16, 24)], [f(16, 1, 24), f(1, 16 * 24)], [f(16, 24), None]):
        want = ref_step(p, grads[0].view(16, 24), m, v.view(16, 24), 1, **HYPER)
        moe.moe_adamw(plan, grads, 1, **HYPER)
        check_param(p, want[0], want[3], "param")
    with pytest.raises(ValueError, match="shape"):  # also after others were taken
        moe.moe_adamw(plan, [f(24, 16), f(16 * 24)], 1, 0.1)


@pytest.mark.parametrize("eps", [1e-8, 1e-3])
def test_8_bit_extremes_step_by_step(eps):
    """Gradients from the smallest to the largest: each step against the formula, from the states that the codes hold.  Numbers
    below 2^-126 round by 2^-150 at most: in m's terms and sum and m's product (four), over eps at least, and p's own; v's
    three are 2^-74 of its root, over eps."""
    g = torch.logspace(-44, 18, 128 * 4, device=DEV)
    p = torch.zeros_like(g)
    m, v = moe.Fp8Moment.zeros(p), moe.Fp8Moment.zeros(p)
    plan = moe.AdamWTensors([p], [m], [v])
    for t in (1, 2, 3):
        r = v.values().double()
        want, m1, _, ep, _, _ = ref_step(p, g, m.values(), r * r, t, 1e-3, 0.9, 0.999, eps, 0.0)
        moe.moe_adamw(plan, [g], step=t, lr=1e-3, eps=eps, weight_decay=0.0)
        size = 1e-3 / (1 - 0.9 ** t) / eps
        low = size * 4 * 2.0 ** -150 + size * m1.abs() * 2.0 * 2.0 ** -74 / math.sqrt(1 - 0.999 ** t) / eps + 4 * 2.0 ** -150
        check_param(p, want, ep + low, f"step {t}")
        assert (p <= 0).all()
