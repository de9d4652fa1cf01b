"""Products with 4-bit weights, dense, gated and by expert, against the
formulas in 64 bits with the values that the codes stand for.  Tolerances count
roundings as in test_gpu_operators.py: the weights are exact in 16 bits, so
only the fp32 sums, the epilogue and the store round."""
import pytest
import torch

import expert_ffn_dispatch_amd as moe
import test_gpu_operators as T
from test_gpu_gated import check_forward
from test_gpu_operators import ACC, ACTS, BF, DEV, F32, FUN, HF, act_ref, check, gen, offsets_of, randn, strided, tiny, u

pytestmark = pytest.mark.gpu

MAGNITUDES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def values(w):
    """By the definition, in 64 bits."""
    mag = MAGNITUDES.to(w.codes.device)
    nib = torch.stack([w.codes & 15, w.codes >> 4], -1).long().flatten(-2)
    v = mag[nib & 7] * torch.where(nib >= 8, -1.0, 1.0).double()
    return v * torch.exp2(w.exps.double() - 127).repeat_interleave(32, -1)


def weights(g, *shape):
    """Random codes of every kind, exponents around those of shape[-1] normal weights."""
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device=DEV, dtype=torch.uint8)
    e = 127 - 2 - round(torch.tensor(float(shape[-1])).log2().item() / 2)
    exps = torch.randint(max(e - 2, 104), e + 3, (*shape[:-1], shape[-1] // 32), generator=g, device=DEV, dtype=torch.uint8)
    return moe.Fp4Weights(codes, exps)


def product_error(x, W, extra=0):
    return 1.01 * (x.shape[1] + 2) * ACC * (x.double().abs() @ W.abs().T + extra)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_every_code_and_exponent(dtype):
    """The identity times every code at every exponent that the type takes: the values themselves."""
    lo, hi = (1, 252) if dtype == BF else (104, 140)
    exps = torch.arange(lo, hi + 1, dtype=torch.uint8, device=DEV)[:, None]
    codes = (torch.arange(16, device=DEV, dtype=torch.uint8).repeat(2)[0::2] | torch.arange(16, device=DEV, dtype=torch.uint8).repeat(2)[1::2] << 4)
    w = moe.Fp4Weights(codes.expand(len(exps), 16).contiguous(), exps)
    for rows in (32, 96):                           # the codes as they are, and widened
        x = torch.eye(32, dtype=dtype, device=DEV).repeat(rows // 32, 1)
        y = moe.moe_linear_fp4(x, w)
        want = values(w).T.repeat(rows // 32, 1)
        ok = want.abs() >= torch.finfo(dtype).tiny if dtype == BF else torch.ones_like(want, dtype=torch.bool)
        assert torch.equal(y.double()[ok], want[ok])
        # below bf16's normal range a matrix instruction may take zeros
        assert ((y.double() - want).abs()[~ok] <= torch.finfo(dtype).tiny).all()
    assert torch.equal(w.values()[:, :].double(), values(w))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_quantise(dtype):
    g = gen(1)
    w = randn(g, 7, 33, 96, dtype=dtype, scale=0.05)
    w[0, 0] = 0
    w[0, 1, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4, device=DEV).to(dtype)   # ties
    w[0, 2, :32] *= 2.0 ** (-10 if dtype == HF else -100)
    w[0, 3, 5] = 6e4 if dtype == HF else 3e38
    w[0, 4, 5], w[0, 4, 6] = 7.0, 6.9
    w[0, 5, 5] = 7.03125
    q = moe.moe_quantize_fp4(w)
    assert q.codes.shape == (7, 33, 48) and q.exps.shape == (7, 33, 3)
    lo, hi = (1, 252) if dtype == BF else (104, 140)
    X = w.double().view(7, 33, 3, 32)
    top = X.abs().amax(-1)
    e = torch.ceil(torch.log2(top.clamp_min(1e-300) / 7))
    e = torch.where(top <= 7 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top > 7 * torch.exp2(e), e + 1, e).clamp(lo - 127, hi - 127)
    assert torch.equal(q.exps.double() - 127, e)
    f = (X / torch.exp2(e)[..., None]).clamp(-6, 6)
    got = (values(q).view(7, 33, 3, 32) / torch.exp2(e)[..., None])
    d = (f.abs()[..., None] - MAGNITUDES.to(DEV)).abs()
    assert torch.equal((got.abs() - f.abs()).abs(), d.amin(-1)), "a nearer code"
    tie = (d == d.amin(-1, keepdim=True)).sum(-1) == 2
    code = (got.abs()[..., None] == MAGNITUDES.to(DEV)).long().argmax(-1)
    assert tie.any() and (code[tie] % 2 == 0).all()
    assert (torch.signbit(got) == torch.signbit(f))[got != 0].all()


# rows, in, out: one token, few rows, odd outputs, partial chunks of the contraction, more rows than a tile
SHAPES = [(1, 32, 1), (1, 64, 64), (1, 2048, 520), (3, 96, 5), (2, 6144, 48), (16, 160, 40), (17, 512, 256), (31, 1056, 130),
          (33, 256, 6200), (48, 128, 77), (64, 992, 136), (65, 256, 264), (130, 288, 392), (300, 4096, 64), (257, 768, 512),
          (700, 1024, 1003), (90, 2048, 768), (130, 160, 4096), (257, 96, 4096), (600, 64, 8200),
          (7000, 1024, 2050), (4000, 2048, 2048), (257, 2080, 100), (129, 4096, 500), (120, 2048, 1000)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,n_in,n_out", SHAPES)
def test_linear(rows, n_in, n_out, act):
    g = gen(rows + n_in + n_out)
    dt = HF if (rows + n_out) % 2 else BF
    x, w = randn(g, rows, n_in, dtype=dt), weights(g, n_out, n_in)
    W = values(w)
    bias = randn(g, n_out, dtype=F32 if act in ("relu", "silu") else dt)
    res = randn(g, rows, n_out, dtype=dt) if act != "gelu" else None
    y = moe.moe_linear_fp4(x, w, bias, res, act=act)
    z = x.double() @ W.T + bias.double()
    ez = product_error(x, W, bias.double().abs())
    ref = act_ref(z, act)
    r = 0 if res is None else res.double()
    err = 1.2 * ez + FUN * ref.abs() + ACC * z.abs()        # slopes of the activations are at most 1.13
    check(y, ref + r, u(dt) * (ref + r).abs() + 1.01 * err + 2 * ACC * (ref + r).abs() + tiny(dt), "y")
    y = moe.moe_linear_fp4(x, w, act=act)
    z = x.double() @ W.T
    ref = act_ref(z, act)
    check(y, ref, u(dt) * ref.abs() + 1.01 * (1.2 * ez + FUN * ref.abs() + ACC * z.abs()) + tiny(dt), "y, plain")


@pytest.mark.parametrize("act", ["silu", "none", "gelu"])
@pytest.mark.parametrize("rows,n_in,width", SHAPES)
def test_gated_linear(rows, n_in, width, act):
    g = gen(rows + n_in + width)
    dt = BF if (rows + width) % 2 else HF
    x, wg, wu = randn(g, rows, n_in, dtype=dt), weights(g, width, n_in), weights(g, width, n_in)
    h = moe.moe_gated_linear_fp4(x, wg, wu, act=act)
    check_forward(x, values(wg), values(wu), act, h, None, None)


GROUPS = [([5], 64, 64), ([1], 32, 1), ([0], 64, 24), ([0, 0, 3, 0], 96, 136), ([1] * 7, 128, 256), ([130, 0, 1, 33, 257], 192, 264),
          ([31, 32, 33, 0, 64, 65, 127, 128, 129], 256, 128), ([3, 9, 0, 2], 64, 131), ([700, 0, 2, 600], 512, 320),
          ([2] * 256, 64, 72), ([0] * 100 + [50] + [0] * 59, 128, 128), ([20] * 16, 1024, 768), ([17, 0, 40, 3, 11], 2048, 200),
          ([60, 90, 0, 10], 288, 96), ([9, 0, 1, 4, 5] + [0] * 9 + [3, 2], 2080, 200), ([1, 0, 3, 0], 4096, 776), ([6000, 0, 4100, 1], 1024, 2056)]


@pytest.mark.parametrize("n_in,n_out", [(2080, 6160), (96, 6144), (4096, 200), (32, 24)])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5])
def test_few_rows(rows, n_in, n_out):
    """Tiles of four rows and of sixteen; the row behind the last stays as it was."""
    g = gen(rows * n_in + n_out)
    x, w, w2 = randn(g, rows, n_in), weights(g, n_out, n_in), weights(g, n_out, n_in)
    y, h = (torch.full((rows + 1, n_out), 7.0, dtype=BF, device=DEV) for _ in range(2))
    moe.moe_linear_fp4(x, w, y=y[:rows])
    moe.moe_gated_linear_fp4(x, w, w2, h=h[:rows])
    ref = x.double() @ values(w).T
    check(y[:rows], ref, u(BF) * ref.abs() + product_error(x, values(w)) + tiny(BF), "y")
    check_forward(x, values(w), values(w2), "silu", h[:rows], None, None)
    assert (y[rows] == 7).all() and (h[rows] == 7).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,n_in,n_out", GROUPS, ids=[f"{len(c)}x{sum(c)}-{i}-{o}" for c, i, o in GROUPS])
def test_grouped(counts, n_in, n_out, dtype):
    g = gen(sum(counts) + n_in)
    front, back = 3, 5                              # rows outside every group
    E, rows = len(counts), sum(counts) + front + back
    off = offsets_of(counts, front)
    x = randn(g, rows, n_in, dtype=dtype)
    x[:front] = float("nan")
    x[rows - back:] = float("nan")
    w, w2 = weights(g, E, n_out, n_in), weights(g, E, n_out, n_in)
    y, h = (torch.full((rows, n_out), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    moe.moe_grouped_matmul_fp4(x, off, w, y=y)
    moe.moe_grouped_gated_fp4(x, off, w, w2, h=h)
    for t in (y, h):
        assert (t[:front] == 7).all() and (t[rows - back:] == 7).all(), "rows outside the groups were written"
    b = front
    for e, c in enumerate(counts):
        if c:
            X, W = x[b:b + c], values(moe.Fp4Weights(w.codes[e], w.exps[e]))
            ref = X.double() @ W.T
            check(y[b:b + c], ref, u(dtype) * ref.abs() + product_error(X, W) + tiny(dtype), f"y {e}")
            check_forward(X, W, values(moe.Fp4Weights(w2.codes[e], w2.exps[e])), "silu", h[b:b + c], None, None, f"{e}")
        b += c


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (8, 1), (5, 3)])
@pytest.mark.parametrize("rows", [1, 10, 30, 60, 150])
def test_strides(rows, pad, shift):
    """Rows at any pitch and alignment, inputs and outputs."""
    g = gen(rows + pad)
    n_in, n_out = 288, 72
    x, r = randn(g, rows, n_in), randn(g, rows, n_out)
    w, w2 = weights(g, n_out, n_in), weights(g, n_out, n_in)
    S = lambda t: strided(t, pad, shift)  # noqa: E731
    y, h = S(torch.zeros_like(r)), S(torch.zeros_like(r))
    moe.moe_linear_fp4(S(x), w, None, S(r), y=y)
    ref = x.double() @ values(w).T + r.double()
    check(y, ref, (u(BF) + 2 * ACC) * ref.abs() + product_error(x, values(w)) + tiny(BF), "y")
    moe.moe_gated_linear_fp4(S(x), w, w2, h=h)
    check_forward(x, values(w), values(w2), "silu", h, None, None)
    off = offsets_of([rows])
    w3 = moe.Fp4Weights(w.codes[None], w.exps[None])
    z = moe.moe_grouped_matmul_fp4(S(x), off, w3, y=S(torch.zeros_like(r)))
    check(z, ref - r.double(), u(BF) * (ref - r.double()).abs() + product_error(x, values(w)) + tiny(BF), "grouped")
    for t in (y, h, z):
        pads = t._base.reshape(-1)[shift:].view(rows, n_out + pad)[:, n_out:]
        assert torch.isnan(pads).all(), "the space between rows was written"


def test_offsets_are_clamped_empty_and_not_a_number():
    g = gen(8)
    x, w, w2 = randn(g, 40, 64), weights(g, 3, 72, 64), weights(g, 3, 72, 64)
    bad = torch.tensor([-5, 10, 7, 1000], dtype=torch.int32, device=DEV)
    for f in (lambda t, o: moe.moe_grouped_matmul_fp4(t, o, w), lambda t, o: moe.moe_grouped_gated_fp4(t, o, w, w2)):
        y = f(x, bad)
        assert torch.equal(y[:7], f(x[:10], offsets_of([10, 0, 0]))[:7])
        assert torch.equal(y[10:], f(x[7:], offsets_of([0, 0, 33]))[3:])
        e = torch.empty(0, 64, dtype=BF, device=DEV)
        assert f(e, torch.zeros(4, dtype=torch.int32, device=DEV)).shape == (0, 72)
    assert moe.moe_linear_fp4(e, moe.Fp4Weights(w.codes[0], w.exps[0])).shape == (0, 72)
    w0 = moe.Fp4Weights(w.codes[0], w.exps[0])
    for rows in (20, 40, 100):
        x = randn(g, rows, 64)
        want = moe.moe_linear_fp4(x, w0)
        x[3, 1], x[7, 5] = float("nan"), float("inf")
        y = moe.moe_linear_fp4(x, w0)
        ok = torch.ones(rows, dtype=torch.bool, device=DEV)
        ok[3] = ok[7] = False
        assert torch.equal(y[ok], want[ok]) and torch.isnan(y[3]).all()
        # infinity times a weight of any sign, or of zero
        col = values(w0)[:, 5]
        assert torch.equal(torch.isnan(y[7]), col == 0) and torch.equal(torch.sign(y[7][col != 0]).double(), torch.sign(col[col != 0]))


def test_rows_past_32_bits():
    """Rows of x behind 4 GiB of a strided matrix, by expert, and the same rows packed."""
    g = gen(10)
    big = torch.zeros(2200, 1 << 20, dtype=BF, device=DEV)
    x, off = big[:, :96], offsets_of([275] * 8)
    x.copy_(randn(g, 2200, 96))
    w, w2 = weights(g, 8, 40, 96), weights(g, 8, 40, 96)
    packed = x.contiguous()
    assert torch.equal(moe.moe_grouped_matmul_fp4(x, off, w), moe.moe_grouped_matmul_fp4(packed, off, w))
    assert torch.equal(moe.moe_grouped_gated_fp4(x, off, w, w2), moe.moe_grouped_gated_fp4(packed, off, w, w2))
    one = moe.Fp4Weights(w.codes[0], w.exps[0])
    assert torch.equal(moe.moe_linear_fp4(x, one), moe.moe_linear_fp4(packed, one))


def _calls(g):
    x, off = randn(g, 150, 256), offsets_of([40, 0, 60, 50])
    one, few, foff = x[:1].contiguous(), x[:8].contiguous(), offsets_of([3, 0, 1, 4])
    w, w2, we, we2 = weights(g, 192, 256), weights(g, 192, 256), weights(g, 4, 192, 256), weights(g, 4, 192, 256)

    def calls(stream=None):
        out = []
        for t, o in ((x, off), (few, foff)):
            out += [moe.moe_linear_fp4(t, w, act="gelu", stream=stream), moe.moe_gated_linear_fp4(t, w, w2, stream=stream),
                    moe.moe_grouped_matmul_fp4(t, o, we, stream=stream), moe.moe_grouped_gated_fp4(t, o, we, we2, stream=stream)]
        return out + [moe.moe_linear_fp4(one, w, stream=stream), *moe.moe_quantize_fp4(x, stream=stream)]
    return calls, (x, one, few)


def test_repeatable_and_on_another_stream():
    calls, _ = _calls(gen(4))
    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        got = calls(stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_captured_and_replayed():
    """Two graphs of the same calls, replayed in turn between eager calls, on inputs that change in place."""
    calls, inputs = _calls(gen(6))
    calls()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = calls()
        graphs.append((gr, out))
    for k in range(3):
        g = gen(100 + k)
        for t in inputs:
            t.copy_(randn(g, *t.shape, scale=0.5))
        want = [t.clone() for t in calls()]
        for gr, out in graphs:
            gr.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b), f"replay {k}"


def test_experts_served_in_4_bits():
    """Route -> permute -> gated projections and down projection in 4 bits -> combine, against the layer with the same
    weights in 16 bits, which hold the codes' values exactly: the two differ in the order of fp32 sums, by a rounding
    step of h (2^-8) in the products of the down projection and one of y."""
    g = gen(33)
    N, M, E, k, H = 40, 256, 8, 2, 128
    d = moe.dims(N, M, E, k, H)
    x = randn(g, N, M)
    wr = randn(g, M, E, scale=M ** -0.5)
    wg, wu, wd = (moe.moe_quantize_fp4(randn(g, E, o, i, scale=i ** -0.5)) for o, i in ((H, M), (H, M), (M, H)))
    ids, wts = moe.moe_route(d, x, wr)
    perm = moe.moe_permute(d, ids, x=x, want_x_sorted=True)
    off = perm["expert_offsets"]
    h = moe.moe_grouped_gated_fp4(perm["x_sorted"], off, wg, wu)
    y = moe.moe_grouped_matmul_fp4(h, off, wd)
    out = moe.moe_combine(d, y, perm["assign_to_sorted"], wts)
    full = moe.moe_layer(d, x, *(w.values().to(BF) for w in (wg, wu, wd)), w_router=wr)
    assert ((out.float() - full.float()).norm() / full.float().norm()).item() < 2 * 2.0 ** -8


def test_weights_past_32_bits():
    """Experts behind 4 GiB of codes."""
    g = gen(9)
    E, n_out, n_in = 220, 8192, 5120                # 4.6 GB of codes
    codes = torch.zeros(E, n_out, n_in // 2, dtype=torch.uint8, device=DEV)
    exps = torch.full((E, n_out, n_in // 32), 120, dtype=torch.uint8, device=DEV)
    last = weights(g, n_out, n_in)
    codes[E - 1], exps[E - 1] = last.codes, last.exps
    x, off = randn(g, 20, n_in), offsets_of([0] * (E - 1) + [20])
    w = moe.Fp4Weights(codes, exps)
    W = values(last)
    ref = x.double() @ W.T
    check(moe.moe_grouped_matmul_fp4(x, off, w), ref, u(BF) * ref.abs() + product_error(x, W) + tiny(BF), "y")
    h = moe.moe_grouped_gated_fp4(x, off, w, w)
    check_forward(x, W, W, "silu", h, None, None)
