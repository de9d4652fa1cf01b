"""Products with 4-bit weights where these are widened into the workspace first:
every code at every exponent, both types, rows at any pitch and alignment, by
expert, captured and on another stream.  The sizes are the smallest that are
widened; tests/test_fp4_plans_cpu.py holds them to that.  Tolerances as in
test_gpu_fp4.py."""
import pytest
import torch

import expert_ffn_dispatch_amd as moe
from test_gpu_fp4 import product_error, values, weights
from test_gpu_gated import check_forward
from test_gpu_operators import ACC, BF, DEV, F32, FUN, HF, act_ref, check, gen, offsets_of, randn, strided, tiny, u

pytestmark = pytest.mark.gpu

# rows, in, out, and the pitch of x beyond its width: whole 16-byte pieces, and not
DENSE = [(3800, 2048, 2048, 0), (3800, 2048, 2048, 8), (1800, 2048, 2048, 3), (1500, 2080, 2500, 1)]
GATED = [(2400, 2048, 2048, 0), (1100, 2048, 2048, 5), (1500, 1056, 2501, 7)]
# rows of each expert, in, out, pitch: the mean decides, some are empty or short
GROUPED = [([5000, 0, 7000, 1], 1024, 2056, 0), ([3000, 0, 2600, 1], 1024, 2056, 3)]
GROUPED_GATED = [([5000, 0, 4600, 1], 1024, 2056, 0), ([2000, 0, 2400, 1], 1024, 2056, 1)]
EVERY = (4096, 2048, 2048)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_every_code_and_exponent(dtype):
    """Two identities times every code at every exponent that the type takes: the values themselves."""
    rows, n_in, n_out = EVERY
    lo, hi = (1, 252) if dtype == BF else (104, 140)
    exps = (torch.arange(n_out * n_in // 32, device=DEV) % (hi - lo + 1) + lo).to(torch.uint8).view(n_out, n_in // 32)
    pair = torch.arange(16, device=DEV, dtype=torch.uint8).repeat(2)
    codes = (pair[0::2] | pair[1::2] << 4).repeat(n_in // 32).expand(n_out, -1).contiguous()
    w = moe.Fp4Weights(codes, exps)
    y = moe.moe_linear_fp4(torch.eye(n_in, dtype=dtype, device=DEV).repeat(rows // n_in, 1), w)
    want = values(w).T.repeat(rows // n_in, 1)
    ok = want.abs() >= torch.finfo(dtype).tiny if dtype == BF else torch.ones_like(want, dtype=torch.bool)
    assert torch.equal(y.double()[ok], want[ok])
    # below bf16's normal range a matrix instruction may take zeros
    assert ((y.double() - want).abs()[~ok] <= torch.finfo(dtype).tiny).all()


@pytest.mark.parametrize("dtype,act", [(BF, "gelu"), (HF, "silu"), (HF, "none")])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("rows,n_in,n_out,pad", DENSE)
def test_linear(rows, n_in, n_out, pad, shift, dtype, act):
    g = gen(rows + pad)
    x, w, res = randn(g, rows, n_in, dtype=dtype), weights(g, n_out, n_in), randn(g, rows, n_out, dtype=dtype)
    bias = randn(g, n_out, dtype=F32 if act == "silu" else dtype)
    W = values(w)
    y = strided(torch.zeros_like(res), pad, shift)
    moe.moe_linear_fp4(strided(x, pad, shift), w, bias, strided(res, pad, shift), act=act, y=y)
    z = x.double() @ W.T + bias.double()
    ez = product_error(x, W, bias.double().abs())
    ref = act_ref(z, act)
    err = 1.2 * ez + FUN * ref.abs() + ACC * z.abs()        # slopes of the activations are at most 1.13
    ref = ref + res.double()
    check(y, ref, u(dtype) * ref.abs() + 1.01 * err + 2 * ACC * ref.abs() + tiny(dtype), "y")
    pads = y._base.reshape(-1)[shift:].view(rows, n_out + pad)[:, n_out:]
    assert torch.isnan(pads).all(), "the space between rows was written"


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("rows,n_in,width,pad", GATED)
def test_gated(rows, n_in, width, pad, shift, dtype):
    g = gen(rows + pad)
    x, wg, wu = randn(g, rows, n_in, dtype=dtype), weights(g, width, n_in), weights(g, width, n_in)
    h = strided(torch.zeros(rows, width, dtype=dtype, device=DEV), pad, shift)
    moe.moe_gated_linear_fp4(strided(x, pad, shift), wg, wu, h=h)
    check_forward(x, values(wg), values(wu), "silu", h, None, None)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("gated,counts,n_in,n_out,pad", [(False, *c) for c in GROUPED] + [(True, *c) for c in GROUPED_GATED],
                         ids=lambda v: f"{len(v)}x{sum(v)}" if isinstance(v, list) else None)
def test_grouped(gated, counts, n_in, n_out, pad, shift, dtype):
    g = gen(sum(counts) + pad)
    front, back = 3, 5                              # rows outside every group
    rows = sum(counts) + front + back
    off = offsets_of(counts, front)
    x = randn(g, rows, n_in, dtype=dtype)
    x[:front] = x[rows - back:] = float("nan")
    w, w2 = weights(g, len(counts), n_out, n_in), weights(g, len(counts), n_out, n_in)
    y = torch.full((rows, n_out), 7.0, dtype=dtype, device=DEV)
    if gated:
        moe.moe_grouped_gated_fp4(strided(x, pad, shift), off, w, w2, h=y)
    else:
        moe.moe_grouped_matmul_fp4(strided(x, pad, shift), off, w, y=y)
    assert (y[:front] == 7).all() and (y[rows - back:] == 7).all(), "rows outside the groups were written"
    b = front
    for e, c in enumerate(counts):
        if c:
            X, W = x[b:b + c], values(moe.Fp4Weights(w.codes[e], w.exps[e]))
            if gated:
                check_forward(X, W, values(moe.Fp4Weights(w2.codes[e], w2.exps[e])), "silu", y[b:b + c], None, None, f"{e}")
            else:
                ref = X.double() @ W.T
                check(y[b:b + c], ref, u(dtype) * ref.abs() + product_error(X, W) + tiny(dtype), f"y {e}")
        b += c


def test_not_a_number_stays_in_its_row():
    rows, n_in, n_out, pad = DENSE[2]
    g = gen(8)
    for p in (0, pad):
        n = 3800 if p == 0 else rows
        x, w = randn(g, n, n_in), weights(g, n_out, n_in)
        want = moe.moe_linear_fp4(strided(x, p), w)
        x[3, 1], x[n - 1, 5] = float("nan"), float("inf")
        y = moe.moe_linear_fp4(strided(x, p), w)
        ok = torch.ones(n, dtype=torch.bool, device=DEV)
        ok[3] = ok[n - 1] = False
        assert torch.equal(y[ok], want[ok]) and torch.isnan(y[3]).all()
        col = values(w)[:, 5]
        assert torch.equal(torch.isnan(y[n - 1]), col == 0)


def _calls(g):
    (rows, n_in, n_out, pad), (grows, gin, gout, gpad) = DENSE[2], GATED[1]
    (counts, ein, eout, epad), (counts2, ein2, eout2, epad2) = GROUPED[1], GROUPED_GATED[1]
    inputs = [strided(randn(g, r, c), p) for r, c, p in
              ((rows, n_in, pad), (3800, n_in, 0), (grows, gin, gpad), (sum(counts), ein, epad), (sum(counts2), ein2, epad2))]
    x, xa, xg, xe, xe2 = inputs
    w, wg, wu = weights(g, n_out, n_in), weights(g, gout, gin), weights(g, gout, gin)
    we, we2, we3 = weights(g, len(counts), eout, ein), weights(g, len(counts2), eout2, ein2), weights(g, len(counts2), eout2, ein2)
    off, off2 = offsets_of(counts), offsets_of(counts2)

    def calls(stream=None):
        return [moe.moe_linear_fp4(x, w, act="gelu", stream=stream), moe.moe_linear_fp4(xa, w, stream=stream),
                moe.moe_gated_linear_fp4(xg, wg, wu, stream=stream), moe.moe_grouped_matmul_fp4(xe, off, we, stream=stream),
                moe.moe_grouped_gated_fp4(xe2, off2, we2, we3, stream=stream)]
    return calls, inputs


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


@pytest.mark.parametrize("at", [1, 2, 3])
def test_exponents_at_any_address(at):
    """Exponents that start at any byte, read one, four or a thread's own at a time: as those of an array of their own."""
    def moved(w):
        buf = torch.zeros(w.exps.numel() + 16, dtype=torch.uint8, device=DEV)
        exps = buf[at:at + w.exps.numel()].view(w.exps.shape)
        exps.copy_(w.exps)
        return moe.Fp4Weights(w.codes, exps)

    g = gen(at)
    for rows, n_in, n_out in [(1, 256, 200), (3, 2048, 130), (10, 384, 96), (40, 256, 520), (150, 160, 72), (600, 512, 264),
                              DENSE[0][:3]]:
        x, w, w2 = randn(g, rows, n_in), weights(g, n_out, n_in), weights(g, n_out, n_in)
        assert torch.equal(moe.moe_linear_fp4(x, moved(w)), moe.moe_linear_fp4(x, w))
        assert torch.equal(moe.moe_gated_linear_fp4(x, moved(w), moved(w2)), moe.moe_gated_linear_fp4(x, w, w2))
    for counts in ([1, 0, 2], [40, 9, 100]):
        x, off, w, w2 = randn(g, sum(counts), 640), offsets_of(counts), weights(g, 3, 136, 640), weights(g, 3, 136, 640)
        assert torch.equal(moe.moe_grouped_matmul_fp4(x, off, moved(w)), moe.moe_grouped_matmul_fp4(x, off, w))
        assert torch.equal(moe.moe_grouped_gated_fp4(x, off, moved(w), moved(w2)), moe.moe_grouped_gated_fp4(x, off, w, w2))
