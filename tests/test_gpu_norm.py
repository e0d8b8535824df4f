"""moe_rmsnorm and its backward against their fp64 definitions (oracle/lowp_oracle.py).

Tolerances from the kernels' fp32 roundings (u = 2^-24).  A row's sum of squares takes at most
32 multiply-adds a thread, 5 steps in the warp and 16 over warps: 53 u of a sum of positive
terms, half of it through the square root, with 4 more for the mean, eps, root and division:
rstd within 32 u.  y adds two products.  16-bit outputs add half a step (2^-8), 8-bit ones
2^-4 of the value and 2^-10 of the scale.  dweight sums at most rows / blocks values a thread,
8 rows of a block, 74 partials and 8 sums of those."""
import numpy as np
import pytest
import torch

import sparsely_gated_mixture_moe_b200 as moe
from oracle import lowp_oracle as lo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F8 = torch.float8_e4m3fn
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def f64(t):
    return (t.float() if t.dtype == F8 else t).double().cpu().numpy()


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def draw(seed, rows, d, dtype, scale=1.0):
    return (torch.randn(rows, d, device="cuda", generator=gen(seed)) * scale).to(dtype)


SHAPES = [(1, 16), (1, 1024), (3, 64), (5, 144), (9, 1040), (130, 768), (4, 4096), (7, 4112), (2, 8208), (3, 16384)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward(rows, d, residual, dtype):
    x, w = draw(1, rows, d, dtype), draw(2, 1, d, dtype)[0]
    res = draw(3, rows, d, dtype, 3.0) if residual else None
    guard = torch.full((rows + 2, d), -7.0, dtype=dtype, device="cuda")
    s, y = torch.empty_like(x), guard[1:-1]
    q = torch.empty(x.shape, dtype=F8, device="cuda")
    qs = torch.empty(moe.scale_blocks(d), rows, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    moe.moe_rmsnorm(x, w, 1e-5, residual=res, residual_out=s, y=y, y_q=q, y_scale=qs, rstd=rstd)
    r = f64(x) + (f64(res) if residual else 0.0)
    # the sum in fp32, then its type
    assert (np.abs(f64(s) - r) <= (HALF[dtype] + U) * np.abs(r) * (1 + U)).all()
    want, wr = lo.rmsnorm(f64(s), f64(w), 1e-5)     # what was stored is what is normalised
    assert (np.abs(f64(rstd) - wr) <= 32 * U * wr).all()
    e = 36 * U * np.abs(want)
    assert (np.abs(f64(y) - want) <= e + HALF[dtype] * (np.abs(want) + e)).all()
    assert (guard[0] == -7).all() and (guard[-1] == -7).all()
    sc = f64(qs)
    step = np.repeat(sc.T, 128, 1)[:, :d]
    assert (np.abs(f64(q) * step - want) <= (2.0 ** -4 * (1 + 8 * U)) * (np.abs(want) + e) + e + step * 2.0 ** -10).all()
    amax = lo.quantize_rows(want)[1]
    assert (np.abs(sc - amax) <= 40 * U * amax).all()
    # each output alone is the same output
    y2, q2, qs2 = torch.empty_like(x), torch.empty_like(q), torch.empty_like(qs)
    moe.moe_rmsnorm(x, w, 1e-5, residual=res, y=y2)
    moe.moe_rmsnorm(x, w, 1e-5, residual=res, y_q=q2, y_scale=qs2)
    assert torch.equal(y2, y) and torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(qs2, qs)


@pytest.mark.parametrize("d", [8, 24, 1000, 4104])
def test_forward_widths_of_8(d):
    x, w = draw(1, 6, d, torch.float32), draw(2, 1, d, torch.float32)[0]
    y = torch.empty_like(x)
    moe.moe_rmsnorm(x, w, 0.0, y=y)
    want, _ = lo.rmsnorm(f64(x), f64(w), 0.0)
    assert (np.abs(f64(y) - want) <= 36 * U * np.abs(want)).all()


def test_forward_in_place():
    """residual_out may be x or the residual itself."""
    x, res, w = (draw(i, n, 528, torch.bfloat16) for i, n in ((1, 40), (2, 40), (3, 1)))
    y0, s0 = torch.empty_like(x), torch.empty_like(x)
    moe.moe_rmsnorm(x, w[0], residual=res, residual_out=s0, y=y0)
    for inplace in ("x", "res"):
        a, b, y = x.clone(), res.clone(), torch.empty_like(x)
        out = a if inplace == "x" else b
        moe.moe_rmsnorm(a, w[0], residual=b, residual_out=out, y=y)
        assert torch.equal(out, s0) and torch.equal(y, y0)


def test_forward_rows_of_zeros_and_not_finite():
    x, w = draw(1, 4, 256, torch.float32), draw(2, 1, 256, torch.float32)[0]
    x[1] = 0.0
    x[2, 7] = float("nan")
    y, q, s = torch.empty_like(x), torch.empty(4, 256, dtype=F8, device="cuda"), torch.empty(2, 4, device="cuda")
    moe.moe_rmsnorm(x, w, 1e-6, y=y, y_q=q, y_scale=s)
    assert not y[1].any() and not q[1].float().any() and (s[:, 1] == 2.0 ** -126).all()
    assert torch.isnan(y[2]).all() and torch.isnan(q[2].float()).all() and torch.isnan(s[:, 2]).all()
    assert torch.isfinite(y[[0, 1, 3]]).all() and torch.isfinite(s[:, [0, 1, 3]]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,d", [(1, 8), (1, 1024), (2, 72), (9, 1000), (700, 768), (333, 2568), (5000, 264),
                                    (40, 8200), (20, 16384)])
def test_backward(rows, d, residual, dtype):
    r, w = draw(1, rows, d, dtype), draw(2, 1, d, dtype)[0]
    dy = draw(3, rows, d, torch.float32)
    dres = draw(4, rows, d, torch.float32) if residual else None
    rstd = torch.empty(rows, device="cuda")
    moe.moe_rmsnorm(r, w, 1e-5, rstd=rstd)
    guard = torch.full((rows + 2, d), -7.0, device="cuda")
    dx, dw = guard[1:-1], torch.full((d,), float("nan"), device="cuda")
    ws = moe.rmsnorm_backward_workspace(rows, d)
    moe.moe_rmsnorm_backward(r, w, rstd, dy, dx, ws, dresidual=dres, dweight=dw)
    R, W, S, D = f64(r), f64(w), f64(rstd), f64(dy)
    want, wdw = lo.rmsnorm_backward(R, W, S, D, f64(dres) if residual else None)
    xhat = R * S[:, None]
    mean_abs = np.abs(D * W * xhat).mean(1, keepdims=True)
    mag = S[:, None] * (np.abs(D * W) + np.abs(xhat) * mean_abs) + (np.abs(f64(dres)) if residual else 0.0)
    assert (np.abs(f64(dx) - want) <= 64 * U * mag).all()
    n = -(-rows // 592) + 8 + 74 + 8 + 2
    assert (np.abs(f64(dw) - wdw) <= n * U * np.abs(D * xhat).sum(0)).all()
    assert (guard[0] == -7).all() and (guard[-1] == -7).all()
    # the weight gradient is repeatable bit for bit; dx alone is the same dx
    dw2, dx2 = torch.empty_like(dw), torch.empty_like(dy)
    moe.moe_rmsnorm_backward(r, w, rstd, dy, dx2, ws, dresidual=dres, dweight=dw2)
    assert torch.equal(dw2, dw)
    if residual:  # in place
        dx2 = dres.clone()
        moe.moe_rmsnorm_backward(r, w, rstd, dy, dx2, dresidual=dx2)
    else:
        moe.moe_rmsnorm_backward(r, w, rstd, dy, dx2)
    assert torch.equal(dx2, dx)


def test_backward_of_no_rows():
    dw = torch.full((64,), 3.0, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    moe.moe_rmsnorm_backward(e, dw.clone(), torch.empty(0, device="cuda"), e, e,
                             torch.empty(256, dtype=torch.uint8, device="cuda"), dweight=dw)
    assert not dw.any()


def test_rows_past_2_31_elements():
    rows, d = 140_000, 16_384
    x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(1))
    w = draw(2, 1, d, torch.bfloat16)[0]
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    moe.moe_rmsnorm(x, w, y=y, rstd=rstd)
    for r in (0, 131_071, 131_072, rows - 1):
        want, wr = lo.rmsnorm(f64(x[r:r + 1]), f64(w), 1e-6)
        assert abs(f64(rstd[r:r + 1]) - wr) <= 32 * U * wr
        assert (np.abs(f64(y[r:r + 1]) - want) <= (36 * U + HALF[torch.bfloat16] * (1 + 36 * U)) * np.abs(want)).all()


def test_captured_and_on_another_stream():
    """Forward and backward captured into one graph and replayed on new inputs equal the eager
    calls, as do calls on a side stream."""
    rows, d = 1500, 768
    x, res, w = draw(1, rows, d, torch.bfloat16), draw(2, rows, d, torch.bfloat16), draw(3, 1, d, torch.bfloat16)[0]
    dy = draw(4, rows, d, torch.float32)
    f32 = dict(dtype=torch.float32, device="cuda")
    ws = moe.rmsnorm_backward_workspace(rows, d)

    def outputs():
        return {"r": torch.empty_like(x), "y": torch.empty_like(x), "q": torch.empty(rows, d, dtype=F8, device="cuda"),
                "s": torch.empty(moe.scale_blocks(d), rows, **f32), "rstd": torch.empty(rows, **f32),
                "dx": torch.empty(rows, d, **f32), "dw": torch.empty(d, **f32)}

    def step(o, stream=None):
        moe.moe_rmsnorm(x, w, residual=res, residual_out=o["r"], y=o["y"], y_q=o["q"], y_scale=o["s"], rstd=o["rstd"],
                        stream=stream)
        moe.moe_rmsnorm_backward(o["r"], w, o["rstd"], dy, o["dx"], ws, dresidual=dy, dweight=o["dw"], stream=stream)

    o = outputs()
    step(o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(o)
    side = torch.cuda.Stream()
    for seed in (11, 12):
        x.copy_(draw(seed, rows, d, torch.bfloat16))
        want = outputs()
        step(want)
        torch.cuda.synchronize()
        for k in o:
            o[k].view(torch.uint8).zero_()
        g.replay()
        torch.cuda.synchronize()
        other = outputs()
        torch.cuda.synchronize()
        step(other, stream=side)
        torch.cuda.synchronize()
        for k in o:
            assert torch.equal(o[k].view(torch.uint8), want[k].view(torch.uint8)), k
            assert torch.equal(other[k].view(torch.uint8), want[k].view(torch.uint8)), k


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,d", [(64, 1024), (33, 2576), (8, 8208)])
def test_forward_ties_of_the_8_bit_output(rows, d, residual):
    """For 16-bit r and w, 448 y / max|y| = 448 r w / max|r w| is a quotient of whole numbers
    below 2^25 but for powers of two.  Where it is not midway between two e4m3 values it is at
    least 2^-22 of itself away, more than an fp32 rounding; where it is midway, it is so
    exactly.  So the output is the rounding to nearest even of the exact quotient, whatever
    the row's rstd."""
    x, w = draw(1, rows, d, torch.bfloat16), (1 + 0.1 * draw(2, 1, d, torch.float32)[0]).to(torch.bfloat16)
    res = draw(3, rows, d, torch.bfloat16) if residual else None
    s = torch.empty_like(x)
    q, qs = torch.empty(rows, d, dtype=F8, device="cuda"), torch.empty(moe.scale_blocks(d), rows, device="cuda")
    moe.moe_rmsnorm(x, w, 1e-5, residual=res, residual_out=s, y_q=q, y_scale=qs)
    want = lo.quantize_rows(f64(s) * f64(w))[0]
    assert (f64(q) == want).all()


@pytest.mark.parametrize("xs,ws", [(1.0, 1e-34), (1.0, 1e-36), (1.0, 1e-38), (1e-18, 1e-30), (1e-3, 3e37),
                                   (1e17, 1e30), (1e17, 1e-30), (1e-18, 1e35)])
def test_forward_small_and_large(xs, ws):
    """Blocks at and below the scale's floor, and outputs near the ends of fp32, from rows whose
    products with the weights alone leave it.  2^-148: steps of subnormal numbers; a block
    below the floor is divided by it to 1.2e-6 = 20 u."""
    x, w = draw(1, 9, 1040, torch.float32, xs), draw(2, 1, 1040, torch.float32)[0].clamp(-2, 2) * ws
    y, q = torch.empty_like(x), torch.empty(9, 1040, dtype=F8, device="cuda")
    s = torch.empty(moe.scale_blocks(1040), 9, device="cuda")
    moe.moe_rmsnorm(x, w, 0.0, y=y, y_q=q, y_scale=s)
    want, _ = lo.rmsnorm(f64(x), f64(w), 0.0)
    e = 36 * U * np.abs(want) + 2.0 ** -148
    assert (np.abs(f64(y) - want) <= e).all()
    sc, amax = f64(s), lo.quantize_rows(want)[1]
    assert (np.abs(sc - amax) <= 40 * U * amax).all() and (sc >= 2.0 ** -126).all()
    step = np.repeat(sc.T, 128, 1)[:, :1040]
    assert (np.abs(f64(q) * step - want) <= (2.0 ** -4 * (1 + 8 * U)) * (np.abs(want) + e) + e + step * 2.0 ** -10).all()


def test_forward_outputs_beyond_fp32():
    """100 ones of 256 values: rstd = 1.6, and y = 1.6 w overflows where w alone does not.  The
    block reads back as NaN throughout, its neighbour as zeros."""
    x = torch.zeros(2, 256, device="cuda")
    x[:, :100] = 1.0
    w = torch.full((256,), 3e38, device="cuda")
    y, q, s = torch.empty_like(x), torch.empty(2, 256, dtype=F8, device="cuda"), torch.empty(2, 2, device="cuda")
    moe.moe_rmsnorm(x, w, 0.0, y=y, y_q=q, y_scale=s)
    assert torch.isinf(y[:, :100]).all() and not y[:, 100:].any()
    back = lo.rows_value(f64(q), f64(s))
    assert np.isnan(back[:, :128]).all() and (back[:, 128:] == 0).all()
