"""Pins of oracle/lowp_oracle.py: e4m3 against torch's conversion, hand-worked scales, the
norm's gradients against differences of its forward, and the grouped product against one
product per row."""
import numpy as np
import pytest
import torch

from oracle import lowp_oracle as lo


def test_e4m3_is_torchs_conversion():
    """Every e4m3 value, the midpoints between neighbours (ties to even) and random values."""
    values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    finite = values[torch.isfinite(values)].unique()
    mid = (finite[1:] + finite[:-1]) / 2
    g = torch.Generator().manual_seed(1)
    rnd = torch.randn(20000, generator=g) * torch.exp2(torch.rand(20000, generator=g) * 20 - 12)
    v = torch.cat([finite, mid, rnd.clamp(-448, 448)])
    assert np.array_equal(lo.e4m3(v.double().numpy()), v.to(torch.float8_e4m3fn).double().numpy())
    assert lo.e4m3(1e9) == 448.0 and lo.e4m3(-1e9) == -448.0 and np.isnan(lo.e4m3(np.nan))


def test_row_scales_by_hand():
    x = np.zeros((2, 200))
    x[0, 3], x[0, 130], x[1, 199] = -896.0, 7.0, np.nan
    q, s = lo.quantize_rows(x)
    assert s.shape == (2, 2)
    assert s[0, 0] == 2.0 and q[0, 3] == -448.0
    assert s[1, 0] == 7.0 / 448.0 and q[0, 130] == 448.0
    assert s[0, 1] == 2.0 ** -126 and not q[1, :128].any()      # zeros
    assert np.isnan(s[1, 1]) and np.isnan(q[1, 128:]).all()     # a NaN takes its block


def test_reads_back_within_half_a_step():
    x = np.random.default_rng(0).normal(size=(50, 333)) * 10
    q, s = lo.quantize_rows(x)
    step = np.repeat(s.T, 128, 1)[:, :333]
    assert (np.abs(lo.rows_value(q, s) - x) <= np.abs(x) * 2.0 ** -4 + step * 2.0 ** -10).all()
    w = np.random.default_rng(1).normal(size=(2, 130, 270))
    qw, sw = lo.quantize_weights(w)
    assert sw.shape == (2, 2, 3)
    assert (np.abs(lo.weights_value(qw, sw) - w) <= np.abs(w) * 2.0 ** -4 + sw.max() * 2.0 ** -10).all()


def test_grouped_product_row_by_row():
    rng = np.random.default_rng(2)
    a, b, off = rng.normal(size=(9, 5)), rng.normal(size=(4, 3, 5)), [1, 4, 4, 7, 8]
    out, mag = lo.grouped_matmul(a, off, b)
    for r in range(9):
        g = [i for i in range(4) if off[i] <= r < off[i + 1]]
        if not g:
            assert np.isnan(out[r]).all()
        for i in g:
            assert np.allclose(out[r], [a[r] @ b[i][n] for n in range(3)])
            assert (mag[r] >= np.abs(out[r]) - 1e-12).all()


@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_gradients_against_differences(with_residual):
    rng = np.random.default_rng(3)
    r, w, dy = rng.normal(size=(4, 11)), rng.normal(size=11), rng.normal(size=(4, 11))
    dres = rng.normal(size=(4, 11)) if with_residual else None

    def loss(r_, w_):
        y, _ = lo.rmsnorm(r_, w_, 1e-3)
        return (dy * y).sum() + (0.0 if dres is None else (dres * r_).sum())

    _, rstd = lo.rmsnorm(r, w, 1e-3)
    dx, dw = lo.rmsnorm_backward(r, w, rstd, dy, dres)
    h = 1e-6
    for i in np.ndindex(4, 11):
        d = np.zeros_like(r)
        d[i] = h
        assert abs((loss(r + d, w) - loss(r - d, w)) / (2 * h) - dx[i]) < 1e-7
    for j in range(11):
        d = np.zeros_like(w)
        d[j] = h
        assert abs((loss(r, w + d) - loss(r, w - d)) / (2 * h) - dw[j]) < 1e-7
