"""Host-side checks of the norm and the 8-bit entry points, without a GPU: every call here
fails validation or has nothing to launch."""
import ctypes

import pytest
import torch

import sparsely_gated_mixture_moe_b200 as moe

P = ctypes.c_void_p(0x100000)      # never dereferenced
ODD = ctypes.c_void_p(0x100004)    # not 16-byte aligned
L = moe.lib


def norm(rows=4, d=64, dtype=1, eps=1e-6, x=P, res=None, w=P, out=None, y=P, q=None, s=None, rstd=None):
    return L.moe_rmsnorm(rows, d, dtype, eps, x, res, w, out, y, q, s, rstd, None)


def test_rmsnorm():
    assert norm(rows=0) == 0
    assert norm(rows=-1) == 1 and norm(d=0) == 1 and norm(dtype=2) == 1
    assert norm(d=60) == 2 and norm(d=16392) == 2 and norm(rows=1 << 31) == 2
    assert norm(d=24, q=P, s=P) == 2                     # 8-bit rows need d % 16 == 0
    assert norm(eps=-1.0) == 1 and norm(eps=float("nan")) == 1
    assert norm(x=None) == 1 and norm(w=None) == 1 and norm(y=None) == 1
    assert norm(q=P) == 1 and norm(s=P) == 1             # both or neither
    for k in ("x", "res", "w", "out", "y"):
        assert norm(**{k: ODD}) == 1


def back(rows=4, d=64, dtype=1, r=P, w=P, rstd=P, dy=P, dres=None, dx=P, dw=None, ws=None):
    return L.moe_rmsnorm_backward(rows, d, dtype, r, w, rstd, dy, dres, dx, dw, ws, None)


def test_rmsnorm_backward():
    assert back(rows=0) == 0
    assert back(rows=-1) == 1 and back(d=60) == 2 and back(dtype=7) == 1
    for k in ("r", "w", "rstd", "dy", "dx"):
        assert back(**{k: None}) == 1
    assert back(dw=P) == 1                                # dweight needs a workspace
    for k in ("r", "w", "dy", "dres", "dx"):
        assert back(**{k: ODD}) == 1
    assert back(dw=P, ws=ODD) == 1
    size = L.moe_rmsnorm_backward_workspace_size
    assert size(1, 64) == 256 and size(10 ** 6, 64) >= 256 and size(4, 60) == 0 and size(-1, 64) == 0
    assert size(10 ** 6, 1024) <= 1024 * 1024 * 4


def test_quantisers():
    rows = lambda n=4, d=64, t=1, x=P, q=P, s=P: L.moe_quantize_rows_fp8(n, d, t, x, q, s, None)  # noqa: E731
    assert rows(n=0) == 0
    assert rows(n=-1) == 1 and rows(d=0) == 1 and rows(t=3) == 1 and rows(d=24) == 2
    assert rows(x=None) == 1 and rows(q=None) == 1 and rows(s=None) == 1 and rows(x=ODD) == 1 and rows(q=ODD) == 1
    w = lambda g=2, n=64, k=64, t=1, x=P, q=P, s=P: L.moe_quantize_weights_fp8(g, n, k, t, x, q, s, None)  # noqa: E731
    assert w(g=0) == 0
    assert w(g=-1) == 1 and w(n=0) == 1 and w(k=0) == 1 and w(t=-1) == 1 and w(k=24) == 2
    assert w(g=1 << 30, n=1024, k=1024) == 2
    big = (1 << 30) + 16                                  # block counts are 32-bit
    assert rows(d=big) == 2 and w(n=big) == 2 and w(k=big) == 2 and w(k=(1 << 31) - 16) == 2
    assert w(x=None) == 1 and w(q=ODD) == 1


def mm(M=4, N=64, K=64, a=P, sa=P, b=P, sb=P, out=P, t=0, ws=P):
    return L.moe_matmul_fp8(M, N, K, a, sa, b, sb, out, t, ws, None)


def gm(rows=4, N=64, K=64, G=2, a=P, sa=P, off=P, b=P, sb=P, out=P, t=0, ws=P):
    return L.moe_grouped_matmul_fp8(rows, N, K, G, a, sa, off, b, sb, out, t, ws, None)


def test_products():
    assert mm(M=0) == 0 and gm(rows=0) == 0
    for f in (mm, gm):
        assert f(N=0) == 1 and f(K=0) == 1 and f(t=2) == 1
        assert f(N=60) == 2 and f(K=24) == 2 and f(K=(1 << 30) + 16) == 2 and f(N=(1 << 31) - 8) == 2
        for k in ("a", "sa", "b", "sb", "out", "ws"):
            assert f(**{k: None}) == 1
        for k in ("a", "b", "out", "ws"):
            assert f(**{k: ODD}) == 1
    assert mm(M=-1) == 1 and mm(M=(1 << 31) - 1) == 2
    assert gm(rows=-1) == 1 and gm(G=0) == 1 and gm(G=1025) == 2 and gm(off=None) == 1
    assert gm(G=1024, N=1 << 22) == 2                     # weight rows past 32-bit coordinates


def cfg(**kw):
    base = dict(T=8, d_model=64, d_ff=64, E=4, k=1, dtype="bf16")
    base.update(kw)
    return ctypes.byref(moe.make_config(**base))


def test_gather_and_ffn():
    def gather(c=None, a=(P,) * 7):
        return L.moe_gather_rows_fp8(c if c is not None else cfg(), *a, None)

    def ffn(c=None, a=(P,) * 11):
        return L.moe_expert_ffn_fp8(c if c is not None else cfg(), *a, None)

    for f, n, loose in ((gather, 7, (1, 2, 3, 5)), (ffn, 11, (1, 2, 4, 6, 8))):
        assert f(c=cfg(T=0)) == 0
        assert f(c=cfg(dtype="f32")) == 2 and f(c=cfg(d_model=96)) == 2 and f(c=cfg(k=5)) == 1
        for i in range(n):
            assert f(a=tuple(None if j == i else P for j in range(n))) == 1
            if i not in loose:   # scales and indices need 4-byte alignment alone
                assert f(a=tuple(ODD if j == i else P for j in range(n))) == 1
    assert ffn(c=cfg(hidden_f16=True)) == 2


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = torch.zeros(4, 64).to(torch.float8_e4m3fn)
    s = torch.zeros(1, 4)
    for call in (lambda: moe.moe_rmsnorm(x, x[0], y=x), lambda: moe.moe_quantize_rows_fp8(x, q, s),
                 lambda: moe.moe_quantize_weights_fp8(x, q, s),
                 lambda: moe.moe_matmul_fp8(q, s, q, s, x, x),
                 lambda: moe.moe_grouped_matmul_fp8(q, s, s, q, s, x, x),
                 lambda: moe.moe_rmsnorm_backward(x, x[0], s, x, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        moe.moe_rmsnorm(None, x, y=x)
