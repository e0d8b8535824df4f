"""The 8-bit operators on the GPU against their fp64 definitions (oracle/lowp_oracle.py).

Tolerances, from the roundings the kernels make (u = 2^-24 for fp32):
  product   the tensor cores sum 128 products (exact in fp32) in an order of their own, at
            worst truncating: 128 * 2u of the sum of magnitudes; then one multiply-add a
            block and the product of the two scales: (blocks + 1) u more.  bf16 adds its half
            step, 2^-8 of the value.
  quotient  correctly rounded for values given in memory: equal to the oracle's for 16-bit
            inputs; the scale within u.
  h         half a step of e4m3 (2^-4 of the value, 2^-10 of the scale below its normal
            range) of the activation, which the product's error reaches with a slope of at
            most 1.13 (GELU), plus the GELU evaluation's 5e-7 (1 + |z|)."""
import numpy as np
import pytest
import torch
from scipy.special import erf

import sparsely_gated_mixture_moe_b200 as moe
from oracle import lowp_oracle as lo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F8 = torch.float8_e4m3fn


def f64(t):
    return (t.float() if t.dtype == F8 else t).double().cpu().numpy()


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def new_ws():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def quantised_rows(x):
    q = torch.empty(x.shape, dtype=F8, device="cuda")
    s = torch.empty(moe.scale_blocks(x.shape[1]), x.shape[0], device="cuda")
    moe.moe_quantize_rows_fp8(x, q, s)
    return q, s


def rows(seed, n, d, dtype=torch.bfloat16):
    x = torch.randn(n, d, device="cuda", generator=gen(seed))
    x[:, ::37] *= 20.0
    return x.to(dtype)


def weights(seed, groups, n, k):
    w = torch.randn(groups, n, k, device="cuda", generator=gen(seed)) * k ** -0.5
    return moe.quantize_weights(w)


def product_tol(mag, want, K, dtype):
    tol = (256 + lo.blocks(K) + 3) * U * mag
    return tol + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0)


# --------------------------------------------------------------------- quantising

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", [(1, 16), (1, 128), (3, 144), (7, 1024), (33, 1040), (1000, 272), (2, 8192)])
def test_quantize_rows(n, d, dtype):
    x = rows(n + d, n, d, dtype)
    x[0, : min(d, 128)] = 0.0
    if n > 2:
        x[2, d // 2] = 3.0e38                 # the largest finite magnitudes
        x[1] *= 1e-36                          # scales near their floor
    q, s = quantised_rows(x)
    wq, wsc = lo.quantize_rows(f64(x))
    assert np.all(np.abs(f64(s) - wsc) <= U * wsc)
    if dtype == torch.bfloat16:
        assert np.array_equal(f64(q), wq)
    else:  # a correctly rounded quotient may still sit on the other side of a midpoint
        amax = np.repeat(wsc.T * 448.0, 128, 1)[:, :d]
        exact = 448.0 * f64(x) / amax
        assert np.all(np.abs(f64(q) - exact) <= np.abs(exact) * (2.0 ** -4 + 4 * U) + 2.0 ** -10)
        assert np.mean(f64(q) != wq) < 1e-4


def test_quantize_rows_not_finite():
    """A NaN or an infinity reads back as NaN over its block and reaches no other."""
    x = rows(5, 4, 384)
    x[1, 200], x[2, 5], x[3, 383] = float("nan"), float("inf"), float("-inf")
    q, s = quantised_rows(x)
    back = lo.rows_value(f64(q), f64(s))
    bad = np.zeros((4, 384), bool)
    bad[1, 128:256] = bad[2, :128] = bad[3, 256:] = True
    assert np.array_equal(np.isnan(back), bad)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(8, 16), (128, 128), (3, 136, 144), (2, 257, 400), (5, 64, 1024)])
def test_quantize_weights(shape, dtype):
    w = (torch.randn(*shape, device="cuda", generator=gen(9)) * 0.05).to(dtype)
    q, s = moe.quantize_weights(w)
    w3 = f64(w).reshape((-1,) + shape[-2:])
    wq, wsc = lo.quantize_weights(w3)
    assert np.all(np.abs(f64(s).reshape(wsc.shape) - wsc) <= U * wsc)
    same = f64(q).reshape(wq.shape) == wq
    assert same.all() if dtype == torch.bfloat16 else np.mean(~same) < 1e-4


# ----------------------------------------------------------------------- products

SHAPES = [(1, 8, 16), (1, 128, 128), (1, 1024, 8192), (3, 136, 144), (17, 4096, 1024), (127, 256, 128),
          (128, 256, 256), (129, 264, 272), (300, 520, 1040), (33, 1000, 2064), (257, 384, 4096),
          (513, 1024, 512), (1025, 768, 768),
          # CTA pairs (ragged rows, columns and depth); 32-row tiles of 256 columns; many blocks
          (4101, 1288, 272), (9000, 256, 400), (4096, 1280, 1024), (20, 19208, 144), (32, 20480, 128),
          (70, 136, 20000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(M, N, K, dtype):
    a, sa = quantised_rows(rows(M, M, K))
    b, sb = (t[0] for t in weights(N, 1, N, K))
    ws = new_ws()
    guard = torch.full((M + 2, N), -7.0, dtype=dtype, device="cuda")
    moe.moe_matmul_fp8(a, sa, b, sb, guard[1:-1], ws)
    assert moe.moe_get_error(ws) == 0
    want, mag = lo.grouped_matmul(lo.rows_value(f64(a), f64(sa)), [0, M],
                                  lo.weights_value(f64(b), f64(sb))[None])
    got = f64(guard)
    assert (got[0] == -7).all() and (got[-1] == -7).all()
    err = np.abs(got[1:-1] - want)
    assert (err <= product_tol(mag, want, K, dtype)).all(), (err / mag).max()


def test_matmul_any_scales():
    """Scales need not come from the quantiser: signs, powers of two, zeros, large spans."""
    M, N, K = 70, 304, 528
    a, sa = quantised_rows(rows(1, M, K))
    b, sb = (t[0] for t in weights(2, 1, N, K))
    sa = torch.randn(sa.shape, device="cuda", generator=gen(3)) * torch.exp2(
        torch.randint(-20, 20, sa.shape, device="cuda", generator=gen(4)).float())
    sa[:, 5] = 0.0
    sb = torch.exp2(torch.randint(-10, 10, sb.shape, device="cuda", generator=gen(5)).float())
    out, ws = torch.empty(M, N, device="cuda"), new_ws()
    moe.moe_matmul_fp8(a, sa, b, sb, out, ws)
    want, mag = lo.grouped_matmul(lo.rows_value(f64(a), f64(sa)), [0, M],
                                  lo.weights_value(f64(b), f64(sb))[None])
    assert (np.abs(f64(out) - want) <= product_tol(mag, want, K, torch.float32)).all()


def test_matmul_not_finite_stays_in_its_row_and_column():
    M, N, K = 40, 264, 272
    a, sa = quantised_rows(rows(1, M, K))
    b, sb = (t[0] for t in weights(2, 1, N, K))
    a.view(torch.uint8)[11, 100] = 0x7F
    b.view(torch.uint8)[130, 271] = 0x7F
    out, ws = torch.empty(M, N, device="cuda"), new_ws()
    moe.moe_matmul_fp8(a, sa, b, sb, out, ws)
    bad = np.zeros((M, N), bool)
    bad[11], bad[:, 130] = True, True
    assert np.array_equal(np.isnan(f64(out)), bad)


def test_matmul_output_on_a_16_byte_boundary():
    M, N, K = 130, 256, 256
    a, sa = quantised_rows(rows(1, M, K))
    b, sb = (t[0] for t in weights(2, 1, N, K))
    ws = new_ws()
    for dtype, skip in ((torch.bfloat16, 8), (torch.float32, 4)):
        ref = torch.empty(M, N, dtype=dtype, device="cuda")
        moe.moe_matmul_fp8(a, sa, b, sb, ref, ws)
        buf = torch.full((M * N + 2 * skip,), -7.0, dtype=dtype, device="cuda")
        moe.moe_matmul_fp8(a, sa, b, sb, buf[skip:-skip].view(M, N), ws)
        assert torch.equal(buf[skip:-skip].view(M, N), ref)
        assert (buf[:skip] == -7).all() and (buf[-skip:] == -7).all()


GROUPS = {
    "one_row_each": [1] * 9,
    "mostly_empty": [0, 0, 5, 0, 0, 0, 1, 0],
    "ragged": [1, 0, 127, 128, 129, 300, 2],
    "one_large": [0, 2000, 3],
    "all_empty": [0, 0, 0],
    "single": [77],
    "pairs_of_tiles": [700, 600, 513, 511],
    "many": [(7 * i) % 5 for i in range(200)],
    "medium": [100 - i for i in range(40)],
    "large": [2300, 1, 0, 2100],
    "large_and_empty": [0, 5000, 0, 255, 257],
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name,N,K", [(g, *nk) for g in GROUPS for nk in ((264, 272), (1024, 512), (5128, 144))
                                      if nk[0] * len(GROUPS[g]) < 200_000])
def test_grouped_matmul(name, N, K, dtype):
    """Rows in front of the first group and behind the last hold NaN bytes and scales, and
    their output rows keep what was there."""
    sizes, lead, tail = GROUPS[name], 3, 40
    n = sum(sizes) + lead + tail
    off = np.concatenate([[0], np.cumsum(sizes)]) + lead
    a, sa = quantised_rows(rows(len(sizes), n, K))
    for i, j in ((0, lead), (n - tail, n)):
        a.view(torch.uint8)[i:j] = 0x7F
        sa[:, i:j] = float("nan")
    b, sb = weights(N, len(sizes), N, K)
    out, ws = torch.full((n, N), -7.0, dtype=dtype, device="cuda"), new_ws()
    moe.moe_grouped_matmul_fp8(a, sa, torch.tensor(off, dtype=torch.int32, device="cuda"), b, sb, out, ws)
    assert moe.moe_get_error(ws) == 0
    want, mag = lo.grouped_matmul(lo.rows_value(f64(a), f64(sa)), off, lo.weights_value(f64(b), f64(sb)))
    got = f64(out)
    assert (got[:lead] == -7).all() and (got[n - tail:] == -7).all()
    inner = slice(lead, n - tail)
    assert (np.abs(got[inner] - want[inner]) <= product_tol(mag, want, K, dtype)[inner]).all()


@pytest.mark.parametrize("off", [[0, 5, 4], [-1, 2, 4], [0, 3, 99]])
def test_grouped_matmul_bad_offsets(off):
    a, sa = quantised_rows(rows(1, 10, 128))
    b, sb = weights(2, 2, 128, 128)
    out, ws = torch.full((10, 128), -7.0, device="cuda"), new_ws()
    moe.moe_grouped_matmul_fp8(a, sa, torch.tensor(off, dtype=torch.int32, device="cuda"), b, sb, out, ws)
    assert moe.moe_get_error(ws) == moe.DEVERR["offsets"]
    assert (out == -7).all()
    moe.moe_grouped_matmul_fp8(a, sa, torch.tensor([0, 5, 10], dtype=torch.int32, device="cuda"), b, sb, out, ws)
    assert moe.moe_get_error(ws) == 0 and not (out == -7).any()


# ----------------------------------------------------------------- gather, experts

def routed(cfg, seed, skew=0.0):
    """Index arrays of a random choice through moe_permute (index arrays only)."""
    T, k, E = cfg.T, cfg.k, cfg.E
    score = torch.randn(T, E, device="cuda", generator=gen(seed)) - skew * torch.arange(E, device="cuda")
    idx = score.topk(k, dim=1).indices.to(torch.int32)
    i32 = dict(dtype=torch.int32, device="cuda")
    r = {"counts": torch.empty(E, **i32), "offsets": torch.empty(E + 1, **i32),
         "perm_src": torch.zeros(T * k, **i32), "slot_pos": torch.empty(T * k, **i32)}
    ws = moe.workspace(cfg)
    moe.moe_permute(cfg, idx, None, r["counts"], r["offsets"], r["perm_src"], r["slot_pos"], None, ws)
    assert moe.moe_get_error(ws) == 0
    r["ws"] = ws
    return r


EXPERTS = {  # T, d, f, E, k, act, capacity factor, skew
    "one_token": (1, 128, 256, 8, 2, "gelu", None, 0.0),
    "decode": (16, 1024, 1024, 64, 2, "gelu", None, 0.0),
    "odd_blocks": (130, 192, 320, 4, 1, "relu", None, 0.5),
    "drops": (500, 128, 192, 6, 2, "gelu", 0.7, 0.3),
    "skewed": (1500, 256, 512, 8, 2, "relu", None, 1.0),
    "large_groups": (2100, 256, 640, 2, 2, "gelu", None, 0.0),
    "pairs_gelu": (3000, 1024, 1344, 4, 2, "gelu", None, 0.3),
    "pairs_relu_drops": (5000, 256, 4160, 3, 1, "relu", 0.9, 0.5),
    "few_rows": (40, 256, 1088, 32, 1, "gelu", None, 0.1),
}


@pytest.mark.parametrize("name", list(EXPERTS))
def test_experts(name):
    T, d, f, E, k, act, cf, skew = EXPERTS[name]
    cfg = moe.make_config(T, d, f, E, k, capacity_factor=cf, act=act)
    r = routed(cfg, 3, skew)
    n, kept = T * k, int(r["offsets"][-1])
    x, xs = quantised_rows(rows(T, T, d))
    xp = torch.full((n, d), 1.0, device="cuda").to(F8)
    xsp = torch.full((moe.scale_blocks(d), n), -7.0, device="cuda")
    moe.moe_gather_rows_fp8(cfg, x, xs, r["perm_src"], r["offsets"], xp, xsp, r["ws"])
    token = (r["perm_src"][:kept] // k).long()
    assert torch.equal(xp[:kept].view(torch.uint8), x.view(torch.uint8)[token])
    assert torch.equal(xsp[:, :kept], xs[:, token])
    assert (xp[kept:].float() == 1).all() and (xsp[:, kept:] == -7).all()

    w1, s1 = weights(1, E, f, d)
    w2, s2 = weights(2, E, d, f)
    h = torch.full((n, f), 1.0, device="cuda").to(F8)
    hs = torch.full((moe.scale_blocks(f), n), -7.0, device="cuda")
    y = torch.full((n, d), -7.0, device="cuda")
    moe.moe_expert_ffn_fp8(cfg, xp, xsp, r["offsets"], w1, s1, w2, s2, h, hs, y, r["ws"])
    assert moe.moe_get_error(r["ws"]) == 0
    assert (h[kept:].float() == 1).all() and (hs[:, kept:] == -7).all() and (y[kept:] == -7).all()

    off = r["offsets"].cpu().numpy()
    z, mag = lo.grouped_matmul(lo.rows_value(f64(xp), f64(xsp)), off, lo.weights_value(f64(w1), f64(s1)))
    z, mag = z[:kept], mag[:kept]
    e = 1.13 * product_tol(mag, z, d, torch.float32)
    if act == "gelu":
        a = 0.5 * z * (1.0 + erf(z / np.sqrt(2.0)))
        e = e + 5e-7 * (1.0 + np.abs(z))
    else:
        a = np.maximum(z, 0.0)
    hk, hsk = f64(h)[:kept], f64(hs)[:, :kept]
    step = np.repeat(hsk.T, 128, 1)[:, :f]
    assert (np.abs(hk * step - a) <= 2.0 ** -4 * (np.abs(a) + e) * (1 + 8 * U) + e + step * 2.0 ** -10).all()
    fb = moe.scale_blocks(f)
    pad = lambda v: np.pad(v, ((0, 0), (0, fb * 128 - f))).reshape(kept, fb, 128)  # noqa: E731
    amax, emax = np.abs(pad(a)).max(2), pad(e).max(2)
    assert (np.abs(hsk.T * 448.0 - amax) <= emax + 4 * U * amax + lo.AMAX_FLOOR).all()
    # the second product from the h it was given
    want, mag = lo.grouped_matmul(lo.rows_value(hk, hsk), off, lo.weights_value(f64(w2), f64(s2)))
    assert (np.abs(f64(y)[:kept] - want) <= product_tol(mag, want, f, torch.float32)).all()


def test_gather_bad_indices():
    cfg = moe.make_config(20, 64, 64, 4, 1)
    r = routed(cfg, 1)
    x, xs = quantised_rows(rows(1, 20, 64))
    xp, xsp = torch.zeros(20, 64, device="cuda").to(F8), torch.zeros(1, 20, device="cuda")
    src = r["perm_src"].clone()
    src[3], src[7] = 20, -1
    moe.moe_gather_rows_fp8(cfg, x, xs, src, r["offsets"], xp, xsp, r["ws"])
    assert moe.moe_get_error(r["ws"]) == moe.DEVERR["slot"]
    assert not xp[3].float().any() and not xp[7].float().any() and xsp[0, 3] == 0 and xsp[0, 8] != 0
    off = r["offsets"].clone()
    off[-1] = 21
    before = xp.clone()
    moe.moe_gather_rows_fp8(cfg, x, xs, r["perm_src"], off, xp, xsp, r["ws"])
    assert moe.moe_get_error(r["ws"]) == moe.DEVERR["offsets"]
    assert torch.equal(xp.view(torch.uint8), before.view(torch.uint8))


# ------------------------------------------------ streams, graphs, sizes, refusals

def product_case(seed, M=300, N=520, K=1040):
    a, sa = quantised_rows(rows(seed, M, K))
    b, sb = (t[0] for t in weights(seed + 1, 1, N, K))
    return a, sa, b, sb


@pytest.mark.parametrize("M,N,K", [(1, 1024, 8192), (300, 520, 1040), (4101, 1288, 272)])
def test_same_bits_every_time_and_on_any_stream(M, N, K):
    args = product_case(7, M, N, K)
    ws = new_ws()
    first = torch.empty(M, N, device="cuda")
    moe.moe_matmul_fp8(*args, first, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(20):
        out = torch.full_like(first, -7.0)
        torch.cuda.synchronize()
        moe.moe_matmul_fp8(*args, out, ws, stream=side if i % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    assert moe.moe_get_error(ws) == 0


def test_captured_graphs_share_a_workspace():
    """Two graphs on one workspace, replayed in turn on one stream with new inputs, give what
    eager calls give."""
    ws = new_ws()
    cases = [product_case(3), product_case(5, 4101, 1288, 272), product_case(9, 2, 256, 4096)]
    outs = [torch.empty(c[0].shape[0], c[2].shape[0], device="cuda") for c in cases]
    for c, o in zip(cases, outs):
        moe.moe_matmul_fp8(*c, o, ws)   # first calls set kernel attributes
    torch.cuda.synchronize()
    graphs = []
    for c, o in zip(cases, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_matmul_fp8(*c, o, ws)
        graphs.append(g)
    for seed in (21, 22):
        want = []
        for c in cases:
            M, K = c[0].shape
            q, s = quantised_rows(rows(seed, M, K))
            c[0].copy_(q)
            c[1].copy_(s)
            want.append(torch.empty(M, c[2].shape[0], device="cuda"))
            moe.moe_matmul_fp8(*c, want[-1], ws)
        for o in outs:
            o.fill_(-7.0)
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    assert moe.moe_get_error(ws) == 0


def test_output_past_2_31_elements():
    M, N, K = 140_000, 16_384, 16
    a, sa = quantised_rows(rows(1, M, K))
    b, sb = (t[0] for t in weights(2, 1, N, K))
    out, ws = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), new_ws()
    moe.moe_matmul_fp8(a, sa, b, sb, out, ws)
    bv = lo.weights_value(f64(b), f64(sb))
    for r in (0, 65_536, 131_071, 131_072, M - 1):
        av = lo.rows_value(f64(a[r:r + 1]), f64(sa[:, r:r + 1]))
        want, mag = lo.grouped_matmul(av, [0, 1], bv[None])
        assert (np.abs(f64(out[r:r + 1]) - want) <= product_tol(mag, want, K, torch.bfloat16)).all()
    assert moe.moe_get_error(ws) == 0


def test_no_rows():
    ws = new_ws()
    e8, e = torch.empty(0, 128, device="cuda").to(F8), torch.empty(1, 0, device="cuda")
    b, sb = weights(1, 2, 128, 128)
    out = torch.empty(0, 128, device="cuda")
    moe.moe_matmul_fp8(e8, e, b[0], sb[0], out, ws)
    moe.moe_grouped_matmul_fp8(e8, e, torch.zeros(3, dtype=torch.int32, device="cuda"), b, sb, out, ws)
    moe.moe_quantize_rows_fp8(torch.empty(0, 128, device="cuda"), e8, e)
    assert moe.last_launch_count() == 0


def test_refusals():
    a, sa, b, sb = product_case(1, 32, 64, 128)
    out, ws = torch.empty(32, 64, device="cuda"), new_ws()
    call = moe.moe_matmul_fp8
    with pytest.raises(ValueError):
        call(a.float(), sa, b, sb, out, ws)                      # type
    with pytest.raises(ValueError):
        call(a, sa.t().contiguous(), b, sb, out, ws)             # scales of another layout
    with pytest.raises(ValueError):
        call(a, sa, b, sb, torch.empty(64, 32, device="cuda").t(), ws)   # strides
    with pytest.raises(ValueError):
        call(a, sa, b, sb, out.half(), ws)
    with pytest.raises(ValueError):
        call(a, sa.cpu(), b, sb, out, ws)
    with pytest.raises(ValueError):
        call(a, sa, b, sb, out, ws[:128])                        # workspace too small
    with pytest.raises(TypeError):
        call(a, sa, b, sb, None, ws)
    with pytest.raises(TypeError):
        call(a, sa, b, sb, out, None)
    q = torch.empty(32, 24, dtype=F8, device="cuda")
    with pytest.raises(moe.MoEError):
        moe.moe_quantize_rows_fp8(torch.zeros(32, 24, device="cuda"), q, torch.empty(1, 32, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_rmsnorm(torch.zeros(4, 64, device="cuda"), torch.ones(32, device="cuda"),
                        y=torch.empty(4, 64, device="cuda"))
    with pytest.raises(moe.MoEError):
        moe.MoELayerFP8(moe.make_config(8, 64, 64, 4, 1, hidden_f16=True), {})
