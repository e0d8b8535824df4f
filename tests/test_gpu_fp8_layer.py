"""The norm, the 8-bit operators and the layer together, as they are used: served through
MoELayerFP8, and trained through the norm, the training forward and both backward passes."""
import numpy as np
import pytest
import torch

import sparsely_gated_mixture_moe_b200 as moe
import workloads
from oracle import lowp_oracle as lo
from oracle import moe_oracle as orc
from tests import gpu_harness as H
from workloads import Workload

pytestmark = pytest.mark.gpu

LAYERS = {
    "decode": Workload("fd", T=8, d_model=256, d_ff=512, E=16, k=2, act="gelu", seed=3),
    "one_token": Workload("f1", T=1, d_model=128, d_ff=128, E=4, k=1, renorm=False, act="relu", seed=3),
    "batch_drops": Workload("fb", T=700, d_model=192, d_ff=320, E=8, k=2, capacity_factor=0.9, act="gelu", seed=4),
    "noisy": Workload("fn", T=300, d_model=128, d_ff=256, E=32, k=4, gating="noisy_topk", act="relu", seed=5),
    "hierarchical": Workload("fh", T=260, d_model=128, d_ff=192, E=16, k=4, gating="hierarchical", groups=4,
                             k_primary=2, act="relu", seed=6),
    "large": Workload("fl", T=6000, d_model=256, d_ff=2560, E=4, k=2, act="gelu", seed=7),
}


def layer_of(w, normed, y_bf16=False):
    inp = workloads.make_inputs(w)
    dev = H.to_device(inp)
    cfg = moe.make_config(w.T, w.d_model, w.d_ff, w.E, w.k, gating=w.gating, renorm=w.renorm,
                          capacity_factor=w.capacity_factor, act=w.act, dtype="bf16", groups=w.groups,
                          k_primary=w.k_primary, y_bf16=y_bf16)
    weights = {k: dev[k] for k in ("w_gate", "w_noise", "w1", "w2") if k in dev}
    if normed:
        g = torch.Generator("cuda").manual_seed(9)
        weights["norm"] = (1 + 0.1 * torch.randn(w.d_model, device="cuda", generator=g)).bfloat16()
    return inp, dev, cfg, weights, moe.MoELayerFP8(cfg, weights)


@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("name", list(LAYERS))
def test_served(name, normed):
    """Against the fp64 layer on the 16-bit rows the router saw, following the GPU's choice.
    Each e4m3 value is off by at most half a step, 2^-4 of itself and 2^-4 / sqrt(3) = 3.6 % in
    the mean square: the first product has two such operands (5.1 %, times at most 1.13 through
    the activation), the second h and its weights: 7.7 % of y's norm together."""
    w = LAYERS[name]
    inp, dev, cfg, weights, layer = layer_of(w, normed)
    residual = None
    if normed:
        residual = torch.randn(w.T, w.d_model, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    y = layer.forward(dev["x"], residual=residual, noise=dev.get("noise"))
    assert moe.moe_get_error(layer.ws) == 0
    rows = layer.n if normed else dev["x"]
    if normed:
        r = H.f64(dev["x"]) + H.f64(residual)
        assert (np.abs(H.f64(layer.residual) - r) <= 2.0 ** -8 * np.abs(r) * (1 + 2.0 ** -20)).all()
        want, _ = lo.rmsnorm(H.f64(layer.residual), H.f64(weights["norm"]), 1e-6)
        assert (np.abs(H.f64(rows) - want) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(want)).all()
    # the same rows through the 16-bit layer's router choose the same experts
    wide = moe.MoELayer(cfg, {k: v for k, v in weights.items() if k != "norm"})
    y16 = wide.forward(rows.contiguous(), noise=dev.get("noise"))
    assert torch.equal(wide.topk_idx, layer.topk_idx) and torch.equal(wide.topk_gate, layer.topk_gate)
    a, b = H.f64(y), H.f64(y16)
    assert np.linalg.norm(a - b) <= 0.077 * np.linalg.norm(b)
    assert np.array_equal((a == 0).all(1), (b == 0).all(1))      # dropped tokens


def test_served_from_a_graph_and_in_bf16():
    """A captured decode step replayed on new rows equals the eager one; y_bf16 is its y
    rounded."""
    w = LAYERS["decode"]
    inp, dev, cfg, weights, layer = layer_of(w, True)
    x = dev["x"].clone()
    res = torch.zeros_like(x)
    layer.forward(x, residual=res)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(x, residual=res)
    eager = moe.MoELayerFP8(cfg, {**weights, "w1": layer.w["w1"], "w2": layer.w["w2"]})
    cfg16 = moe.MoEConfig.from_buffer_copy(cfg)
    cfg16.y_bf16 = 1
    short = moe.MoELayerFP8(cfg16, {**weights, "w1": layer.w["w1"], "w2": layer.w["w2"]})
    for seed in (31, 32, 33):
        gen = torch.Generator("cuda").manual_seed(seed)
        x.copy_(torch.randn(x.shape, device="cuda", generator=gen))
        res.copy_(torch.randn(x.shape, device="cuda", generator=gen))
        layer.y.fill_(-7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.y, eager.forward(x, residual=res))
        assert torch.equal(short.forward(x, residual=res), layer.y.bfloat16())
    assert moe.moe_get_error(layer.ws) == 0


def test_trained_through_the_norm():
    """r = x + residual -> norm -> moe_forward_train -> moe_backward -> moe_rmsnorm_backward, with a
    gradient past the layer on the residual stream: the norm's gradients against the fp64
    formula at the layer's own dx, and the layer's dx against its 16-bit self alone."""
    w = Workload("ft", T=600, d_model=128, d_ff=256, E=8, k=2, act="gelu", seed=1)
    inp = workloads.make_inputs(w)
    dev = H.to_device(inp)
    cfg = H.config_of(w)
    T, d, f, E, k = w.T, w.d_model, w.d_ff, w.E, w.k
    new = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    gen = torch.Generator("cuda").manual_seed(5)
    bf16, i32 = torch.bfloat16, torch.int32
    residual = torch.randn(T, d, device="cuda", generator=gen).to(bf16)
    gain = (1 + 0.1 * torch.randn(d, device="cuda", generator=gen)).to(bf16)
    r, n, rstd = new(T, d, t=bf16), new(T, d, t=bf16), new(T)
    moe.moe_rmsnorm(dev["x"], gain, 1e-5, residual=residual, residual_out=r, y=n, rstd=rstd)
    y, idx, gate, counts = new(T, d), new(T, k, t=i32), new(T, k), new(E, t=i32)
    state, ws = moe.train_state(cfg), moe.backward_workspace(cfg)
    moe.moe_forward_train(cfg, n, dev["w_gate"], dev["w1"], dev["w2"], y, idx, gate, counts, state, ws)
    dout = torch.randn(T, d, device="cuda", generator=gen)   # gradient of r + y
    dn, dw_gate, dw1, dw2, dgates = new(T, d), new(E, d), new(E, f, d), new(E, d, f), new(T, k)
    moe.moe_backward(cfg, n, dev["w_gate"], dev["w1"], dev["w2"], idx, gate, state, dout, dn, dw_gate, dw1, dw2,
                     dgates, ws)
    dx, dgain = new(T, d), new(d)
    moe.moe_rmsnorm_backward(r, gain, rstd, dn, dx, moe.rmsnorm_backward_workspace(T, d), dresidual=dout,
                             dweight=dgain)
    assert moe.moe_get_error(ws) == 0
    R, W, S, D = (H.f64(t) for t in (r, gain, rstd, dn))
    want, wgain = lo.rmsnorm_backward(R, W, S, D, H.f64(dout))
    mag = S[:, None] * (np.abs(D * W) + np.abs(R * S[:, None]) * np.abs(D * W * R * S[:, None]).mean(1, keepdims=True))
    assert (np.abs(H.f64(dx) - want) <= 64 * 2.0 ** -24 * (mag + np.abs(H.f64(dout)))).all()
    assert (np.abs(H.f64(dgain) - wgain) <= 100 * 2.0 ** -24 * np.abs(D * R * S[:, None]).sum(0)).all()
    # the chain's directional derivative against differences of the fp64 norm at the layer's dx:
    # sum(dn * norm(r)) + sum(dout * r) along a random direction
    v = np.random.default_rng(0).normal(size=(T, d))
    loss = lambda q: (D * lo.rmsnorm(q, W, 1e-5)[0]).sum() + (H.f64(dout) * q).sum()  # noqa: E731
    h = 1e-5
    num = (loss(R + h * v) - loss(R - h * v)) / (2 * h)
    # rstd within 32 u of the formula's, as in the forward's test
    assert abs((H.f64(dx) * v).sum() - num) <= 1e-5 * np.abs(H.f64(dx) * v).sum()


def test_layer_refuses_other_rows():
    """Rows of another type, shape or device are refused, with a norm and without."""
    for normed in (False, True):
        inp, dev, cfg, weights, layer = layer_of(LAYERS["decode"], normed)
        x = dev["x"]
        for bad in (x.float(), x[:4], x[:, :128].contiguous(), x.cpu(), x.t().contiguous().t()):
            with pytest.raises(ValueError):
                layer.forward(bad)
        if not normed:
            with pytest.raises(ValueError):
                layer.forward(x, residual=x)
