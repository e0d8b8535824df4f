"""Cases of the 8-bit expert path and the norm in front of it, in plain torch and through libmoe.

A run of them together is one MoE block as it is served: the residual's addition and the
root-mean-square norm write the token rows in 8 bits, a dense product or the experts'
grouped products take them with a scale for each block of 128, and the gate-weighted
combine adds the experts' rows up.  The norm's backward is the training side of the block.

8-bit format: e4m3 values q with one fp32 scale s for 128 consecutive values of an
activation row and for each 128 x 128 block of a weight matrix: s = max|v| / 448, at least
2^-126, and q = 448 v / max|v| rounded to nearest even.  Activation scales lie block-major,
[blocks, rows]; weight scales [.., blocks of rows, blocks of columns].
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -126
EPS = 1e-6
KINDS = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the norm in front of a layer: one decode step of a few sequences (latency), the
        # widest training batch of the benchmark's layers, and an fp32 layer of odd width
        {"name": "norm_decode", "op": "norm", "rows": 4, "d": 1024, "dtype": "bf16", "residual": True, "y": True, "q": True},
        {"name": "norm_batch", "op": "norm", "rows": 65536, "d": 1024, "dtype": "bf16", "residual": True, "y": True, "q": True},
        {"name": "norm_f32_odd", "op": "norm", "rows": 4099, "d": 4104, "dtype": "f32", "residual": False, "y": True, "q": False},
        # its gradients: a training batch, and a short fp32 one of odd sizes
        {"name": "norm_grad_batch", "op": "norm_grad", "rows": 32768, "d": 1024, "dtype": "bf16", "residual": True},
        {"name": "norm_grad_f32_odd", "op": "norm_grad", "rows": 333, "d": 2568, "dtype": "f32", "residual": False},
        # a dense layer beside the experts: one token at a time from bf16 rows, a ragged
        # prompt whose width is no multiple of the block, and a long prefill
        {"name": "linear_decode", "op": "linear", "rows": 1, "n": 1024, "k": 8192, "a": "bf16", "out": "bf16"},
        {"name": "linear_odd", "op": "linear", "rows": 777, "n": 2056, "k": 1040, "a": "fp8", "out": "f32"},
        {"name": "linear_prefill", "op": "linear", "rows": 16384, "n": 8192, "k": 4096, "a": "fp8", "out": "bf16"},
        # products grouped by expert: a decode batch that leaves most experts empty or with
        # a row or two, and skewed experts of very different sizes
        {"name": "grouped_decode", "op": "grouped", "rows": 96, "n": 4096, "k": 1024, "groups": 64, "skew": 0.9, "out": "f32"},
        {"name": "grouped_skewed", "op": "grouped", "rows": 32771, "n": 4096, "k": 1024, "groups": 16, "skew": 1.2, "out": "bf16"},
        # dispatch, the experts' two products and the combine: a decode step, and the
        # benchmark's largest layer
        {"name": "experts_decode", "op": "experts", "tokens": 16, "d": 1024, "f": 4096, "experts": 64, "k": 2, "act": "gelu", "skew": 0.0},
        {"name": "experts_batch", "op": "experts", "tokens": 32768, "d": 1024, "f": 8192, "experts": 64, "k": 2, "act": "gelu", "skew": 0.0},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "grouped", "experts"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "norm":
        q = rng.random() < 0.6
        return {"op": op, "rows": _log(rng, 1, 32768), "d": _log(rng, 64, 8192, 16 if q else 8), "dtype": rng.choice(list(KINDS)),
                "residual": flag(), "y": True if not q else flag(), "q": q}
    if op == "norm_grad":
        return {"op": op, "rows": _log(rng, 1, 16384), "d": _log(rng, 64, 8192, 8), "dtype": rng.choice(list(KINDS)), "residual": flag()}
    if op == "linear":
        return {"op": op, "rows": _log(rng, 1, 8192), "n": _log(rng, 64, 8192, 8), "k": _log(rng, 64, 8192, 16),
                "a": rng.choice(["bf16", "fp8"]), "out": rng.choice(["bf16", "f32"])}
    if op == "grouped":
        return {"op": op, "rows": _log(rng, 1, 16384), "n": _log(rng, 64, 4096, 8), "k": _log(rng, 64, 4096, 16),
                "groups": _log(rng, 1, 128), "skew": rng.choice([0.0, 0.6, 1.2]), "out": rng.choice(["bf16", "f32"])}
    experts = _log(rng, 2, 128)
    return {"op": op, "tokens": _log(rng, 1, 8192), "d": _log(rng, 64, 1024, 64), "f": _log(rng, 64, 4096, 64), "experts": experts,
            "k": rng.randint(1, min(4, experts)), "act": rng.choice(["relu", "gelu"]), "skew": rng.choice([0.0, 0.8])}


def _blocks(n):
    return -(-n // BLOCK)


# ----------------------------------------------------------------------------- inputs

def _quantised_weights(g, groups, n, k):
    """Weights N(0, 1/k) as e4m3 with a scale for each 128 x 128 block."""
    dev = "cuda"
    nb, kb = _blocks(n), _blocks(k)
    w = torch.empty(groups, n, k, device=dev).normal_(0.0, k ** -0.5, generator=g)
    top = torch.zeros(groups, nb * BLOCK, kb * BLOCK, device=dev)
    top[:, :n, :k] = w.abs()
    scale = (top.view(groups, nb, BLOCK, kb, BLOCK).amax((2, 4)) / E4M3_MAX).clamp_min(TINY)
    del top
    w /= scale.repeat_interleave(BLOCK, 1)[:, :n].repeat_interleave(BLOCK, 2)[:, :, :k]
    return w.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _rows(g, rows, d):
    """Activations as a layer meets them: normal, a few channels much larger than the
    rest, and now and then a row of padding."""
    x = torch.empty(rows, d, device="cuda").normal_(generator=g)
    x[:, 5::257] *= 12.0
    if rows > 16:
        x[7::1000] = 0.0
    return x


def _quantised_rows(x):
    """(q [rows, k], scale [blocks, rows]).  The quotient in 64 bits: 16-bit values over the
    largest of their block often lie midway between two e4m3 values, where an error in the
    last place of 32 bits decides."""
    rows, k = x.shape
    v = torch.zeros(rows, _blocks(k) * BLOCK, device=x.device)
    v[:, :k] = x
    v = v.view(rows, -1, BLOCK)
    top = v.abs().amax(2).clamp_min(E4M3_MAX * TINY)
    q = (v.double() * E4M3_MAX / top.double()[:, :, None]).float().to(torch.float8_e4m3fn)
    return q.view(rows, -1)[:, :k].contiguous(), (top / E4M3_MAX).t().contiguous()


def _choice(g, tokens, experts, k, skew):
    """Chosen experts [tokens, k], distinct within a token; expert e's share falls with
    (e + 1)^-skew."""
    u = torch.rand(tokens, experts, device="cuda", generator=g).clamp_min(1e-9)
    gumbel = -torch.log(-torch.log(u))
    return (gumbel - skew * torch.log(torch.arange(1, experts + 1, device="cuda"))).topk(k, dim=1).indices


def _offsets(ids, groups):
    counts = torch.bincount(ids, minlength=groups)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    new = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device=dev)  # noqa: E731
    s = {"case": dict(case)}
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, d, t = case["rows"], case["d"], KINDS[case["dtype"]]
        s["x"] = _rows(g, rows, d).to(t)
        s["weight"] = (1.0 + 0.1 * torch.randn(d, device=dev, generator=g)).to(t)
    if op == "norm":
        s["residual"] = (2.0 * torch.randn(rows, d, device=dev, generator=g)).to(t) if case["residual"] else None
        s["sum"] = new(rows, d, t=t) if case["residual"] else None
        s["y"] = new(rows, d, t=t) if case["y"] else None
        s["q"] = new(rows, d, t=torch.float8_e4m3fn) if case["q"] else None
        s["scale"] = new(_blocks(d), rows) if case["q"] else None
        s["rstd"] = new(rows)
    elif op == "norm_grad":
        s["rstd"] = (s["x"].double().square().mean(1) + EPS).rsqrt().float()
        s["dy"] = torch.randn(rows, d, device=dev, generator=g) / math.sqrt(d)
        s["dsum"] = torch.randn(rows, d, device=dev, generator=g) / math.sqrt(d) if case["residual"] else None
        s["dx"], s["dweight"] = new(rows, d), new(d)
        s["ws"] = torch.zeros(1024 * d * 4, dtype=torch.uint8, device=dev)
    elif op == "linear":
        rows, n, k = case["rows"], case["n"], case["k"]
        x = _rows(g, rows, k)
        if case["a"] == "fp8":
            s["a"], s["a_scale"] = _quantised_rows(x)
        else:
            s["x"] = x.to(torch.bfloat16)
            s["a"], s["a_scale"] = new(rows, k, t=torch.float8_e4m3fn), new(_blocks(k), rows)
        w, ws = _quantised_weights(g, 1, n, k)
        s["w"], s["w_scale"] = w[0], ws[0]
        s["out"] = new(rows, n, t=KINDS[case["out"]])
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device=dev)
    elif op == "grouped":
        rows, n, k = case["rows"], case["n"], case["k"]
        s["offsets"] = _offsets(_choice(g, rows, case["groups"], 1, case["skew"])[:, 0], case["groups"])
        s["a"], s["a_scale"] = _quantised_rows(_rows(g, rows, k))
        s["w"], s["w_scale"] = _quantised_weights(g, case["groups"], n, k)
        s["out"] = new(rows, n, t=KINDS[case["out"]])
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device=dev)
    else:
        tokens, d, f, k, experts = (case[c] for c in ("tokens", "d", "f", "k", "experts"))
        rows = tokens * k
        ids = _choice(g, tokens, experts, k, case["skew"]).reshape(-1)
        s["offsets"] = _offsets(ids, experts)
        order = ids.sort(stable=True).indices
        s["perm_src"] = order.to(torch.int32)
        s["slot_pos"] = torch.empty_like(order).scatter_(0, order, torch.arange(rows, device=dev)).to(torch.int32)
        s["gates"] = torch.randn(tokens, k, device=dev, generator=g).softmax(1)
        s["x"], s["x_scale"] = _quantised_rows(_rows(g, tokens, d))
        s["w1"], s["w1_scale"] = _quantised_weights(g, experts, f, d)
        s["w2"], s["w2_scale"] = _quantised_weights(g, experts, d, f)
        f8 = torch.float8_e4m3fn
        s["x_perm"], s["x_perm_scale"] = new(rows, d, t=f8), new(_blocks(d), rows)
        s["h"], s["h_scale"] = new(rows, f, t=f8), new(_blocks(f), rows)
        s["y_perm"], s["y"] = new(rows, d), new(tokens, d, t=torch.bfloat16)
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------- the plain forms

def _read_rows(q, scale):
    """e4m3 rows and their [blocks, rows] scales as fp32 values."""
    return q.float() * scale.t().repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _read_weights(q, scale):
    return q.float() * scale.repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :].repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _padded(rows, offsets):
    """Rows [n, k] as [groups, longest, k], zeros behind each group's end; and where each
    padded place came from, and which of them hold a row."""
    start, count = offsets[:-1].long(), (offsets[1:] - offsets[:-1]).long()
    at = torch.arange(int(count.max()), device=rows.device)
    held = at < count[:, None]
    src = (start[:, None] + at).where(held, 0)
    return rows[src] * held[:, :, None], src, held


def _grouped(rows, offsets, weights):
    """out[s] = rows[s] . weights[g]^T for the rows s of each group g."""
    padded, src, held = _padded(rows, offsets)
    out = torch.bmm(padded, weights.transpose(1, 2))
    return torch.empty(rows.shape[0], weights.shape[1], device=rows.device).index_copy_(0, src[held], out[held])


def _act(z, act):
    return z.clamp_min(0.0) if act == "relu" else 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        x = s["x"].float()
        out = {}
        if c["residual"]:
            out["sum"] = (x + s["residual"].float()).to(s["x"].dtype)  # the stored sum is what is normalised
            x = out["sum"].float()
        out["rstd"] = (x.square().mean(1) + EPS).rsqrt()
        y = x * out["rstd"][:, None] * s["weight"].float()
        if c["y"]:
            out["y"] = y.to(s["x"].dtype)
        if c["q"]:
            out["q"], out["scale"] = _quantised_rows(y)
        return out
    if c["op"] == "norm_grad":
        xhat = s["x"].float() * s["rstd"][:, None]
        wdy = s["dy"] * s["weight"].float()
        dx = s["rstd"][:, None] * (wdy - xhat * (wdy * xhat).mean(1, keepdim=True))
        return {"dx": dx if s["dsum"] is None else dx + s["dsum"], "dweight": (s["dy"] * xhat).sum(0)}
    if c["op"] == "linear":
        a, scale = (s["a"], s["a_scale"]) if c["a"] == "fp8" else _quantised_rows(s["x"].float())
        out = _read_rows(a, scale) @ _read_weights(s["w"], s["w_scale"]).t()
        return {"out": out.to(KINDS[c["out"]])}
    if c["op"] == "grouped":
        out = _grouped(_read_rows(s["a"], s["a_scale"]), s["offsets"], _read_weights(s["w"], s["w_scale"]))
        return {"out": out.to(KINDS[c["out"]])}
    token = s["perm_src"].long() // c["k"]
    h = _grouped(_read_rows(s["x"], s["x_scale"])[token], s["offsets"], _read_weights(s["w1"], s["w1_scale"]))
    h = _read_rows(*_quantised_rows(_act(h, c["act"])))
    y_perm = _grouped(h, s["offsets"], _read_weights(s["w2"], s["w2_scale"]))
    y = (y_perm[s["slot_pos"].long()].view(c["tokens"], c["k"], -1) * s["gates"][:, :, None]).sum(1)
    return {"y": y.to(torch.bfloat16)}


# ----------------------------------------------------------------------------- a pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain(s)
    import sparsely_gated_mixture_moe_b200 as moe
    if c["op"] == "norm":
        moe.moe_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["sum"], y=s["y"], y_q=s["q"],
                        y_scale=s["scale"], rstd=s["rstd"])
        return {k: s[k] for k in ("sum", "rstd", "y", "q", "scale") if s[k] is not None}
    if c["op"] == "norm_grad":
        moe.moe_rmsnorm_backward(s["x"], s["weight"], s["rstd"], s["dy"], s["dx"], s["ws"], dresidual=s["dsum"], dweight=s["dweight"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if c["op"] == "linear":
        if c["a"] == "bf16":
            moe.moe_quantize_rows_fp8(s["x"], s["a"], s["a_scale"])
        moe.moe_matmul_fp8(s["a"], s["a_scale"], s["w"], s["w_scale"], s["out"], s["ws"])
        return {"out": s["out"]}
    if c["op"] == "grouped":
        moe.moe_grouped_matmul_fp8(s["a"], s["a_scale"], s["offsets"], s["w"], s["w_scale"], s["out"], s["ws"])
        return {"out": s["out"]}
    cfg = moe.make_config(c["tokens"], c["d"], c["f"], c["experts"], c["k"], act=c["act"], y_bf16=True)
    moe.moe_gather_rows_fp8(cfg, s["x"], s["x_scale"], s["perm_src"], s["offsets"], s["x_perm"], s["x_perm_scale"], s["ws"])
    moe.moe_expert_ffn_fp8(cfg, s["x_perm"], s["x_perm_scale"], s["offsets"], s["w1"], s["w1_scale"], s["w2"], s["w2_scale"],
                           s["h"], s["h_scale"], s["y_perm"], s["ws"])
    moe.moe_combine(cfg, s["y_perm"], s["slot_pos"], s["gates"], s["y"], s["ws"])
    return {"y": s["y"]}


# --------------------------------------------------------------------- what it takes

def work(case):
    """Bytes: every input and output once (of the experts' weights those that the rows can
    reach, a row at most one expert's); flops: 2 for each multiply-add of the products."""
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, d = case["rows"], case["d"]
        e = 2 if case["dtype"] == "bf16" else 4
        n = rows * d
        if op == "norm":
            b = n * e * (1 + 2 * case["residual"] + case["y"]) + rows * 4 + d * e
            b += case["q"] * (n + 4 * rows * _blocks(d))
            return {"bytes": b, "flops": 4 * n}
        return {"bytes": n * (e + 8 + 4 * case["residual"]) + rows * 4 + d * (e + 4), "flops": 10 * n}
    if op in ("linear", "grouped"):
        rows, n, k = case["rows"], case["n"], case["k"]
        groups = min(case.get("groups", 1), rows)
        a = rows * k * 2 if case.get("a") == "bf16" else rows * (k + 4 * _blocks(k))
        b = a + groups * (n * k + 4 * _blocks(n) * _blocks(k)) + rows * n * (2 if case["out"] == "bf16" else 4)
        return {"bytes": b, "flops": 2 * rows * n * k}
    tokens, d, f, k = (case[c] for c in ("tokens", "d", "f", "k"))
    rows = tokens * k
    experts = min(case["experts"], rows)
    b = tokens * (d + 4 * _blocks(d)) + experts * (2 * d * f + 8 * _blocks(d) * _blocks(f)) + rows * 12 + tokens * d * 2
    return {"bytes": b, "flops": 4 * rows * d * f}


# ------------------------------------------------------------ the definition, 64 bits

def _e4m3(v):
    """The nearest e4m3 value, ties to even: 3 bits behind the point from 2^-6 on, a fixed
    step of 2^-9 below."""
    exponent = torch.frexp(v.abs().clamp_min(2.0 ** -30))[1] - 1
    step = torch.ldexp(torch.ones_like(v), exponent.clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _quantised_exactly(y):
    rows, d = y.shape
    pad = torch.nn.functional.pad(y, (0, _blocks(d) * BLOCK - d)).unflatten(1, (-1, BLOCK))
    top = torch.clamp(pad.abs().max(dim=2).values, min=E4M3_MAX * TINY)
    return _e4m3(E4M3_MAX * pad / top.unsqueeze(2)).flatten(1)[:, :d], top / E4M3_MAX


def _value64(q, scale):
    """Rows' values in 64 bits; scale [rows, blocks]."""
    block = torch.arange(q.shape[1], device=q.device) // BLOCK
    return q.double() * scale.double()[:, block]


def _weights64(q, scale):
    i = torch.arange(q.shape[0], device=q.device) // BLOCK
    j = torch.arange(q.shape[1], device=q.device) // BLOCK
    return q.double() * scale.double()[i][:, j]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def by_group(rows, q, scale):
        out = rows.new_zeros(rows.shape[0], q.shape[1])
        at = s["offsets"].tolist()
        for e in range(q.shape[0]):
            if at[e + 1] > at[e]:
                out[at[e]:at[e + 1]] = rows[at[e]:at[e + 1]] @ _weights64(q[e], scale[e]).T
        return out

    if op == "norm":
        v, out = s["x"].double(), {}
        if case["residual"]:
            out["sum"] = v + s["residual"].double()
            v = out["sum"].to(s["x"].dtype).double()
        out["rstd"] = 1.0 / torch.sqrt((v * v).sum(1) / case["d"] + EPS)
        y = v * out["rstd"].unsqueeze(1) * s["weight"].double()
        if case["y"]:
            out["y"] = y
        if case["q"]:
            out["q"], scale = _quantised_exactly(y)
            out["scale"] = scale.T.contiguous()
        return out
    if op == "norm_grad":
        v, w, dy = s["x"].double(), s["weight"].double(), s["dy"].double()
        r = s["rstd"].double().unsqueeze(1)
        inner = (v * w * dy).sum(1, keepdim=True)
        dx = w * dy * r - v * r ** 3 * inner / case["d"]
        return {"dx": dx + s["dsum"].double() if case["residual"] else dx, "dweight": torch.einsum("td,td->d", dy, v * r)}
    if op == "linear":
        if case["a"] == "fp8":
            a = _value64(s["a"], s["a_scale"].T)
        else:
            a = _value64(*_quantised_exactly(s["x"].double()))
        return {"out": a @ _weights64(s["w"], s["w_scale"]).T}
    if op == "grouped":
        return {"out": by_group(_value64(s["a"], s["a_scale"].T), s["w"], s["w_scale"])}
    x = _value64(s["x"], s["x_scale"].T)[torch.div(s["perm_src"].long(), case["k"], rounding_mode="floor")]
    z = by_group(x, s["w1"], s["w1_scale"])
    h = torch.relu(z) if case["act"] == "relu" else z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    y_perm = by_group(_value64(*_quantised_exactly(h)), s["w2"], s["w2_scale"])
    y = torch.zeros(case["tokens"], case["d"], dtype=torch.float64, device=x.device)
    for j in range(case["k"]):
        y += s["gates"][:, j:j + 1].double() * y_perm[s["slot_pos"].view(-1, case["k"])[:, j].long()]
    return {"y": y}
