"""Cases of the feed-forward operators around the expert layer: layer norm and its gradient, the
gated block with its backward products, and products in 8-bit floating point with a scale for
each block of 128.

Each case is one call a training or serving program makes.  `run` computes it either in
plain torch operations in 32 bits, or (where `own` is true) with the library's entry points.
`exact` computes it again from its definition in 64 bits.

Rows are sorted by expert: expert e owns rows offsets[e] .. offsets[e+1] - 1, with the
offsets on the device, as a router leaves them.  A dense case has one weight and no offsets.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
E4M3 = torch.float8_e4m3fn
BLOCK = 128      # elements that share a scale
EPS = 1e-5

# The most work a drawn case may have: below the largest listed one.
MOST_FLOPS = 4.0e11
MOST_BYTES = 1.5e9


def listed():
    return [
        # A decoding batch in front of a layer: latency.
        dict(name="norm decode", op="norm", rows=32, cols=4096, dtype="bf16", keep=False),
        # A training step's rows, with the statistics that the backward pass takes.
        dict(name="norm train", op="norm", rows=16384, cols=4096, dtype="bf16", keep=True),
        # A small model in 32 bits with odd sizes, its weight gradients added to what the flat
        # buffer holds.
        dict(name="norm grad odd", op="norm_grad", rows=2005, cols=771, dtype="fp32", accumulate=True),
        # The backward pass of a training step.
        dict(name="norm grad train", op="norm_grad", rows=16384, cols=4096, dtype="bf16",
             accumulate=False),
        # A decoding batch of 32 tokens, each sent to 6 of 64 experts: weight reads.
        dict(name="gated decode", op="gated", tokens=32, top=6, experts=64, k=2048, n=1408, dense=False,
             trans=False, dtype="bf16", weighted=True, keep=False, skew=0.4),
        # A dense feed-forward layer in training, weights stored (out, in), both projections kept.
        dict(name="gated dense train", op="gated", tokens=4096, top=1, experts=1, k=4096, n=14336,
             dense=True, trans=True, dtype="bf16", weighted=False, keep=True, skew=0.0),
        # Backward through the down projection and the activation over a long batch, with the
        # gradient of the router's weights.
        dict(name="gated grad train", op="gated_grad", tokens=16384, top=6, experts=64, k=2048, n=1408,
             dense=False, trans=True, dtype="bf16", weighted=True, skew=0.4),
        # Backward through both projections to the layer's input (an odd number of rows).
        dict(name="input grad train", op="mm_sum", tokens=4095, top=6, experts=64, k=1408, n=2048,
             dense=False, trans=True, dtype="bf16", out="bf16", skew=0.4),
        # Activations of a training step on their way into an 8-bit product.
        dict(name="quantize rows", op="quantize_rows", rows=24570, cols=2048, dtype="bf16"),
        # The experts' weights after a step, turned so that the product reads along its sum.
        dict(name="quantize weights", op="quantize_weights", experts=64, m=2048, n=1408, dtype="bf16",
             transpose=True),
        # A decoding batch through the down projections in 8 bits.
        dict(name="fp8 decode", op="mm_fp8", tokens=32, top=6, experts=64, k=1408, n=2048, out="bf16",
             skew=0.4),
        # A long batch through them.
        dict(name="fp8 train", op="mm_fp8", tokens=16384, top=6, experts=64, k=1408, n=2048, out="bf16",
             skew=0.4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "gated", "gated", "gated_grad", "mm_sum", "quantize_rows",
                     "quantize_weights", "mm_fp8", "mm_fp8"])
    if op in ("norm", "norm_grad", "quantize_rows"):
        cols = _log(rng, 8, 16384)
        rows = max(1, min(_log(rng, 1, 65536), 80_000_000 // cols))
        case = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
        if op == "norm":
            case["keep"] = rng.random() < 0.5
        elif op == "norm_grad":
            case["accumulate"] = rng.random() < 0.5
        return case
    dense = op in ("gated", "gated_grad", "mm_sum") and rng.random() < 0.3
    experts = 1 if dense else _log(rng, 1, 128)
    # multiples of 16 most of the time, odd sizes otherwise
    step = rng.choice([16, 16, 16, 1])
    a, b = (max(step, _log(rng, 16, 6144) // step * step) for _ in range(2))
    if op == "quantize_weights":
        case = dict(op=op, experts=experts, m=a, n=b, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    transpose=rng.random() < 0.5)
        while work(case)["bytes"] > MOST_BYTES:
            case["experts"] = max(1, case["experts"] // 2)
        return case
    case = dict(op=op, tokens=_log(rng, 1, 16384), top=rng.randint(1, min(8, experts)), experts=experts,
                k=a, n=b, skew=rng.choice([0.0, 0.4, 1.0]))
    if op == "mm_fp8":
        case["out"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    else:
        case.update(dense=dense, trans=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "mm_sum":
        case["out"] = rng.choice([case["dtype"], case["dtype"], "fp32"])
    elif op != "mm_fp8":
        case["weighted"] = rng.random() < 0.6
    if op == "gated":
        case["keep"] = rng.random() < 0.6
    while work(case)["flops"] > MOST_FLOPS or work(case)["bytes"] > MOST_BYTES:
        if case["tokens"] > 1 and work(dict(case, tokens=1))["bytes"] < MOST_BYTES / 2:
            case["tokens"] = max(1, case["tokens"] * 2 // 3)
        else:
            case["experts"] = max(case["top"], case["experts"] * 2 // 3)
            case["n"] = max(step, case["n"] * 2 // 3 // step * step)
    return case


def _rows(case):
    return case["tokens"] * case["top"]


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _sizes(case, seed):
    """Rows of each expert: every token's `top` experts by its own noisy scores."""
    rng = np.random.default_rng([seed, 21])
    e = case["experts"]
    score = case["skew"] * rng.normal(size=e) + rng.gumbel(size=(case["tokens"], e))
    pick = np.argpartition(-score, case["top"] - 1, axis=1)[:, : case["top"]]
    return np.bincount(pick.reshape(-1), minlength=e).astype(np.int64)


def _scale(amax):
    """The smallest power of two s with amax / s <= 448, the largest e4m3 value (1 for zeros)."""
    m, e = torch.frexp(amax)                       # amax = m 2^e with m in [1/2, 1); 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126)
    return torch.where(amax > 0, ((e + 127) << 23).to(torch.int32).view(torch.float32),
                       torch.ones_like(amax))


def _padded(t, *dims):
    """t with zeros behind the ends of the given dimensions, up to whole blocks."""
    pad = [0, 0] * t.dim()
    for d in dims:
        pad[2 * (t.dim() - 1 - d) + 1] = -t.shape[d] % BLOCK
    return torch.nn.functional.pad(t, pad)


def _quantize_rows(x):
    """(values / scale in e4m3, scales (blocks of columns, rows))"""
    rows, cols = x.shape
    b = _padded(x.float(), 1).view(rows, -1, BLOCK)
    s = _scale(b.abs().amax(2))
    return (b / s[:, :, None]).view(rows, -1)[:, :cols].to(E4M3), s.T.contiguous()


def _quantize_weights(w, transpose):
    """(values / scale in e4m3, scales (experts, blocks of rows, blocks of columns))"""
    w = w.float().transpose(1, 2) if transpose else w.float()
    e, m, n = w.shape
    b = _padded(w, 1, 2).view(e, _blocks(m), BLOCK, _blocks(n), BLOCK)
    s = _scale(b.abs().amax((2, 4)))
    return ((b / s[:, :, None, :, None]).view(e, _blocks(m) * BLOCK, -1)[:, :m, :n].to(E4M3).contiguous(),
            s)


def _on_16_bytes(q):
    """q with rows that start on 16 bytes."""
    cols = q.shape[-1]
    if cols % 16 == 0:
        return q.contiguous()
    room = torch.zeros(*q.shape[:-1], cols + -cols % 16, dtype=torch.uint8, device=q.device)
    room[..., :cols] = q.view(torch.uint8)
    return room.view(E4M3)[..., :cols]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 29)

    def normal(*shape, std=1.0, dtype="fp32"):
        return torch.randn(shape, generator=gen, device=dev).mul_(std).to(TYPES[dtype])

    op, st = case["op"], dict(case)
    if op in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        # a residual stream: columns with means and sizes of their own
        x = normal(rows, cols) * torch.exp(0.5 * normal(cols)) + 0.5 * normal(cols)
        st["x"] = x.to(TYPES[case["dtype"]])
        st["w"], st["b"] = 1.0 + 0.1 * normal(cols), 0.1 * normal(cols)
        if op == "norm_grad":
            st["dy"] = normal(rows, cols, std=0.1, dtype=case["dtype"])
            xd = st["x"].double()
            var, mean = torch.var_mean(xd, 1, correction=0)
            st["mean"], st["rstd"] = mean.float(), (var + EPS).rsqrt().float()
            st["dw"], st["db"] = normal(cols), normal(cols)
        return st
    if op == "quantize_rows":
        st["x"] = normal(case["rows"], case["cols"], dtype=case["dtype"])
        return st
    if op == "quantize_weights":
        st["w"] = normal(case["experts"], case["m"], case["n"], std=0.02, dtype=case["dtype"])
        return st
    rows, e, k, n = _rows(case), case["experts"], case["k"], case["n"]
    sizes = _sizes(case, seed)
    st["sizes"] = [int(v) for v in sizes]
    st["offsets"] = None if case.get("dense") else \
        torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)])).to(dev)
    if op == "mm_fp8":
        q, st["xs"] = _quantize_rows(normal(rows, k))
        st["x"] = _on_16_bytes(q)
        parts = [_quantize_weights(normal(1, n, k, std=0.02), False) for _ in range(e)]
        st["w"] = _on_16_bytes(torch.cat([q.view(torch.uint8) for q, _ in parts]).view(E4M3))
        st["ws"] = torch.cat([s for _, s in parts])
        return st

    def weights():
        return torch.stack([normal(*((n, k) if case["trans"] else (k, n)), std=0.02, dtype=case["dtype"])
                            for _ in range(e)])

    st["p"] = torch.rand(rows, generator=gen, device=dev) if case.get("weighted") else None
    if op == "gated":
        st["x"] = normal(rows, k, dtype=case["dtype"])
        st["wg"], st["wu"] = weights(), weights()
    elif op == "gated_grad":
        st["dy"] = normal(rows, k, std=0.1, dtype=case["dtype"])
        st["wd"] = weights()
        st["g"], st["u"] = normal(rows, n, dtype=case["dtype"]), normal(rows, n, dtype=case["dtype"])
    else:
        st["xa"], st["xb"] = (normal(rows, k, std=0.1, dtype=case["dtype"]) for _ in range(2))
        st["wa"], st["wb"] = weights(), weights()
    return st


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _product(x, w, s):
    """Every expert's product in 32 bits (w in the order that s["trans"] says)."""
    return torch.cat([a.float() @ (b.float().T if s["trans"] else b.float())
                      for a, b in zip(x.split(s["sizes"]), w) if len(a)])


def _run_plain(s):
    op = s["op"]
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1)
        x = x - mean[:, None]
        rstd = (x.square().mean(1) + EPS).rsqrt()
        y = (x * rstd[:, None] * s["w"] + s["b"]).to(s["x"].dtype)
        return {"y": y, "mean": mean, "rstd": rstd} if s["keep"] else {"y": y}
    if op == "norm_grad":
        dy = s["dy"].float()
        xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        t = dy * s["w"]
        dx = s["rstd"][:, None] * (t - t.mean(1)[:, None] - xh * (t * xh).mean(1)[:, None])
        dw, db = (dy * xh).sum(0), dy.sum(0)
        if s["accumulate"]:
            dw, db = s["dw"].add_(dw), s["db"].add_(db)
        return {"dx": dx.to(s["x"].dtype), "dw": dw, "db": db}
    if op == "gated":
        g, u = _product(s["x"], s["wg"], s), _product(s["x"], s["wu"], s)
        out = g * torch.sigmoid(g) * u
        if s["weighted"]:
            out = out * s["p"][:, None]
        t = s["x"].dtype
        return {"out": out.to(t), "gate": g.to(t), "up": u.to(t)} if s["keep"] else {"out": out.to(t)}
    if op == "gated_grad":
        g, u, dh = s["g"].float(), s["u"].float(), _product(s["dy"], s["wd"], s)
        sig = torch.sigmoid(g)
        silu = g * sig
        out = silu * u
        dp = (dh * out).sum(1) if s["weighted"] else None
        if s["weighted"]:
            dh, out = dh * s["p"][:, None], out * s["p"][:, None]
        t = s["g"].dtype
        return {"dgate": (dh * u * sig * (1 + g * (1 - sig))).to(t), "dup": (dh * silu).to(t),
                "out": out.to(t), "dp": dp}
    if op == "mm_sum":
        return {"y": (_product(s["xa"], s["wa"], s) + _product(s["xb"], s["wb"], s)).to(TYPES[s["out"]])}
    if op == "quantize_rows":
        q, scale = _quantize_rows(s["x"])
        return {"q": q, "scale": scale}
    if op == "quantize_weights":
        q, scale = _quantize_weights(s["w"], s["transpose"])
        return {"q": q, "scale": scale}
    n, k = s["n"], s["k"]
    x = s["x"].float() * s["xs"].T.repeat_interleave(BLOCK, 1)[:, :k]
    scale = s["ws"].repeat_interleave(BLOCK, 1)[:, :n]
    return {"y": torch.cat([a @ (w.float() * c.repeat_interleave(BLOCK, 1)[:, :k]).T
                            for a, w, c in zip(x.split(s["sizes"]), s["w"], scale) if len(a)]
                           ).to(TYPES[s["out"]])}


def _run_own(s):
    from muon_optimizer_step_gb300 import capi
    op = s["op"]
    if op == "norm":
        x, y = s["x"], torch.empty_like(s["x"])
        mean, rstd = (torch.empty(2, len(x), device=x.device) if s["keep"] else (None, None))
        capi.muon_layer_norm(x, s["w"], s["b"], y, mean=mean, rstd=rstd, eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd} if s["keep"] else {"y": y}
    if op == "norm_grad":
        dx = torch.empty_like(s["x"])
        dw, db = (s["dw"], s["db"]) if s["accumulate"] else \
            (torch.empty_like(s["dw"]), torch.empty_like(s["db"]))
        capi.muon_layer_norm_grad(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], dx, dw, db,
                                  accumulate=s["accumulate"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "quantize_rows":
        x = s["x"]
        q = torch.empty(x.shape, dtype=E4M3, device=x.device)
        scale = torch.empty(_blocks(s["cols"]), s["rows"], device=x.device)
        capi.muon_quantize_rows(x, q, scale)
        return {"q": q, "scale": scale}
    if op == "quantize_weights":
        w = s["w"]
        e, m, n = w.shape
        if s["transpose"]:
            m, n = n, m
        q = torch.empty(e, m, n, dtype=E4M3, device=w.device)
        scale = torch.empty(e, _blocks(m), _blocks(n), device=w.device)
        capi.muon_quantize_weights(w, q, scale, transpose=s["transpose"])
        return {"q": q, "scale": scale}
    rows = s["tokens"] * s["top"]
    if op == "mm_fp8":
        y = torch.empty(rows, s["n"], dtype=TYPES[s["out"]], device=s["x"].device)
        capi.muon_grouped_mm_fp8(s["x"], s["xs"], s["w"], s["ws"], s["offsets"], y)
        return {"y": y}
    if op == "mm_sum":
        y = torch.empty(rows, s["n"], dtype=TYPES[s["out"]], device=s["xa"].device)
        capi.muon_grouped_mm_sum(s["xa"], s["wa"], s["xb"], s["wb"], s["offsets"], y, trans_w=s["trans"])
        return {"y": y}
    t = TYPES[s["dtype"]]

    def new():
        return torch.empty(rows, s["n"], dtype=t, device="cuda")

    if op == "gated":
        out = new()
        gate, up = (new(), new()) if s["keep"] else (None, None)
        capi.muon_gated_mm(s["x"], s["wg"], s["wu"], s["offsets"], out, gate=gate, up=up,
                           row_weight=s["p"], trans_w=s["trans"])
        return {"out": out, "gate": gate, "up": up} if s["keep"] else {"out": out}
    dgate, dup, out = new(), new(), new()
    dp = torch.empty_like(s["p"]) if s["weighted"] else None
    capi.muon_gated_mm_grad(s["dy"], s["wd"], s["offsets"], s["g"], s["u"], dgate, dup, out=out,
                            row_weight=s["p"], d_row_weight=dp, trans_w=s["trans"])
    return {"dgate": dgate, "dup": dup, "out": out, "dp": dp}


def _edges(s):
    return np.concatenate([[0], np.cumsum(s["sizes"])])


def _exact_product(x, w, s):
    edge = _edges(s)
    y = torch.empty(x.shape[0], s["n"], dtype=torch.float64, device=x.device)
    for e in np.flatnonzero(np.diff(edge)):
        rows = slice(edge[e], edge[e + 1])
        y[rows] = torch.einsum("rk,nk->rn" if s["trans"] else "rk,kn->rn", x[rows].double(), w[e].double())
    return y


def _power(e):
    """2^e in 64 bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_scale(amax):
    """From a power that is surely too small, up while the largest magnitude does not fit."""
    e = torch.floor(torch.log2(amax.clamp(min=1e-300) / 448.0)).clamp(min=-125) - 1
    for _ in range(3):
        e = torch.where(amax > 448.0 * _power(e), e + 1, e)
    return torch.where(amax > 0, _power(e), torch.ones_like(amax))


def _e4m3(v):
    """v (64 bits) rounded to 3 fraction bits, ties to even, smallest exponent -6."""
    size = v.abs().clamp(min=2.0 ** -6)
    e = torch.floor(torch.log2(size))
    e = torch.where(_power(e) > size, e - 1, e)
    step = _power(e - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = torch.addcmul(s["b"].double(), (x - mean[:, None]) * rstd[:, None], s["w"].double())
        return {"y": y, "mean": mean, "rstd": rstd} if case["keep"] else {"y": y}
    if op == "norm_grad":
        x, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
        mean, rstd = s["mean"].double(), s["rstd"].double()
        xh = torch.einsum("rc,r->rc", x - mean[:, None], rstd)
        cols = case["cols"]
        first = torch.einsum("rc,c->r", dy, w) / cols
        second = torch.einsum("rc,c,rc->r", dy, w, xh) / cols
        dx = torch.einsum("rc,r->rc", dy * w - first[:, None] - xh * second[:, None], rstd)
        old = 1.0 if case["accumulate"] else 0.0
        return {"dx": dx, "dw": torch.einsum("rc,rc->c", dy, xh) + old * s["dw"].double(),
                "db": torch.einsum("rc->c", dy) + old * s["db"].double()}
    if op == "gated":
        g, u = _exact_product(s["x"], s["wg"], s), _exact_product(s["x"], s["wu"], s)
        out = g / (1.0 + torch.exp(-g)) * u
        if case["weighted"]:
            out *= s["p"].double()[:, None]
        return {"out": out, "gate": g, "up": u} if case["keep"] else {"out": out}
    if op == "gated_grad":
        dh = _exact_product(s["dy"], s["wd"], s)
        g, u = s["g"].double(), s["u"].double()
        p = s["p"].double()[:, None] if case["weighted"] else 1.0
        z = torch.exp(-g)
        silu = g / (1.0 + z)
        return {"dgate": dh * p * u * (1.0 + z + g * z) / (1.0 + z) ** 2, "dup": dh * p * silu,
                "out": p * silu * u,
                "dp": torch.einsum("rc,rc,rc->r", dh, silu, u) if case["weighted"] else None}
    if op == "mm_sum":
        return {"y": _exact_product(s["xa"], s["wa"], s) + _exact_product(s["xb"], s["wb"], s)}
    if op in ("quantize_rows", "quantize_weights"):
        if op == "quantize_rows":
            t = s["x"].double()[None]
            high, wide = 1, BLOCK
        else:
            t = s["w"].double()
            t = t.transpose(1, 2) if case["transpose"] else t
            high, wide = BLOCK, BLOCK
        e, m, n = t.shape
        mb, nb = -(-m // high), -(-n // wide)
        room = torch.zeros(e, mb * high, nb * wide, dtype=torch.float64, device=t.device)
        room[:, :m, :n] = t
        amax = room.view(e, mb, high, nb, wide).abs().amax((2, 4))
        scale = _exact_scale(amax)
        spread = scale.repeat_interleave(high, 1)[:, :m].repeat_interleave(wide, 2)[:, :, :n]
        q = _e4m3(t / spread)
        if op == "quantize_rows":
            return {"q": q[0], "scale": scale[0].T}
        return {"q": q, "scale": scale}
    y = torch.empty(_rows(case), case["n"], dtype=torch.float64, device="cuda")
    edge, k, n = _edges(s), case["k"], case["n"]
    for e in np.flatnonzero(np.diff(edge)):
        rows = slice(edge[e], edge[e + 1])
        sums = 0.0
        for b in range(_blocks(k)):
            at = slice(b * BLOCK, min(k, (b + 1) * BLOCK))
            part = torch.einsum("rk,nk->rn", s["x"][rows, at].double(), s["w"][e][:, at].double())
            column = s["ws"][e, torch.arange(n, device="cuda") // BLOCK, b].double()
            sums = sums + part * s["xs"][b, rows].double()[:, None] * column
        y[rows] = sums
    return {"y": y}


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad", "quantize_rows"):
        rows, cols, b = case["rows"], case["cols"], BYTES[case["dtype"]]
        if op == "norm":
            return {"bytes": rows * cols * 2 * b + 8 * cols + (8 * rows if case["keep"] else 0),
                    "flops": 8.0 * rows * cols}
        if op == "norm_grad":
            return {"bytes": rows * cols * 3 * b + 8 * rows + cols * (20 if case["accumulate"] else 12),
                    "flops": 15.0 * rows * cols}
        return {"bytes": rows * (cols * (b + 1) + 4 * _blocks(cols)), "flops": 3.0 * rows * cols}
    if op == "quantize_weights":
        e, m, n = case["experts"], case["m"], case["n"]
        return {"bytes": e * (m * n * (BYTES[case["dtype"]] + 1) + 4 * _blocks(m) * _blocks(n)),
                "flops": 3.0 * e * m * n}
    rows, e, k, n = _rows(case), case["experts"], case["k"], case["n"]
    hit = e * (1.0 - (1.0 - case["top"] / e) ** case["tokens"])  # experts with rows
    offsets = 0 if case.get("dense") else 8 * (e + 1)
    if op == "mm_fp8":
        return {"bytes": rows * (k + 4 * _blocks(k) + n * BYTES[case["out"]]) + offsets
                + hit * (k * n + 4 * _blocks(k) * _blocks(n)), "flops": 2.0 * rows * k * n}
    b = BYTES[case["dtype"]]
    if op == "gated":
        return {"bytes": rows * (k * b + n * b * (3 if case["keep"] else 1) + (4 if case["weighted"] else 0))
                + 2 * hit * k * n * b + offsets, "flops": 4.0 * rows * k * n}
    if op == "gated_grad":
        return {"bytes": rows * (k * b + 5 * n * b + (8 if case["weighted"] else 0)) + hit * k * n * b
                + offsets, "flops": 2.0 * rows * k * n}
    return {"bytes": rows * (2 * k * b + n * BYTES[case["out"]]) + 2 * hit * k * n * b + offsets,
            "flops": 4.0 * rows * k * n}
