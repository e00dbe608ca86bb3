"""Cases of the expert-layer operators: the products grouped by expert, the gated activation
between them, and the global gradient norm with clipping.

Each case is one call a training or serving program makes.  `run` computes it either in
plain torch operations in 32 bits, or (where `own` is true) with the library's entry points.
`exact` computes it again from its definition in 64 bits.

Rows are sorted by expert: expert e owns rows offsets[e] .. offsets[e+1] - 1, with the
offsets on the device, as a router leaves them.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}

# Parameter lists of this repository's workloads (elements of each tensor).
TENSORS = {
    "ragged_small": (300 * 200, 37, 130 * 520, 200 * 200, 50, 21, 64 * 1000, 257 * 129, 1, 384 * 256),
    "moe_64e": (2048 * 1408,) * 192 + (2048 * 2048,) * 4,
}

# The most work a drawn case may have: below the largest listed one.
MOST_FLOPS = 5.0e11
MOST_BYTES = 5.0e9


def listed():
    return [
        # One token of a serving batch, sent to 6 of 64 experts: latency and weight reads.
        dict(name="mm single token", op="mm", tokens=1, top=6, experts=64, k=2048, n=1408,
             trans=False, dtype="bf16", out="bf16", skew=0.4),
        # A decoding batch of 32 tokens through the down projections.
        dict(name="mm decode batch", op="mm", tokens=32, top=6, experts=64, k=1408, n=2048,
             trans=False, dtype="bf16", out="bf16", skew=0.4),
        # A training step's gate projection (an odd number of rows).
        dict(name="mm train gate", op="mm", tokens=4095, top=6, experts=64, k=2048, n=1408,
             trans=False, dtype="bf16", out="bf16", skew=0.4),
        # The gradient with respect to its input over a long batch: the stored weight read
        # along its other axis.
        dict(name="mm grad input", op="mm", tokens=16384, top=6, experts=64, k=1408, n=2048,
             trans=True, dtype="bf16", out="bf16", skew=0.4),
        # Few large experts whose weights are stored (out, in).
        dict(name="mm wide experts", op="mm", tokens=2048, top=2, experts=8, k=4096, n=14336,
             trans=True, dtype="bf16", out="bf16", skew=0.4),
        # Odd sizes whose rows do not start on 16 bytes, half precision, result in 32 bits.
        dict(name="mm odd", op="mm", tokens=1003, top=1, experts=7, k=771, n=517,
             trans=False, dtype="fp16", out="fp32", skew=1.0),
        # Weight gradients of small ragged experts, added to what the buffer holds (a later
        # micro-batch).
        dict(name="wgrad odd", op="wgrad", tokens=2005, top=1, experts=13, m=130, n=520,
             dtype="fp16", accumulate=True, skew=1.0),
        # Weight gradients of a training step, written where the optimizer reads them.
        dict(name="wgrad train", op="wgrad", tokens=16384, top=6, experts=64, m=2048, n=1408,
             dtype="bf16", accumulate=False, skew=0.4),
        # The activation of a decoding batch, with the router's weight of each row.
        dict(name="swiglu decode", op="swiglu", rows=192, cols=1408, dtype="bf16", weighted=True),
        # Its gradient in training, with the gradient of the router's weights.
        dict(name="swiglu grad train", op="swiglu_grad", rows=98304, cols=1408, dtype="bf16",
             weighted=True),
        # Clipping a small model's ten gradients (odd starts, a single element).
        dict(name="clip small", op="clip", tensors="ragged_small", count=0, numel=0, dtype="fp32",
             max_norm=1.0),
        # Clipping the 196 gradients of the mixture-of-experts set into the flat buffer.
        dict(name="clip experts", op="clip", tensors="moe_64e", count=0, numel=0, dtype="fp32",
             max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mm", "mm", "wgrad", "wgrad", "swiglu", "swiglu_grad", "clip"])
    if op in ("mm", "wgrad"):
        experts = _log(rng, 1, 128)
        top = rng.randint(1, min(8, experts))
        case = dict(op=op, tokens=_log(rng, 1, 16384), top=top, experts=experts,
                    dtype=rng.choice(["bf16", "bf16", "fp16"]), skew=rng.choice([0.0, 0.4, 1.0]))
        # multiples of 8 (rows that start on 16 bytes) most of the time, odd sizes otherwise
        step = rng.choice([8, 8, 8, 1])
        a, b = (max(step, _log(rng, 16, 6144) // step * step) for _ in range(2))
        if op == "mm":
            case.update(k=a, n=b, trans=rng.random() < 0.5,
                        out=rng.choice([case["dtype"], case["dtype"], "fp32"]))
        else:
            case.update(m=a, n=b, accumulate=rng.random() < 0.5)
        while work(case)["flops"] > MOST_FLOPS or work(case)["bytes"] > MOST_BYTES:
            if case["tokens"] > 1 and work(dict(case, tokens=1))["bytes"] < MOST_BYTES / 2:
                case["tokens"] = max(1, case["tokens"] * 2 // 3)
            else:
                case["experts"] = max(case["top"], case["experts"] * 2 // 3)
                case["n"] = max(step, case["n"] * 2 // 3 // step * step)
        return case
    if op in ("swiglu", "swiglu_grad"):
        cols = _log(rng, 8, 16384)
        return dict(op=op, rows=max(1, min(_log(rng, 1, 98304), 140_000_000 // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), weighted=rng.random() < 0.7)
    return dict(op="clip", tensors="", count=_log(rng, 1, 512), numel=_log(rng, 1000, 400_000_000),
                dtype=rng.choice(["fp32", "fp32", "bf16"]), max_norm=rng.choice([0.5, 1.0, 1e6]))


def _rows(case):
    return case["tokens"] * case["top"]


def _sizes(case, seed):
    """Rows of each expert: every token's `top` experts by its own noisy scores."""
    rng = np.random.default_rng([seed, 11])
    e = case["experts"]
    score = case["skew"] * rng.normal(size=e) + rng.gumbel(size=(case["tokens"], e))
    pick = np.argpartition(-score, case["top"] - 1, axis=1)[:, : case["top"]]
    return np.bincount(pick.reshape(-1), minlength=e).astype(np.int64)


def _numels(case, seed):
    if case["tensors"]:
        return list(TENSORS[case["tensors"]])
    # vectors and matrices of a model: sizes spread over their logarithm, `numel` in all
    share = np.exp(np.random.default_rng([seed, 12]).uniform(0.0, 7.0, case["count"]))
    return [max(1, int(v)) for v in share / share.sum() * case["numel"]]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 13)

    def normal(*shape, std=1.0, dtype="fp32"):
        return torch.randn(shape, generator=gen, device=dev).mul_(std).to(TYPES[dtype])

    op, st = case["op"], dict(case)
    if op in ("mm", "wgrad"):
        sizes = _sizes(case, seed)
        st["sizes"] = [int(v) for v in sizes]
        st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)])).to(dev)
    if op == "mm":
        e, k, n = case["experts"], case["k"], case["n"]
        st["x"] = normal(_rows(case), k, dtype=case["dtype"])
        w = [normal(*((n, k) if case["trans"] else (k, n)), std=0.02, dtype=case["dtype"])
             for _ in range(e)]
        st["w"] = torch.stack(w)
    elif op == "wgrad":
        st["a"] = normal(_rows(case), case["m"], dtype=case["dtype"])
        st["b"] = normal(_rows(case), case["n"], std=0.1, dtype=case["dtype"])
        shape = (case["experts"], case["m"], case["n"])
        st["dw"] = normal(*shape) if case["accumulate"] else torch.zeros(shape, device=dev)
    elif op in ("swiglu", "swiglu_grad"):
        shape = (case["rows"], case["cols"])
        st["g"], st["u"] = normal(*shape, dtype=case["dtype"]), normal(*shape, dtype=case["dtype"])
        st["p"] = torch.rand(case["rows"], generator=gen, device=dev) if case["weighted"] else None
        if op == "swiglu_grad":
            st["da"] = normal(*shape, std=0.1, dtype=case["dtype"])
    else:
        numels = _numels(case, seed)
        flat = normal(sum(numels), std=1e-3, dtype=case["dtype"])
        st["grads"] = list(flat.split(numels))
        scale = np.exp(np.random.default_rng([seed, 13]).normal(size=len(numels)))
        for g, s in zip(st["grads"], scale):
            g.mul_(float(s))
        st["out"] = torch.zeros(sum(numels), device=dev)
        st["outs"] = list(st["out"].split(numels))
    return st


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    op = s["op"]
    if op == "mm":
        return {"y": torch.cat([x.float() @ (w.float().T if s["trans"] else w.float())
                                for x, w in zip(s["x"].split(s["sizes"]), s["w"]) if len(x)]
                               ).to(TYPES[s["out"]])}
    if op == "wgrad":
        dw = torch.stack([a.float().T @ b.float()
                          for a, b in zip(s["a"].split(s["sizes"]), s["b"].split(s["sizes"]))])
        if s["accumulate"]:
            dw = s["dw"].add_(dw)
        return {"dw": dw}
    if op == "swiglu":
        g, u = s["g"].float(), s["u"].float()
        a = g * torch.sigmoid(g) * u
        if s["weighted"]:
            a = a * s["p"][:, None]
        return {"a": a.to(s["g"].dtype)}
    if op == "swiglu_grad":
        g, u, da = s["g"].float(), s["u"].float(), s["da"].float()
        sig = torch.sigmoid(g)
        silu = g * sig
        dp = (da * silu * u).sum(1) if s["weighted"] else None
        if s["weighted"]:
            da = da * s["p"][:, None]
        return {"dg": (da * u * sig * (1 + g * (1 - sig))).to(s["g"].dtype),
                "du": (da * silu).to(s["g"].dtype), "dp": dp}
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    torch.cat([g.float() * coef for g in s["grads"]], out=s["out"])
    return {"norm": torch.stack([norm, coef]), "clipped": s["out"]}


def _run_own(s):
    from muon_optimizer_step_gb300 import capi
    op = s["op"]
    if op == "mm":
        y = torch.empty(s["x"].shape[0], s["n"], dtype=TYPES[s["out"]], device=s["x"].device)
        capi.muon_grouped_mm(s["x"], s["w"], s["offsets"], y, trans_w=s["trans"])
        return {"y": y}
    if op == "wgrad":
        dw = s["dw"] if s["accumulate"] else torch.empty_like(s["dw"])
        capi.muon_grouped_wgrad(s["a"], s["b"], s["offsets"], dw, accumulate=s["accumulate"])
        return {"dw": dw}
    if op == "swiglu":
        a = torch.empty_like(s["g"])
        capi.muon_swiglu(s["g"], s["u"], a, row_weight=s["p"])
        return {"a": a}
    if op == "swiglu_grad":
        dg, du = torch.empty_like(s["g"]), torch.empty_like(s["u"])
        dp = torch.empty_like(s["p"]) if s["weighted"] else None
        capi.muon_swiglu_grad(s["da"], s["g"], s["u"], dg, du, row_weight=s["p"], d_row_weight=dp)
        return {"dg": dg, "du": du, "dp": dp}
    norm = torch.empty(2, device=s["out"].device)
    capi.muon_clip_grads(s["grads"], s["outs"], s["max_norm"], norm)
    return {"norm": norm, "clipped": s["out"]}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "mm":
        y = torch.empty(s["x"].shape[0], case["n"], dtype=torch.float64, device=s["x"].device)
        edge = np.concatenate([[0], np.cumsum(s["sizes"])])
        for e in np.flatnonzero(np.diff(edge)):
            w = s["w"][e].double()
            y[edge[e]:edge[e + 1]] = torch.einsum("rk,nk->rn" if case["trans"] else "rk,kn->rn",
                                                  s["x"][edge[e]:edge[e + 1]].double(), w)
        return {"y": y}
    if op == "wgrad":
        dw = s["dw"].double()
        row = 0
        for e, size in enumerate(s["sizes"]):
            dw[e] += torch.einsum("rm,rn->mn", s["a"][row:row + size].double(),
                                  s["b"][row:row + size].double())
            row += size
        return {"dw": dw}
    if op in ("swiglu", "swiglu_grad"):
        rows = case["rows"]
        p = torch.ones(rows, dtype=torch.float64, device="cuda")
        if case["weighted"]:
            p = s["p"].double()
        g, u = s["g"].double(), s["u"].double()
        z = torch.exp(-g)
        silu = g / (1 + z)
        if op == "swiglu":
            return {"a": p[:, None] * silu * u}
        da = s["da"].double()
        slope = (1 + z + g * z) / (1 + z) ** 2
        return {"dg": da * p[:, None] * u * slope, "du": da * p[:, None] * silu,
                "dp": torch.einsum("rc,rc,rc->r", da, silu, u) if case["weighted"] else None}
    flat = torch.cat([g.double() for g in s["grads"]])
    norm = torch.linalg.vector_norm(flat)
    coef = torch.minimum(torch.ones_like(norm), case["max_norm"] / (norm + 1e-6))
    return {"norm": torch.stack([norm, coef]), "clipped": flat * coef}


def work(case):
    op = case["op"]
    if op in ("mm", "wgrad"):
        rows, e, b = _rows(case), case["experts"], BYTES[case["dtype"]]
        if op == "mm":
            k, n = case["k"], case["n"]
            hit = e * (1.0 - (1.0 - case["top"] / e) ** case["tokens"])  # experts with rows
            return {"bytes": rows * (k * b + n * BYTES[case["out"]]) + hit * k * n * b + 8 * (e + 1),
                    "flops": 2.0 * rows * k * n}
        m, n = case["m"], case["n"]
        return {"bytes": rows * (m + n) * b + e * m * n * (8 if case["accumulate"] else 4) + 8 * (e + 1),
                "flops": 2.0 * rows * m * n}
    if op in ("swiglu", "swiglu_grad"):
        rows, cols, b = case["rows"], case["cols"], BYTES[case["dtype"]]
        moved, per_row = (3, 4) if op == "swiglu" else (5, 8)
        return {"bytes": rows * cols * b * moved + (rows * per_row if case["weighted"] else 0),
                "flops": rows * cols * (6.0 if op == "swiglu" else 14.0)}
    numel = sum(TENSORS[case["tensors"]]) if case["tensors"] else case["numel"]
    return {"bytes": numel * (BYTES[case["dtype"]] + 4.0) + 8, "flops": 3.0 * numel}
