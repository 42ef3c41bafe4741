"""Timed cases of the operators around the projector's training step.

Five operators, each as a plain formula in elementary torch operations and as the call a
user makes of this package:

  lookup    rows of the token-embedding table, scaled, into the embedding sequence; rows of
            the image placeholder stay as they were
  scatter   the gradient of that table: rows of the sequence's gradient summed by token
  ln        layer norm over the last axis, with the statistics its backward pass reads
  ln_grad   its gradients with respect to the input, the weight and the bias
  clip      the global norm over many gradient tensors, and the clipped gradients

A case is a dict of plain values; ``listed`` names twelve, ``draw`` makes more of the same
ranges. ``run`` is one pass of the operator a case names.
"""
import math

import numpy as np
import torch

own = False

IMAGE_TOKEN = 100015
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one decoding step of 32 sequences: a handful of rows out of a table of a gigabyte
        {"name": "lookup_decode", "op": "lookup", "n": 32, "seq": 1, "N": 4096, "vocab": 102400, "images": 0.0,
         "table": "bf16", "out": "bf16"},
        # a prompt batch of 16 sequences of 8192 tokens, a tenth of them image placeholders
        {"name": "lookup_prefill", "op": "lookup", "n": 131072, "seq": 8192, "N": 4096, "vocab": 102400, "images": 0.1,
         "table": "bf16", "out": "bf16"},
        # fp32 master table read into bf16 rows, odd width and count
        {"name": "lookup_odd", "op": "lookup", "n": 3001, "seq": 3001, "N": 1001, "vocab": 1000, "images": 0.25,
         "table": "f32", "out": "bf16"},
        # one short sequence with one image (the smallest workload of the benchmark)
        {"name": "scatter_tiny", "op": "scatter", "n": 200, "seq": 200, "N": 128, "vocab": 1000, "images": 0.7,
         "grad": "bf16"},
        # 32 tiled-image sequences of 2048 tokens, most of them image rows: few text rows, large table
        {"name": "scatter_tiled", "op": "scatter", "n": 65536, "seq": 2048, "N": 2560, "vocab": 102400, "images": 0.7,
         "grad": "bf16"},
        # 16 sequences of 8192 tokens, mostly text
        {"name": "scatter_long", "op": "scatter", "n": 131072, "seq": 8192, "N": 4096, "vocab": 102400, "images": 0.1,
         "grad": "bf16"},
        # 32 images x 7 views of 27 x 27 patches, 1152 channels
        {"name": "ln_tiled", "op": "ln", "rows": 163296, "C": 1152, "x": "bf16", "y": "bf16"},
        # one image of 24 x 24 patches and a class row, fp32, odd width
        {"name": "ln_odd", "op": "ln", "rows": 577, "C": 1001, "x": "f32", "y": "f32"},
        # 16 images of mixed grids, about 50,000 patches
        {"name": "ln_grad_mixed", "op": "ln_grad", "rows": 50176, "C": 1152, "x": "bf16", "y": "bf16"},
        # 8192 projected rows, 5120 wide
        {"name": "ln_grad_wide", "op": "ln_grad", "rows": 8192, "C": 5120, "x": "bf16", "y": "bf16"},
        # gradients of the smallest projector of the benchmark
        {"name": "clip_tiny", "op": "clip", "C": 64, "k": 2, "N1": 256, "N2": 128, "grad": "f32", "max_norm": 1.0},
        # gradients of a 40 M parameter projector
        {"name": "clip_merger", "op": "clip", "C": 1152, "k": 2, "N1": 4608, "N2": 4096, "grad": "f32",
         "max_norm": 1.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lookup", "scatter", "ln", "ln_grad", "clip"])
    if op in ("lookup", "scatter"):
        n, N, vocab = _log(rng, 1, 131072), _log(rng, 32, 5120), _log(rng, 100, 102400)
        n, vocab = min(n, 131072 * 4096 // N), min(vocab, 102400 * 4096 // N)
        if rng.random() < 0.5:
            N = -(-N // 64) * 64
            n, vocab = max(1, min(n, 131072 * 4096 // N)), max(1, min(vocab, 102400 * 4096 // N))
        case = {"op": op, "n": n, "seq": max(1, n // rng.choice([1, 2, 8])), "N": N, "vocab": vocab,
                "images": rng.choice([0.0, 0.1, 0.25, 0.7])}
        if op == "lookup":
            case["table"], case["out"] = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16")])
        else:
            case["grad"] = rng.choice(["bf16", "f16", "f32"])
        return case
    if op in ("ln", "ln_grad"):
        C = _log(rng, 48, 9216)
        if rng.random() < 0.6:
            C = -(-C // 64) * 64
        rows = min(_log(rng, 1, 163296), (163296 if op == "ln" else 50176) * 1152 // C)
        x, y = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16")])
        return {"op": op, "rows": rows, "C": C, "x": x, "y": y}
    return {"op": "clip", "C": 64 * rng.randint(1, 18), "k": rng.choice([1, 2]), "N1": 64 * _log(rng, 1, 64),
            "N2": 32 * _log(rng, 1, 128), "grad": rng.choice(["f32", "bf16", "f16"]),
            "max_norm": rng.choice([0.1, 1.0, 1e4])}


def _normal(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def _ids(case, g):
    """Token ids by a 1/rank law over the vocabulary, as text has them (most rows of a batch
    share a few tokens, many tokens do not occur), and one run of image placeholders in
    each sequence."""
    n, vocab, seq = case["n"], case["vocab"], case["seq"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = torch.exp(u * math.log(vocab + 1.0)).sub_(1.0).floor_().long().clamp_(0, vocab - 1)
    # the rank law in an order of its own, so that frequent tokens lie anywhere in the table
    ids = torch.randperm(vocab, generator=g, device="cuda")[ids]
    run = int(case["images"] * seq)
    at = torch.arange(n, device="cuda") % seq
    return torch.where((at >= seq // 8) & (at < seq // 8 + run), IMAGE_TOKEN if vocab <= IMAGE_TOKEN else vocab - 1, ids)


def _token(case):
    return IMAGE_TOKEN if case["vocab"] <= IMAGE_TOKEN else case["vocab"] - 1


def _clip_shapes(case):
    k1 = case["k"] ** 2 * case["C"]
    return [(case["N1"], k1), (case["N1"],), (case["N2"], case["N1"]), (case["N2"],), (case["C"],), (case["C"],)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case)}
    if case["op"] == "lookup":
        s["scale"] = math.sqrt(case["N"])
        s["table"] = _normal(g, (case["vocab"], case["N"]), DTYPES[case["table"]], 0.02)
        s["ids"] = _ids(case, g)
        s["out"] = _normal(g, (case["n"], case["N"]), DTYPES[case["out"]])     # holds the image rows already
    elif case["op"] == "scatter":
        s["scale"] = math.sqrt(case["N"])
        s["ids"] = _ids(case, g)
        s["d_out"] = _normal(g, (case["n"], case["N"]), DTYPES[case["grad"]])
        s["d_table"] = torch.empty(case["vocab"], case["N"], device="cuda")
    elif case["op"] in ("ln", "ln_grad"):
        rows, C = case["rows"], case["C"]
        # rows of a tower differ in level and size; a few channels stand out
        x = torch.randn(rows, C, generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
        x += torch.randn(rows, 1, generator=g, device="cuda")
        x[:, ::97] *= 8
        s["x"] = x.to(DTYPES[case["x"]])
        s["gamma"] = 1 + _normal(g, (C,), torch.float32, 0.1)
        s["beta"] = _normal(g, (C,), torch.float32, 0.02)
        s["mean"], s["rstd"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        if case["op"] == "ln":
            s["y"] = torch.empty(rows, C, device="cuda", dtype=DTYPES[case["y"]])
        else:
            x64 = s["x"].double()
            s["mean"].copy_(x64.mean(1))
            s["rstd"].copy_(1 / torch.sqrt(x64.var(1, unbiased=False) + 1e-5))
            s["d_y"] = _normal(g, (rows, C), DTYPES[case["y"]])
            s["d_x"] = torch.empty(rows, C, device="cuda", dtype=DTYPES[case["x"]])
            s["d_gamma"], s["d_beta"] = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    else:
        s["grads"] = [_normal(g, sh, DTYPES[case["grad"]], 0.01 * (i + 1)) for i, sh in enumerate(_clip_shapes(case))]
        s["clipped"] = [torch.empty_like(t) for t in s["grads"]]
        s["norm"] = torch.empty(1, device="cuda")
    return s


def run(state):
    case = state["case"]
    if own:
        return _run_own(case["op"], case, state)
    return _PLAIN[case["op"]](case, state)


def _run_own(op, case, s):
    import vision_language_projector_b200 as vp

    if op == "lookup":
        vp.embed(s["ids"], s["table"], s["out"], scale=s["scale"], image_token_id=_token(case))
        return s["out"]
    if op == "scatter":
        vp.embed_backward(s["ids"], s["d_out"], s["d_table"], scale=s["scale"], image_token_id=_token(case))
        return s["d_table"]
    if op == "ln":
        vp.layernorm(s["x"], s["y"], gamma=s["gamma"], beta=s["beta"], eps=1e-5, mean=s["mean"], rstd=s["rstd"])
        return s["y"], s["mean"], s["rstd"]
    if op == "ln_grad":
        vp.layernorm_backward(s["x"], s["mean"], s["rstd"], s["d_y"], gamma=s["gamma"], d_x=s["d_x"],
                              d_gamma=s["d_gamma"], d_beta=s["d_beta"])
        return s["d_x"], s["d_gamma"], s["d_beta"]
    vp.clip_grads(s["grads"], case["max_norm"], norm=s["norm"], out=s["clipped"])
    return [s["norm"]] + s["clipped"]


# ---- plain forms: elementary operations in 32 bits, rounded once at the end
def _lookup(case, s):
    text = (s["ids"] != _token(case)).unsqueeze(1)
    rows = s["table"][s["ids"].clamp(max=case["vocab"] - 1)].float()
    return torch.where(text, (rows * s["scale"]).to(s["out"].dtype), s["out"])


def _scatter(case, s):
    vocab = case["vocab"]
    at = torch.where(s["ids"] == _token(case), vocab, s["ids"])       # image rows to a row of their own, dropped
    total = torch.zeros(vocab + 1, case["N"], device="cuda")
    total.index_add_(0, at, s["d_out"].float())
    return total[:vocab] * s["scale"]


def _ln(case, s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5)
    y = d * rstd * s["gamma"] + s["beta"]
    return y.to(s["y"].dtype), mean.squeeze(1), rstd.squeeze(1)


def _ln_grad(case, s):
    xhat = (s["x"].float() - s["mean"].unsqueeze(1)) * s["rstd"].unsqueeze(1)
    dy = s["d_y"].float()
    g = dy * s["gamma"]
    dx = s["rstd"].unsqueeze(1) * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx.to(s["d_x"].dtype), (dy * xhat).sum(0), dy.sum(0)


def _clip(case, s):
    grads = [t.float() for t in s["grads"]]
    norm = torch.sqrt(torch.stack([(t * t).sum(dtype=torch.float64) for t in grads]).sum())
    coef = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0).float()
    return [norm.float().reshape(1)] + [(t * coef).to(u.dtype) for t, u in zip(grads, s["grads"])]


_PLAIN = {"lookup": _lookup, "scatter": _scatter, "ln": _ln, "ln_grad": _ln_grad, "clip": _clip}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        want = s["out"].double()
        at = torch.nonzero(s["ids"] != _token(case)).flatten()
        want[at] = torch.index_select(s["table"], 0, s["ids"][at]).double() * s["scale"]
        return want
    if op == "scatter":
        # rows in token order; each token's sum is a difference of the running column sums
        ids, order = torch.sort(s["ids"], stable=True)
        keep = ids != _token(case)
        ids, order = ids[keep], order[keep]
        tokens, counts = torch.unique_consecutive(ids, return_counts=True)
        ends = torch.cumsum(counts, 0)
        want = torch.zeros(case["vocab"], case["N"], device="cuda", dtype=torch.float64)
        for c0 in range(0, case["N"], 512):
            run_ = torch.cumsum(s["d_out"][:, c0:c0 + 512][order].double(), 0)
            run_ = torch.cat([torch.zeros_like(run_[:1]), run_]) if len(run_) else torch.zeros(
                1, min(512, case["N"] - c0), device="cuda", dtype=torch.float64)
            want[tokens, c0:c0 + 512] = run_[ends] - run_[ends - counts]
        return want * s["scale"]
    if op == "ln":
        x = s["x"].double()
        mean = x.sum(1) / case["C"]
        var = ((x - mean[:, None]) ** 2).sum(1) / case["C"]
        rstd = (var + 1e-5) ** -0.5
        return (x - mean[:, None]) * rstd[:, None] * s["gamma"].double() + s["beta"].double(), mean, rstd
    if op == "ln_grad":
        # the Jacobian's three terms from the sums a row needs: S0 = sum g, S1 = sum g x
        x, dy = s["x"].double(), s["d_y"].double()
        mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
        g = dy * s["gamma"].double()
        s0 = g.sum(1, keepdim=True)
        s1 = (g * (x - mean)).sum(1, keepdim=True) * rstd
        dx = rstd * g - rstd / case["C"] * s0 - rstd * rstd / case["C"] * s1 * (x - mean)
        return dx, torch.einsum("rc,rc->c", dy, (x - mean) * rstd), torch.einsum("rc->c", dy)
    flat = torch.cat([t.double().reshape(-1) for t in s["grads"]])
    norm = float(torch.dot(flat, flat)) ** 0.5
    coef = min(1.0, case["max_norm"] / (norm + 1e-6))
    return [torch.tensor([norm], dtype=torch.float64)] + [t.double() * coef for t in s["grads"]]


def _size(name):
    return 4 if name == "f32" else 2


def _distinct(n, vocab):
    """Expected number of different tokens among n drawn by the rank law of _ids."""
    t = np.arange(vocab, dtype=np.float64)
    p = np.log((t + 2) / (t + 1)) / math.log(vocab + 1.0)
    return float((1 - np.exp(n * np.log1p(-np.minimum(p, 1 - 1e-12)))).sum())


def work(case):
    op = case["op"]
    if op in ("lookup", "scatter"):
        n, N = case["n"], case["N"]
        text = n - (n // case["seq"]) * int(case["images"] * case["seq"])
        if op == "lookup":
            rows = _distinct(text, case["vocab"])
            return {"bytes": 8 * n + rows * N * _size(case["table"]) + text * N * _size(case["out"]), "flops": text * N}
        return {"bytes": 8 * n + text * N * _size(case["grad"]) + 4 * case["vocab"] * N, "flops": 2 * text * N}
    if op in ("ln", "ln_grad"):
        rows, C = case["rows"], case["C"]
        x, y = _size(case["x"]), _size(case["y"])
        if op == "ln":
            return {"bytes": rows * C * (x + y) + 8 * C + 8 * rows, "flops": 7 * rows * C}
        return {"bytes": rows * C * (2 * x + y) + 12 * C + 8 * rows, "flops": 14 * rows * C}
    total = sum(math.prod(sh) for sh in _clip_shapes(case))
    return {"bytes": 2 * total * _size(case["grad"]) + 4, "flops": 3 * total}
