"""Norms and the loss of a language model's head, as cases to be measured.

Around a block stand the norm before it and, at the end of the model, the loss
of its projection to a vocabulary.  Six operators:

* ``ln``, ``rms``          layer norm and RMS norm of each row;
* ``ln_bwd``, ``rms_bwd``  their gradients from the kept statistics, the
                           weight's (and bias's) reduced over the rows;
* ``xent``                 loss and log-sum-exp of  z = x W^T  for each token;
* ``xent_bwd``             the gradients of both with respect to x and W, from
                           the kept log-sum-exp.

``run`` computes them in plain torch, in 32 bits, or, where ``own`` is true,
through this repository's entry points.
"""
import math

import torch

own = False

EPS = {"ln": 1e-5, "rms": 1e-6}
IGNORE = -100
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # The norm of one token's decode step: latency alone.
        dict(name="ln_1x1024", op="ln", T=1, D=1024, dtype="f16", wtype="f16", save=False),
        # A training batch's norm, its statistics kept.
        dict(name="ln_8192x4096", op="ln", T=8192, D=4096, dtype="bf16", wtype="bf16", save=True),
        # A serving batch of single tokens.
        dict(name="rms_24x8192", op="rms", T=24, D=8192, dtype="bf16", wtype="bf16", save=False),
        # Full precision, rows that start on any element.
        dict(name="rms_3001x1003", op="rms", T=3001, D=1003, dtype="f32", wtype="f32", save=True),
        # Fine-tuning on a short, odd batch.
        dict(name="ln_bwd_333x1032", op="ln_bwd", T=333, D=1032, dtype="f16", wtype="f32"),
        # A training step's gradient through a wide norm.
        dict(name="ln_bwd_8192x8192", op="ln_bwd", T=8192, D=8192, dtype="bf16", wtype="bf16"),
        # Many tokens of a narrow model, master weights in 32 bits.
        dict(name="rms_bwd_16384x2048", op="rms_bwd", T=16384, D=2048, dtype="bf16", wtype="f32"),
        # The log-probability of one token: the vocabulary's bytes.
        dict(name="xent_1x4096x32000", op="xent", T=1, D=4096, V=32000, dtype="f16", save=False),
        # A small evaluation batch, no dimension a multiple of a tile.
        dict(name="xent_1000x1032x20011", op="xent", T=1000, D=1032, V=20011, dtype="f16", save=True),
        # A training forward over a large vocabulary.
        dict(name="xent_4096x4096x131072", op="xent", T=4096, D=4096, V=131072, dtype="bf16", save=True),
        # Fine-tuning on a short, odd batch, loss scaled as fp16 needs it.
        dict(name="xent_bwd_333x1032x10007", op="xent_bwd", T=333, D=1032, V=10007, dtype="f16", zloss=False),
        # A training step's gradient over a large vocabulary, the log-sum-exp
        # itself penalised.
        dict(name="xent_bwd_4096x4096x131072", op="xent_bwd", T=4096, D=4096, V=131072, dtype="bf16", zloss=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("ln", "rms", "ln_bwd", "rms_bwd", "xent", "xent_bwd"))
    if op in ("xent", "xent_bwd"):
        c = dict(op=op, T=_log(rng, 1, 4096), D=max(8, _log(rng, 256, 4096) // 8 * 8), V=_log(rng, 1000, 131072),
                 dtype=rng.choice(("f16", "bf16")))
        if op == "xent":
            c["save"] = rng.random() < 0.5
        else:
            c["zloss"] = rng.random() < 0.5
        return c
    T, D = _log(rng, 1, 16384), _log(rng, 64, 16384)
    if rng.random() < 0.5:
        D = max(8, D // 8 * 8)
    T = max(1, min(T, 8192 * 8192 // D))
    dtype = rng.choice(("f16", "bf16", "f32"))
    c = dict(op=op, T=T, D=D, dtype=dtype, wtype=rng.choice((dtype, "f32")))
    if not op.endswith("_bwd"):
        c["save"] = rng.random() < 0.5
    return c


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    dt, T, D = DTYPES[case["dtype"]], case["T"], case["D"]
    if case["op"] in ("xent", "xent_bwd"):
        V = case["V"]
        w = _randn(gen, V, D).mul_(2.0 * D ** -0.5)
        s["targets"] = torch.randint(0, V, (T,), generator=gen, device="cuda")
        # A trained model's logits: the target's stand out from the others.
        s["x"] = _randn(gen, T, D).add_(w[s["targets"]], alpha=2.0).to(dt)
        s["w"] = w.to(dt)
        if T > 1:  # a prompt's tokens, which carry no loss
            s["targets"][: T // 8] = IGNORE
        if case["op"] == "xent_bwd":
            kept = max(1, int((s["targets"] != IGNORE).sum()))
            # The mean over the tokens that count, scaled up where fp16 needs it.
            scale = 1024.0 if case["dtype"] == "f16" else 1.0
            s["dloss"] = torch.full((1,), scale / kept, device="cuda").expand(T)
            xf = s["x"].float()
            s["lse"] = torch.logsumexp(torch.stack([torch.logsumexp(xf @ p.float().t(), 1) for p in s["w"].split(16384)]), 0)
            # 1e-4 lse^2 of the same tokens.
            s["dlse"] = 2e-4 * scale / kept * s["lse"] * (s["targets"] != IGNORE) if case["zloss"] else None
        return s
    wt, kind = DTYPES[case["wtype"]], case["op"].split("_")[0]
    # A residual stream: rows of different size, a few columns far larger.
    x = _randn(gen, T, D).mul_(torch.exp(0.5 * _randn(gen, T, 1))).add_(_randn(gen, 1, D).mul_(0.3))
    x[:, :: max(1, D // 4)] *= 8.0
    s["x"] = x.to(dt)
    s["weight"] = _randn(gen, D).mul_(0.1).add_(1.0).to(wt)
    s["bias"] = _randn(gen, D).mul_(0.1).to(wt) if kind == "ln" else None
    if case["op"].endswith("_bwd"):
        s["dy"] = _randn(gen, T, D).to(dt)
        s["stats"] = _stats(s["x"].float(), kind)
    return s


def _stats(x, kind):
    """Mean and reciprocal deviation of each row, or the reciprocal alone."""
    if kind == "rms":
        return (x.square().mean(1, keepdim=True) + EPS[kind]).rsqrt()
    mean = x.mean(1, keepdim=True)
    return torch.cat((mean, ((x - mean).square().mean(1, keepdim=True) + EPS[kind]).rsqrt()), 1)


def _plain(s):
    dt = DTYPES[s["dtype"]]
    x = s["x"].float()
    if s["op"] in ("ln", "rms"):
        stats = _stats(x, s["op"])
        h = (x - stats[:, :1]) * stats[:, 1:] if s["op"] == "ln" else x * stats
        y = h * s["weight"].float()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return {"y": y.to(dt), "stats": stats} if s["save"] else {"y": y.to(dt)}
    if s["op"] in ("ln_bwd", "rms_bwd"):
        ln, stats, dy, wt = s["op"] == "ln_bwd", s["stats"], s["dy"].float(), DTYPES[s["wtype"]]
        r = stats[:, -1:]
        h = (x - stats[:, :1]) * r if ln else x * r
        g = dy * s["weight"].float()
        dx = g - h * (g * h).mean(1, keepdim=True)
        if ln:
            dx = dx - g.mean(1, keepdim=True)
        out = {"dx": (dx * r).to(dt), "dweight": (dy * h).sum(0).to(wt)}
        if ln:
            out["dbias"] = dy.sum(0).to(wt)
        return out
    w, targets = s["w"].float(), s["targets"]
    kept = targets != IGNORE
    at = torch.where(kept, targets, 0)
    z = x @ w.t()
    if s["op"] == "xent":
        top = z.amax(1, keepdim=True)
        lse = torch.exp(z - top).sum(1).log() + top[:, 0]
        loss = torch.where(kept, lse - z.gather(1, at[:, None])[:, 0], 0.0)
        return {"loss": loss, "lse": lse} if s["save"] else {"loss": loss}
    dloss = s["dloss"] * kept
    dz = torch.exp(z - s["lse"][:, None]) * (dloss + s["dlse"] if s["dlse"] is not None else dloss)[:, None]
    dz[torch.arange(len(at), device=at.device), at] -= dloss
    return {"dx": (dz @ w).to(dt), "dw": (dz.t() @ x).to(dt)}


def run(state):
    if not own:
        return _plain(state)
    import dense_fp16_gemm_04_gb300 as g
    s = state
    if s["op"] == "ln":
        if s["save"]:
            y, stats = g.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS["ln"], save=True)
            return {"y": y, "stats": stats}
        return {"y": g.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS["ln"])}
    if s["op"] == "rms":
        if s["save"]:
            y, stats = g.rms_norm(s["x"], s["weight"], eps=EPS["rms"], save=True)
            return {"y": y, "stats": stats}
        return {"y": g.rms_norm(s["x"], s["weight"], eps=EPS["rms"])}
    if s["op"] == "ln_bwd":
        dx, dweight, dbias = g.layer_norm_backward(s["dy"], s["x"], s["weight"], s["stats"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if s["op"] == "rms_bwd":
        dx, dweight = g.rms_norm_backward(s["dy"], s["x"], s["weight"], s["stats"])
        return {"dx": dx, "dweight": dweight}
    if s["op"] == "xent":
        if s["save"]:
            loss, lse = g.linear_cross_entropy(s["x"], s["w"], s["targets"], ignore_index=IGNORE, save=True)
            return {"loss": loss, "lse": lse}
        return {"loss": g.linear_cross_entropy(s["x"], s["w"], s["targets"], ignore_index=IGNORE)}
    dx, dw = g.linear_cross_entropy_backward(s["dloss"], s["x"], s["w"], s["targets"], s["lse"], ignore_index=IGNORE,
                                             dlse=s["dlse"])
    return {"dx": dx, "dw": dw}


def work(case):
    T, D, e = case["T"], case["D"], 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("xent", "xent_bwd"):
        V = case["V"]
        if case["op"] == "xent":
            return {"bytes": e * (T + V) * D + T * (8 + 4 + (4 if case["save"] else 0)), "flops": 2 * T * D * V}
        # The logits again, dx and dw.
        return {"bytes": 2 * e * (T + V) * D + T * (8 + 4 + (4 if case["zloss"] else 0)), "flops": 6 * T * D * V}
    we, ln = 4 if case["wtype"] == "f32" else 2, case["op"].startswith("ln")
    stats, vectors = 4 * T * (2 if ln else 1), we * D * (2 if ln else 1)
    if case["op"].endswith("_bwd"):
        return {"bytes": 3 * e * T * D + stats + we * D + vectors, "flops": (11 if ln else 9) * T * D}
    return {"bytes": 2 * e * T * D + vectors + (stats if case["save"] else 0), "flops": (7 if ln else 4) * T * D}


def exact(case, seed):
    """The definitions in 64 bits."""
    if work(case)["flops"] > 1.4e13:
        return None
    s = prepare(case, seed)
    d = torch.float64
    x = s["x"].to(d)
    if case["op"] in ("xent", "xent_bwd"):
        w, t = s["w"].to(d), s["targets"]
        rows = torch.nonzero(t >= 0)[:, 0]
        if case["op"] == "xent":
            loss, lse = torch.zeros(len(t), dtype=d, device="cuda"), []
            for a in range(0, len(t), 1024):
                lse.append(torch.logsumexp(torch.einsum("td,vd->tv", x[a:a + 1024], w), 1))
            lse = torch.cat(lse)
            loss[rows] = lse[rows] - torch.einsum("td,td->t", x[rows], w[t[rows]])
            return {"loss": loss, "lse": lse} if case["save"] else {"loss": loss}
        dloss = torch.zeros(len(t), dtype=d, device="cuda")
        dloss[rows] = s["dloss"].to(d)[rows]
        total = dloss + (s["dlse"].to(d) if s["dlse"] is not None else 0.0)
        dx, dw = torch.zeros_like(x), torch.zeros_like(w)
        for a in range(0, len(w), 16384):  # by pieces of the vocabulary
            wp = w[a:a + 16384]
            p = torch.exp(torch.einsum("td,vd->tv", x, wp) - s["lse"].to(d).unsqueeze(1)) * total.unsqueeze(1)
            here = rows[(t[rows] >= a) & (t[rows] < a + len(wp))]
            p[here, t[here] - a] -= dloss[here]
            dx += torch.einsum("tv,vd->td", p, wp)
            dw[a:a + 16384] = torch.einsum("tv,td->vd", p, x)
        return {"dx": dx, "dw": dw}
    n, ln = case["D"], case["op"].startswith("ln")
    weight = s["weight"].to(d)
    if not case["op"].endswith("_bwd"):
        mean = x.sum(1) / n if ln else torch.zeros(len(x), dtype=d, device="cuda")
        c = x - mean.unsqueeze(1)
        r = 1.0 / torch.sqrt(torch.einsum("td,td->t", c, c) / n + EPS[case["op"]])
        y = torch.einsum("td,t,d->td", c, r, weight)
        if ln:
            y += s["bias"].to(d)
        if not case["save"]:
            return {"y": y}
        return {"y": y, "stats": torch.stack((mean, r), 1) if ln else r.unsqueeze(1)}
    r, dy = s["stats"][:, -1].to(d), s["dy"].to(d)
    h = torch.einsum("td,t->td", x - s["stats"][:, :1].to(d) if ln else x, r)
    g = dy * weight
    # The Jacobian of a row's h, applied to g.
    back = g - torch.einsum("td,t->td", h, torch.einsum("td,td->t", g, h) / n)
    if ln:
        back = back - (g.sum(1) / n).unsqueeze(1)
    out = {"dx": torch.einsum("td,t->td", back, r), "dweight": torch.einsum("td,td->d", dy, h)}
    if ln:
        out["dbias"] = dy.sum(0)
    return out
