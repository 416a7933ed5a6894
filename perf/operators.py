"""The operators of a gated feed-forward block, as cases to be measured.

A gated block is  y = (act(x Wg^T) * (x Wu^T)) Wd^T.  Four operators train and
serve it:

* ``ffn``     the block's forward pass, from one token to a training batch;
* ``ffn_bwd`` its backward pass from the saved gate and up projections;
* ``ns``      the orthogonalised update of its weights (five Newton-Schulz
              steps of a quintic polynomial on the normalised matrix);
* ``w4``      its products for a few tokens from weights held in 4 bits with a
              scale (and optionally a zero point) per group of the row.

``run`` computes them in plain torch, in 32 bits, or, where ``own`` is true,
through this repository's entry points.
"""
import math

import torch

own = False

NS_COEFFS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One token through a small block: the latency of a decode step.
        dict(name="ffn_decode_1x1024x4096", op="ffn", T=1, D=1024, F=4096, act="silu", dtype="f16", save=False),
        # A serving batch of single tokens: the weights' bytes are the bound.
        dict(name="ffn_batch_24x4096x8192", op="ffn", T=24, D=4096, F=8192, act="silu", dtype="bf16", save=False),
        # A training forward with no dimension a multiple of a tile; the
        # projections are kept for the backward pass.
        dict(name="ffn_ragged_3000x4104x5000", op="ffn", T=3000, D=4104, F=5000, act="gelu_tanh", dtype="f16", save=True),
        # A long prompt through a wide block.
        dict(name="ffn_prefill_8192x8192x16384", op="ffn", T=8192, D=8192, F=16384, act="silu", dtype="f16", save=False),
        # Fine-tuning a small block on a short, odd batch.
        dict(name="ffn_bwd_333x1032x2744", op="ffn_bwd", T=333, D=1032, F=2744, act="relu", dtype="bf16"),
        # A training step's backward pass.
        dict(name="ffn_bwd_8192x4096x8192", op="ffn_bwd", T=8192, D=4096, F=8192, act="silu", dtype="f16"),
        # A square projection of a decode step, symmetric codes.
        dict(name="w4_1x4096x4096_g128", op="w4", T=1, N=4096, K=4096, group=128, zeros=False, gated=False, act="", dtype="f16"),
        # A few sequences decoded together, with zero points.
        dict(name="w4_5x8192x8192_g64", op="w4", T=5, N=8192, K=8192, group=64, zeros=True, gated=False, act="", dtype="bf16"),
        # The gate and up projections of a wide block for one token.
        dict(name="w4_gated_1x16384x8192_g32", op="w4", T=1, N=16384, K=8192, group=32, zeros=False, gated=True, act="silu", dtype="f16"),
        # The update of one small square matrix.
        dict(name="ns_512x512", op="ns", B=1, M=512, N=512, rank=32, src="f32", dtype="f16"),
        # Tall ragged matrices of several layers, updated together.
        dict(name="ns_6x1000x344", op="ns", B=6, M=1000, N=344, rank=64, src="bf16", dtype="bf16"),
        # The update of a wide block's down projection.
        dict(name="ns_4096x8192", op="ns", B=1, M=4096, N=8192, rank=256, src="f32", dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log8(rng, lo, hi):
    return max(8, (_log(rng, lo, hi) + 4) // 8 * 8)


def draw(rng):
    op = rng.choice(("ffn", "ffn_bwd", "w4", "ns"))
    if op in ("ffn", "ffn_bwd"):
        c = dict(op=op, T=_log(rng, 1, 8192), D=_log8(rng, 256, 8192), F=_log8(rng, 512, 16384),
                 act=rng.choice(("silu", "gelu_tanh", "relu")), dtype=rng.choice(("f16", "bf16")))
        if op == "ffn":
            c["save"] = rng.random() < 0.5
        elif c["T"] * c["D"] * c["F"] > 8192 * 4096 * 16384:
            c["T"] = (c["T"] + 1) // 2  # twice the forward's work a token
        return c
    if op == "w4":
        group = rng.choice((32, 64, 128))
        gated = rng.random() < 0.4
        return dict(op="w4", T=_log(rng, 1, 16), N=_log(rng, 512, 16384), K=max(1, _log(rng, 512, 16384) // group) * group,
                    group=group, zeros=rng.random() < 0.5, gated=gated, act=rng.choice(("silu", "gelu_tanh", "relu")) if gated else "",
                    dtype=rng.choice(("f16", "bf16")))
    m, n = _log(rng, 128, 4096), _log(rng, 128, 8192)
    if rng.random() < 0.5:
        m, n = n, m
    b = rng.choice((1, 1, 2, 5)) if m * n <= 1 << 20 else 1
    return dict(op="ns", B=b, M=m, N=n, rank=max(1, min(m, n) // 16), src=rng.choice(("f32", "bf16", "f16")), dtype=rng.choice(("f16", "bf16")))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("ffn", "ffn_bwd"):
        T, D, F = case["T"], case["D"], case["F"]
        s["x"] = _randn(gen, T, D).to(dt)
        s["w_in"] = _randn(gen, 2 * F, D).mul_(D ** -0.5).to(dt)     # gate rows, then up rows
        s["w_down"] = _randn(gen, D, F).mul_(F ** -0.5).to(dt)
        if case["op"] == "ffn_bwd":
            s["dy"] = _randn(gen, T, D).to(dt)
            s["gu"] = s["x"] @ s["w_in"].t()                         # what the forward pass kept
    elif case["op"] == "w4":
        T, N, K, g = case["T"], case["N"], case["K"], case["group"]
        rows = 2 * N if case["gated"] else N
        s["x"] = _randn(gen, T, K).to(dt)
        # Two codes a byte, the even column in the low half.
        s["codes"] = torch.randint(0, 256, (rows, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
        s["scales"] = (_randn(gen, rows, K // g).abs_() * 0.1 + 0.2).mul_(K ** -0.5).to(dt)
        s["zeros"] = torch.randint(5, 12, (rows, K // g), generator=gen, device="cuda", dtype=torch.uint8) if case["zeros"] else None
    else:
        # A momentum: a few strong directions over a weak background.
        B, M, N, r = case["B"], case["M"], case["N"], case["rank"]
        m = torch.matmul(_randn(gen, B, M, r), _randn(gen, B, r, N)).mul_(r ** -0.5)
        m.add_(_randn(gen, B, M, N), alpha=0.1).mul_(1e-3)
        s["m"] = (m if B > 1 else m[0]).to(DTYPES[case["src"]]).contiguous()
    return s


def _act(name, g):
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "relu":
        return torch.clamp_min(g, 0.0)
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(name, g):
    if name == "silu":
        p = torch.sigmoid(g)
        return p * (1.0 + g * (1.0 - p))
    if name == "relu":
        return (g > 0).to(g.dtype)
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g)


def _dequant(s):
    q = torch.stack((s["codes"] & 15, s["codes"] >> 4), dim=-1).flatten(1).float()
    q = q.unflatten(1, (-1, s["group"]))
    z = s["zeros"].float().unsqueeze(-1) if s["zeros"] is not None else 8.0
    return ((q - z) * s["scales"].float().unsqueeze(-1)).flatten(1)


def _ns(m, dtype):
    a, b, c = NS_COEFFS
    x = m.float()
    x = x / (x.square().sum(dim=(-2, -1), keepdim=True).sqrt() + NS_EPS)
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT.contiguous() if tall else x
    for _ in range(NS_STEPS):
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return (x.mT if tall else x).to(dtype).contiguous()


def _plain(s):
    dt = DTYPES[s["dtype"]]
    if s["op"] == "ffn":
        gu = s["x"].float() @ s["w_in"].float().t()
        g, u = gu[:, :s["F"]], gu[:, s["F"]:]
        y = ((_act(s["act"], g) * u) @ s["w_down"].float().t()).to(dt)
        return {"y": y, "gu": gu.to(dt)} if s["save"] else {"y": y}
    if s["op"] == "ffn_bwd":
        F, dy, x = s["F"], s["dy"].float(), s["x"].float()
        g, u = s["gu"][:, :F].float(), s["gu"][:, F:].float()
        a = _act(s["act"], g)
        dh = dy @ s["w_down"].float()
        dgu = torch.cat((dh * u * _act_grad(s["act"], g), dh * a), dim=1)
        return {"dx": (dgu @ s["w_in"].float()).to(dt), "dw_in": (dgu.t() @ x).to(dt), "dw_down": (dy.t() @ (a * u)).to(dt)}
    if s["op"] == "w4":
        y = s["x"].float() @ _dequant(s).t()
        if s["gated"]:
            y = _act(s["act"], y[:, :s["N"]]) * y[:, s["N"]:]
        return {"y": y.to(dt)}
    return {"o": _ns(s["m"], dt)}


def run(state):
    if not own:
        return _plain(state)
    import dense_fp16_gemm_04_gb300 as g
    s = state
    if s["op"] == "ffn":
        if s["save"]:
            y, gu = g.gated_ffn(s["x"], s["w_in"], s["w_down"], act=s["act"], save=True)
            return {"y": y, "gu": gu}
        return {"y": g.gated_ffn(s["x"], s["w_in"], s["w_down"], act=s["act"])}
    if s["op"] == "ffn_bwd":
        dx, dw_in, dw_down = g.gated_ffn_backward(s["dy"], s["x"], s["w_in"], s["w_down"], s["gu"], act=s["act"])
        return {"dx": dx, "dw_in": dw_in, "dw_down": dw_down}
    if s["op"] == "w4":
        if s["gated"]:
            return {"y": g.w4_gated(s["x"], s["codes"], s["scales"], s["zeros"], act=s["act"])}
        return {"y": g.w4_linear(s["x"], s["codes"], s["scales"], s["zeros"])}
    return {"o": g.orthogonalize(s["m"], steps=NS_STEPS, coeffs=NS_COEFFS, eps=NS_EPS, dtype=DTYPES[s["dtype"]])}


def work(case):
    e = 2
    if case["op"] in ("ffn", "ffn_bwd"):
        T, D, F = case["T"], case["D"], case["F"]
        if case["op"] == "ffn":
            return {"bytes": e * (2 * T * D + 3 * D * F + (2 * T * F if case["save"] else 0)), "flops": 6 * T * D * F}
        return {"bytes": e * (3 * T * D + 6 * D * F + 2 * T * F), "flops": 12 * T * D * F}
    if case["op"] == "w4":
        rows = case["N"] * (2 if case["gated"] else 1)
        per_group = e + (1 if case["zeros"] else 0)
        return {"bytes": rows * case["K"] // 2 + rows * (case["K"] // case["group"]) * per_group + e * case["T"] * (case["K"] + case["N"]),
                "flops": 2 * case["T"] * rows * case["K"]}
    # Both Gram products are symmetric: half of each is enough.
    B, m, n = case["B"], min(case["M"], case["N"]), max(case["M"], case["N"])
    return {"bytes": B * m * n * (e + (4 if case["src"] == "f32" else 2)), "flops": B * NS_STEPS * (3 * m * m * n + m * m * m)}


def exact(case, seed):
    """The definitions in 64 bits."""
    w = work(case)
    if w["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    d = torch.float64
    k = math.sqrt(2.0 / math.pi)

    def act(v):
        if s["act"] == "silu":
            return v / (1.0 + torch.exp(-v))
        if s["act"] == "relu":
            return torch.where(v > 0, v, torch.zeros_like(v))
        return v / (1.0 + torch.exp(-2.0 * k * (v + 0.044715 * v ** 3)))

    def slope(v):
        if s["act"] == "relu":
            return torch.where(v > 0, torch.ones_like(v), torch.zeros_like(v))
        arg, darg = (v, 1.0) if s["act"] == "silu" else (2.0 * k * (v + 0.044715 * v ** 3), 2.0 * k * (1.0 + 0.134145 * v ** 2))
        p = 1.0 / (1.0 + torch.exp(-arg))
        return p + v * p * (1.0 - p) * darg

    if s["op"] == "ffn":
        g = torch.einsum("td,fd->tf", s["x"].to(d), s["w_in"][:s["F"]].to(d))
        u = torch.einsum("td,fd->tf", s["x"].to(d), s["w_in"][s["F"]:].to(d))
        y = torch.einsum("tf,df->td", act(g) * u, s["w_down"].to(d))
        return {"y": y, "gu": torch.cat((g, u), dim=1)} if s["save"] else {"y": y}
    if s["op"] == "ffn_bwd":
        F = s["F"]
        g, u, dy, x = s["gu"][:, :F].to(d), s["gu"][:, F:].to(d), s["dy"].to(d), s["x"].to(d)
        dh = torch.einsum("td,df->tf", dy, s["w_down"].to(d))
        dg, du = dh * u * slope(g), dh * act(g)
        dx = torch.einsum("tf,fd->td", dg, s["w_in"][:F].to(d)) + torch.einsum("tf,fd->td", du, s["w_in"][F:].to(d))
        dw_in = torch.cat((torch.einsum("tf,td->fd", dg, x), torch.einsum("tf,td->fd", du, x)))
        return {"dx": dx, "dw_in": dw_in, "dw_down": torch.einsum("td,tf->df", dy, act(g) * u)}
    if s["op"] == "w4":
        x, K, grp = s["x"].to(d), s["K"], s["group"]
        cols = torch.arange(K, device="cuda")
        q = (s["codes"][:, cols // 2].int() >> (4 * (cols % 2)).int()) & 15
        at = cols // grp
        z = s["zeros"][:, at].to(d) if s["zeros"] is not None else 8.0
        y = torch.einsum("tk,nk->tn", x, (q.to(d) - z) * s["scales"][:, at].to(d))
        return {"y": act(y[:, :s["N"]]) * y[:, s["N"]:] if s["gated"] else y}
    a, b, c = NS_COEFFS
    x = s["m"].to(d)
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + NS_EPS)
    wide = x.shape[-1] >= x.shape[-2]
    for _ in range(NS_STEPS):
        p = x @ x.mT if wide else x.mT @ x
        q = b * p + c * (p @ p)
        x = a * x + (q @ x if wide else x @ q)
    return {"o": x}
