"""The loss over a vocabulary and its gradients against their definitions in 64 bits.

Tolerances are bounds, computed per element.  A logit is an fp32 sum of D products,
off by (D + 16) 2^-23 of the sum of their magnitudes.  An exponential is off by 2^-22
of itself and by what rounding its argument costs; the shares of a row are joined in
at most 16 + V / 2^15 steps, each with two of them.  dz is rounded to 16 bits, in fp16
with a floor of 2^-38 of the largest |dloss| (|dloss + dlse|).  Rounding to type t is
off by eps(t) / 2 of the value (fp16 below its normal range: 2^-25)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F64 = torch.float64
DTYPES = [torch.float16, torch.bfloat16]
E = 2.0 ** -24


@pytest.fixture(scope="module")
def g():
    import dense_fp16_gemm_04_gb300 as m
    m.build()
    return m


def u(dt):
    return torch.finfo(dt).eps / 2


def sum_eps(K):
    return (K + 16) * 2.0 ** -23


def check(got, ref, err, what):
    dt = got.dtype
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
    bound = 1.01 * (err + u(dt) * (ref.abs() + err)) + tiny + 1e-37
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = ((got.to(F64) - ref).abs() / bound).max().item() if got.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"


def make(T, D, V, dt, seed=0, ignore=-100):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    def r(*s):
        return torch.randn(*s, generator=gen, device="cuda")
    x, w = r(T, D).to(dt), (2 * r(V, D) * D ** -0.5).to(dt)
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda")
    if T:
        targets[0] = V - 1
    if T > 2:
        targets[1] = 0
        targets[torch.rand(T, generator=gen, device="cuda") < 0.2] = ignore
    dloss = r(T).abs() / max(T, 1) + 1e-3 / max(T, 1)
    return x, w, targets, dloss


def logits(x, w):
    return x.to(F64) @ w.to(F64).t(), sum_eps(x.shape[1]) * (x.to(F64).abs() @ w.to(F64).abs().t())


def forward_ref(x, w, targets, ignore=-100):
    z, ez = logits(x, w)
    V = z.shape[1]
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    e = (p * ez).sum(1) + 4 * E * (z.abs().amax(1) + 2 * (16 + V / 2 ** 15)) + 2 * E * lse.abs()
    kept = targets != ignore
    at = torch.where(kept, targets, 0)[:, None]
    zt = z.gather(1, at)[:, 0]
    loss = torch.where(kept, lse - zt, 0.0)
    return (loss, torch.where(kept, e + ez.gather(1, at)[:, 0] + 2 * E * (lse.abs() + zt.abs()), 0.0)), (lse, e)


def backward_ref(dloss, dlse, x, w, targets, lse, dt, ignore=-100):
    z, ez = logits(x, w)
    T, V = z.shape
    lse = lse.to(F64)[:, None]
    kept = targets != ignore
    b = torch.where(kept, dloss.to(F64), 0.0)
    a = b + dlse.to(F64) if dlse is not None else b
    dz = a[:, None] * torch.exp(z - lse)
    edz = dz.abs() * (ez + 4 * E * (z.abs() + lse.abs() + 2))
    rows = torch.nonzero(kept)[:, 0]
    dz[rows, targets[rows]] -= b[rows]
    edz += 4 * E * dz.abs() + (4 * E * a.abs())[:, None] * (dz != 0)
    del z, ez
    top = torch.maximum(a.abs().max(), b.abs().max())
    edz += u(dt) * (dz.abs() + edz) + (2.0 ** -38 * top if dt == torch.float16 else 0.0)
    xa, wa, da = x.to(F64).abs(), w.to(F64).abs(), dz.abs() + edz
    dx = dz @ w.to(F64), edz @ wa + (sum_eps(V) + 64 * E) * (da @ wa)
    dw = dz.t() @ x.to(F64), edz.t() @ xa + (sum_eps(T) + 4 * E) * (da.t() @ xa)
    return dx, dw


def run(g, x, w, targets, dloss, dlse=None, ignore=-100):
    T = x.shape[0]
    out = torch.full((T,), float("nan"), device="cuda")
    loss, lse = g.linear_cross_entropy(x, w, targets, ignore_index=ignore, save=True, out=out)
    assert loss.data_ptr() == out.data_ptr() or T == 0
    assert torch.equal(g.linear_cross_entropy(x, w, targets, ignore_index=ignore), loss)
    dx, dw = g.linear_cross_entropy_backward(dloss, x, w, targets, lse, ignore_index=ignore, dlse=dlse)
    g.default_ops().check_error()
    rl, rz = forward_ref(x, w, targets, ignore)
    check(loss, *rl, "loss")
    check(lse, *rz, "lse")
    assert not loss[targets == ignore].any()
    rx, rw = backward_ref(dloss, dlse, x, w, targets, lse, x.dtype, ignore)
    check(dx, *rx, "dx")
    check(dw, *rw, "dw")
    return loss, lse, dx, dw


# One token and one entry; around tiles of 128 and 256 rows and columns; few tiles with
# long rows, which clusters of 2, 4 and 8 CTAs share; pairs of CTAs.
SHAPES = [(1, 8, 1), (1, 64, 1000), (2, 16, 2), (3, 136, 129), (5, 4096, 300), (17, 512, 2000), (64, 2048, 1500),
          (100, 1024, 6000), (33, 264, 4099), (128, 1032, 8191), (130, 72, 20001), (257, 520, 5003), (700, 1000, 9973),
          (2000, 256, 33000), (1500, 2056, 12345), (300, 200, 7001)]


@pytest.mark.parametrize("dt", DTYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)), ids=["x".join(map(str, s)) for s in SHAPES])
def test_xent(g, i, shape, dt):
    x, w, targets, dloss = make(*shape, dt, seed=i)
    dlse = None if i % 2 else 0.3 * dloss * torch.sign(torch.randn(shape[0], device="cuda"))
    run(g, x, w, targets, dloss, dlse)


@pytest.mark.parametrize("shape", [(16500, 64, 16500), (70000, 64, 9001), (40000, 136, 20000), (17000, 72, 5000)])
def test_xent_in_pieces(g, shape):
    """More tokens than one launch of the forward pass takes, and more of dz than is
    held at a time: pieces of the vocabulary, the last one shorter."""
    x, w, targets, dloss = make(*shape, torch.bfloat16, seed=1)
    first = run(g, x, w, targets, dloss)
    loss, lse = g.linear_cross_entropy(x, w, targets, save=True)
    again = (loss, lse, *g.linear_cross_entropy_backward(dloss, x, w, targets, lse))
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_xent_against_differences(g):
    """<gradient, v> against central differences of the 64-bit loss along the gradient
    itself, where rounding dz and the result costs a few u of the gradient's size."""
    dt = torch.float16
    x, w, targets, dloss = make(60, 136, 777, dt, seed=5)
    dlse = 0.5 * dloss
    _, lse = g.linear_cross_entropy(x, w, targets, save=True)
    grads = g.linear_cross_entropy_backward(dloss * 1024, x, w, targets, lse, dlse=dlse * 1024)
    kept = targets >= 0
    def loss(xx, ww):
        z = xx @ ww.t()
        l = torch.logsumexp(z, 1)
        t = z.gather(1, targets.clamp_min(0)[:, None])[:, 0]
        return 1024 * ((l - t) * kept * dloss.to(F64) + l * dlse.to(F64)).sum()
    base = [x.to(F64), w.to(F64)]
    for i, gr in enumerate(grads):
        v = gr.to(F64) / gr.to(F64).norm()
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + 1e-4 * v, base[i] - 1e-4 * v
        num, ana = (loss(*hi) - loss(*lo)) / 2e-4, (gr.to(F64) * v).sum()
        assert abs(num - ana) <= 8 * u(dt) * ana.abs(), (i, num.item(), ana.item())


@pytest.mark.parametrize("shape", [(4, 264, 1000), (300, 136, 5000)])
def test_xent_strided(g, shape):
    x, w, targets, dloss = make(*shape, torch.float16)
    def pad(t, extra):
        big = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device="cuda")
        v = big[:, 8:8 + t.shape[1]]
        v.copy_(t)
        return v
    loss, lse = g.linear_cross_entropy(x, w, targets, save=True)
    loss2, lse2 = g.linear_cross_entropy(pad(x, 16), pad(w, 24), targets, save=True)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    one = torch.full((1,), 0.25, device="cuda").expand(shape[0])
    two = torch.full((shape[0], 3), 0.25, device="cuda")
    two[:, 1:] = float("nan")
    a = g.linear_cross_entropy_backward(one, x, w, targets, lse, dlse=two[:, 0])
    b = g.linear_cross_entropy_backward(one.contiguous(), pad(x, 16), pad(w, 24), targets, lse, dlse=one)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T", [1, 300])
def test_xent_empty_and_ignored(g, T):
    x, w, targets, dloss = make(T, 64, 500, torch.float16)
    loss, lse = g.linear_cross_entropy(x[:0], w, targets[:0], save=True)
    assert loss.shape == lse.shape == (0,)
    dx, dw = g.linear_cross_entropy_backward(dloss[:0], x[:0], w, targets[:0], lse)
    assert dx.shape == (0, 64) and dw.shape == w.shape and not dw.any()
    none = torch.full_like(targets, -100)
    loss, lse = g.linear_cross_entropy(x, w, none, save=True)
    assert not loss.any()
    check(lse, *forward_ref(x, w, none)[1], "lse")
    dx, dw = g.linear_cross_entropy_backward(dloss, x, w, none, lse)
    assert not dx.any() and not dw.any()
    # Only the lse has a gradient.
    dx, dw = g.linear_cross_entropy_backward(dloss, x, w, none, lse, dlse=dloss)
    rx, rw = backward_ref(dloss, dloss, x, w, none, lse, torch.float16)
    check(dx, *rx, "dx")
    check(dw, *rw, "dw")
    # Nothing has.
    dx, dw = g.linear_cross_entropy_backward(0 * dloss, x, w, targets, lse)
    assert not dx.any() and not dw.any()


@pytest.mark.parametrize("shape", [(5, 64, 700), (300, 136, 5000), (4000, 72, 40000), (9000, 64, 33000)])
@pytest.mark.parametrize("kept", [0.0, 0.01, 0.3, 0.9])
def test_xent_tokens_without_a_gradient_take_no_part(g, shape, kept):
    """Ignored tokens' x may hold anything, and the others' gradients are those of a
    batch of them alone."""
    T = shape[0]
    x, w, targets, dloss = make(*shape, torch.bfloat16, seed=4)
    targets.clamp_min_(0)
    gone = torch.rand(T, generator=torch.Generator().manual_seed(T)).cuda() >= kept
    targets[gone] = -100
    lse = torch.zeros(T, device="cuda")
    if (~gone).any():
        lse[~gone] = g.linear_cross_entropy(x[~gone], w, targets[~gone], save=True)[1]
    bad = x.clone()
    bad[gone] = float("nan")
    lse[gone], dloss[gone] = float("nan"), float("inf")
    dx, dw = g.linear_cross_entropy_backward(dloss, bad, w, targets, lse)
    g.default_ops().check_error()
    assert not dx[gone].any() and torch.isfinite(dx).all() and torch.isfinite(dw).all()
    if (~gone).any():
        rx, rw = backward_ref(dloss[~gone], None, x[~gone], w, targets[~gone], lse[~gone], torch.bfloat16)
        check(dx[~gone], *rx, "dx")
        check(dw, *rw, "dw")
    else:
        assert not dw.any()
    # A dloss of 0 is as good as an ignored token; a dlse takes part.
    dloss[gone] = 0.0
    dx2, dw2 = g.linear_cross_entropy_backward(dloss, bad, w, targets.clamp_min(0), lse)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_xent_other_ignore_index_and_bad_targets(g):
    x, w, targets, dloss = make(40, 64, 500, torch.bfloat16, ignore=7)
    run(g, x, w, targets, dloss, ignore=7)
    clean = g.linear_cross_entropy(x, w, targets, ignore_index=7, save=True)
    bad = targets.clone()
    bad[3], bad[5], bad[8] = 500, -1, 2 ** 40
    loss, lse = g.linear_cross_entropy(x, w, bad, ignore_index=7, save=True)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[3] = keep[5] = keep[8] = False
    assert torch.isnan(loss[~keep]).all() and torch.equal(loss[keep], clean[0][keep]) and torch.equal(lse, clean[1])
    dx, _ = g.linear_cross_entropy_backward(dloss, x, w, bad, lse, ignore_index=7)
    dx0, _ = g.linear_cross_entropy_backward(dloss, x, w, targets, lse, ignore_index=7)
    assert torch.isnan(dx[~keep]).all() and torch.equal(dx[keep], dx0[keep])


@pytest.mark.parametrize("T", [6, 200])
def test_xent_infinities_and_nan(g, T):
    x, w, targets, dloss = make(T, 64, 1000, torch.float16, ignore=-100)
    targets[:] = torch.arange(T, device="cuda") + 10
    x[:, 3] = 1.0
    x[2, 3] = -1.0
    loss0, lse0 = g.linear_cross_entropy(x, w, targets, save=True)
    # A NaN stays in its row.
    x2 = x.clone()
    x2[4, 1] = float("nan")
    loss, lse = g.linear_cross_entropy(x2, w, targets, save=True)
    keep = torch.arange(T, device="cuda") != 4
    assert torch.isnan(loss[4]) and torch.isnan(lse[4])
    assert torch.equal(loss[keep], loss0[keep]) and torch.equal(lse[keep], lse0[keep])
    dx = g.linear_cross_entropy_backward(dloss, x2, w, targets, lse)[0]
    assert torch.isnan(dx[4]).all()
    assert torch.equal(dx[keep], g.linear_cross_entropy_backward(dloss, x, w, targets, lse0)[0][keep])
    # An entry of infinite logits: +inf for all tokens but the third, -inf there.
    w2 = w.clone()
    w2[10] = 0.0
    w2[10, 3] = float("inf")  # (times the other elements' zeros it would be NaN)
    xs = x.clone()
    xs[:, :3], xs[:, 4:] = 1.0, 1.0
    loss, lse = g.linear_cross_entropy(xs, w2, targets, save=True)
    z = xs.to(F64) @ w2.to(F64).t()
    want = torch.logsumexp(z, 1) - z.gather(1, targets[:, None])[:, 0]
    assert torch.isposinf(lse[keep.new_tensor([i != 2 for i in range(T)])]).all() and torch.isfinite(lse[2])
    assert torch.equal(loss.isnan(), want.isnan()) and torch.equal(loss.isposinf(), want.isposinf())
    assert torch.isnan(loss[0]) and torch.isposinf(loss[1]) and torch.isfinite(loss[2])
    # Every logit -inf: lse -inf, loss NaN.
    w3 = torch.zeros_like(w)
    w3[:, 3] = float("-inf")
    loss, lse = g.linear_cross_entropy(xs[:2], w3, targets[:2], save=True)
    assert torch.isneginf(lse).all() and torch.isnan(loss).all()


@pytest.mark.parametrize("dt", DTYPES, ids=["f16", "bf16"])
def test_xent_sharp_and_far_logits(g, dt):
    """Logits up to 400 apart, and all of them far from zero."""
    x, w, targets, dloss = make(50, 64, 900, dt, seed=2)
    run(g, x * 40, w, targets, dloss)
    shifted = w.clone()
    shifted[:, 0] += 30.0
    x2 = x.clone()
    x2[:, 0] = 8.0
    run(g, x2, shifted, targets, dloss)


@pytest.mark.parametrize("shape", [(300, 4096, 3000), (5, 4096, 3000), (40, 4096, 300)])
def test_xent_gradients_of_sure_tokens(g, shape):
    """Tokens that the model is sure of, exp(-loss) within 1e-5 of 1: the target's dz is
    the difference of two numbers near 1.  Their errors must agree: a logit of 20 summed
    by the tensor cores alone is off by 1e-4.  Logits here are off by 16 truncations of
    2^-23 of at most the sum of magnitudes of 256 products, and the lse by as much: 2e-6
    of dloss for each, 2e-5 and half an exponent's rounding in all."""
    T, D, V = shape
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(V, D, generator=gen, device="cuda") * D ** -0.5
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda")
    x = (20 * w[targets]).half()
    w = w.half()
    loss, lse = g.linear_cross_entropy(x, w, targets, save=True)
    z = x.to(F64) @ w.to(F64).t()
    p = torch.softmax(z, 1)
    pt = p.gather(1, targets[:, None])[:, 0]
    assert (1 - pt).max() < 1e-4 and (loss.to(F64) + pt.log()).abs().max() < 2e-5
    dloss = torch.full((T,), 1024.0, device="cuda")  # (dx would be below fp16's normal range)
    dx, _ = g.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    dz = p.clone()
    dz[torch.arange(T, device="cuda"), targets] -= 1
    ref = 1024 * (dz @ w.to(F64))
    # dz off by 2e-5 at the target, the rest of it by 2^-11 of itself.
    err = 2e-5 * w[targets].to(F64).abs() + 2.0 ** -9 * (p @ w.to(F64).abs() - pt[:, None] * w[targets].to(F64).abs()).abs()
    check(dx, ref, 1024 * err + 2.0 ** -20 * ref.abs(), "dx")


@pytest.mark.parametrize("scale", [1e-30, 1e-9, 1.0, 1e20])
def test_xent_gradients_of_any_scale(g, scale):
    """fp16's dz is scaled by the largest dloss, tokens of far smaller ones beside it."""
    x, w, targets, dloss = make(100, 64, 2000, torch.float16, seed=3)
    targets.clamp_min_(0)
    _, lse = g.linear_cross_entropy(x, w, targets, save=True)
    d = torch.ones(100, device="cuda")
    d[10:20] = 2.0 ** -10
    want = g.linear_cross_entropy_backward(d, x, w, targets, lse)
    for a, (r, e) in zip(want, backward_ref(d, None, x, w, targets, lse, torch.float16)):
        check(a, r, e, "gradient")
    got = g.linear_cross_entropy_backward(d.bfloat16().float() * scale, x.bfloat16(), w.bfloat16(), targets, lse)
    refs = backward_ref(d * scale, None, x.bfloat16(), w.bfloat16(), targets, lse, torch.bfloat16)
    for a, (r, e) in zip(got, refs):
        check(a, r, e, "gradient")
    # An infinite or NaN dloss stays in its token's dx.
    d2 = d * 100
    d2[5], d2[6] = float("inf"), float("nan")
    dx = g.linear_cross_entropy_backward(d2, x, w, targets, lse)[0]
    base = g.linear_cross_entropy_backward(d * 100, x, w, targets, lse)[0]
    keep = torch.ones(100, dtype=torch.bool, device="cuda")
    keep[5] = keep[6] = False
    assert torch.equal(dx[keep], base[keep]) and not torch.isfinite(dx[~keep]).any()


def test_xent_single_entries_are_exact(g):
    """One-hot x: logits are w's own elements; a vocabulary of equal logits has
    lse = z + log V."""
    D, V = 64, 300
    w = torch.randn(V, D, device="cuda").to(torch.float16)
    x = torch.eye(D, device="cuda", dtype=torch.float16)
    targets = torch.arange(D, device="cuda")
    loss, lse = g.linear_cross_entropy(x, w, targets, save=True)
    rl, rz = forward_ref(x, w, targets)
    check(lse, rz[0], 8 * E * (rz[0].abs() + 8), "lse")
    check(lse - loss, w[targets, targets].to(F64), 4 * E * (rz[0].abs() + 8), "target")
    same = w[:1].expand(V, D).contiguous()
    lse = g.linear_cross_entropy(x, same, targets, save=True)[1]
    check(lse, w[0].to(F64) + torch.log(torch.tensor(300.0, dtype=F64, device="cuda")), 32 * E * 8, "lse")


def test_xent_many_tokens(g):
    """dz of 2.5e9 elements: tokens' offsets past 32 bits, ignored ones among them."""
    T, D, V = 600_000, 64, 4096
    x, w, targets, dloss = make(T, D, V, torch.bfloat16, seed=9)
    dloss = dloss * T
    loss, lse = g.linear_cross_entropy(x, w, targets, save=True)
    dx, dw = g.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    g.default_ops().check_error()
    pick = torch.cat((torch.arange(300, device="cuda"), torch.arange(T - 300, T, device="cuda"),
                      torch.randint(0, T, (2000,), device="cuda")))
    rl, rz = forward_ref(x[pick], w, targets[pick])
    check(loss[pick], *rl, "loss")
    check(lse[pick], *rz, "lse")
    rx, _ = backward_ref(dloss[pick], None, x[pick], w, targets[pick], lse[pick], x.dtype)
    check(dx[pick], *rx, "dx")
    assert not dx[targets < 0].any()
    ref, err = torch.zeros(V, D, dtype=F64, device="cuda"), torch.zeros(V, D, dtype=F64, device="cuda")
    for a in range(0, T, 30_000):
        b = slice(a, a + 30_000)
        _, (r, e) = backward_ref(dloss[b], None, x[b], w, targets[b], lse[b], x.dtype)
        ref += r
        err += e
    # (each part's bound has sum_eps of its own tokens; the sums of all of them pass on as many times more)
    check(dw, ref, err + sum_eps(T) / sum_eps(30_000) * err, "dw")


def test_xent_large_vocabulary(g):
    """W of 2.5e9 elements: entries' offsets past 32 bits, in either pass."""
    T, D, V = 3, 4096, 600_001
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(V, D, dtype=torch.float16, device="cuda")
    for part in w.split(100_000):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * 2 * D ** -0.5)
    x = torch.randn(T, D, generator=gen, device="cuda").half()
    targets = torch.tensor([V - 1, 524_288, 5], device="cuda")
    loss, lse = g.linear_cross_entropy(x, w, targets, save=True)
    dloss = torch.full((T,), 64.0, device="cuda")
    dx, dw = g.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    g.default_ops().check_error()
    zs = [logits(x, part) for part in w.split(100_000)]
    z, ez = (torch.cat(t, 1) for t in zip(*zs))
    ref = torch.logsumexp(z, 1)
    e = (torch.exp(z - ref[:, None]) * ez).sum(1) + 4 * E * (z.abs().amax(1) + 2 * (16 + V / 2 ** 15)) + 2 * E * ref.abs()
    check(lse, ref, e, "lse")
    zt = z.gather(1, targets[:, None])[:, 0]
    check(loss, ref - zt, e + ez.gather(1, targets[:, None])[:, 0] + 2 * E * (ref.abs() + zt.abs()), "loss")
    sel = torch.cat((targets, torch.randint(0, V, (500,), generator=gen, device="cuda"), torch.arange(V - 200, V, device="cuda")))
    hit = (sel[:, None] == targets).to(F64)
    dz = 64 * (torch.exp(z[:, sel] - lse.to(F64)[:, None]) - hit.t())
    edz = 64 * torch.exp(z[:, sel] - lse.to(F64)[:, None]) * (ez[:, sel] + 4 * E * (z[:, sel].abs() + lse[:, None].abs() + 2))
    edz = edz + u(w.dtype) * (dz.abs() + edz) + 2.0 ** -38 * 64 + 8 * E * 64
    xd = x.to(F64)
    check(dw[sel], dz.t() @ xd, edz.t() @ xd.abs() + sum_eps(T) * (dz.abs() + edz).t() @ xd.abs(), "dw")
    want, err = torch.zeros(T, D, dtype=F64, device="cuda"), torch.zeros(T, D, dtype=F64, device="cuda")
    for i, part in enumerate(w.split(100_000)):
        c = slice(i * 100_000, i * 100_000 + len(part))
        p = 64 * torch.exp(z[:, c] - lse.to(F64)[:, None])
        ep = p * (ez[:, c] + 4 * E * (z[:, c].abs() + lse[:, None].abs() + 2))
        ep = ep + u(w.dtype) * (p + ep) + 2.0 ** -38 * 64
        for t in range(T):
            if i * 100_000 <= targets[t] < i * 100_000 + len(part):
                p[t, targets[t] - i * 100_000] -= 64
                ep[t, targets[t] - i * 100_000] += (u(w.dtype) + 8 * E) * 64
        want += p @ part.to(F64)
        err += (ep + sum_eps(V) * (p.abs() + ep)) @ part.to(F64).abs()
    check(dx, want, err, "dx")


# ------------------------------------------------------------ streams, graphs --
def test_xent_streams_and_graphs(g):
    x, w, targets, dloss = make(300, 264, 5000, torch.bfloat16)
    def all_(stream=None):
        loss, lse = g.linear_cross_entropy(x, w, targets, save=True, stream=stream)
        return (loss, lse, *g.linear_cross_entropy_backward(dloss, x, w, targets, lse, stream=stream))
    want = [t.clone() for t in all_()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = all_(stream)
        trash = [torch.full((n,), float("nan"), device="cuda") for n in (1 << k for k in range(6, 24)) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del trash
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    got = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            got.append(all_())
    for t in got[0] + got[1]:
        t.fill_(float("nan"))
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for one in got:
        assert all(torch.equal(a, b) for a, b in zip(one, want))


def test_xent_refusals(g):
    x, w, targets, dloss = make(4, 64, 100, torch.float16)
    _, lse = g.linear_cross_entropy(x, w, targets, save=True)
    for call in (lambda: g.linear_cross_entropy(x, w[:, :32], targets), lambda: g.linear_cross_entropy(x, w, targets[:3]),
                 lambda: g.linear_cross_entropy(x, w.cpu(), targets), lambda: g.linear_cross_entropy(x, w, targets.cpu()),
                 lambda: g.linear_cross_entropy(x[0], w, targets),
                 lambda: g.linear_cross_entropy(x, w, targets.repeat(2)[::2]),
                 lambda: g.linear_cross_entropy(x, w, targets, out=torch.empty(3, device="cuda")),
                 lambda: g.linear_cross_entropy_backward(dloss[:2], x, w, targets, lse),
                 lambda: g.linear_cross_entropy_backward(dloss, x, w, targets, lse[:3]),
                 lambda: g.linear_cross_entropy_backward(dloss, x, w, targets, lse, dlse=dloss[:1])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: g.linear_cross_entropy(x.float(), w, targets), lambda: g.linear_cross_entropy(x, w.bfloat16(), targets),
                 lambda: g.linear_cross_entropy(x, w, targets.int()), lambda: g.linear_cross_entropy(x, w, targets, ignore_index=None),
                 lambda: g.linear_cross_entropy_backward(dloss.half(), x, w, targets, lse),
                 lambda: g.linear_cross_entropy_backward(dloss, x, w, targets, None)):
        with pytest.raises(TypeError):
            call()
    e16 = lambda *s: torch.empty(*s, dtype=torch.float16, device="cuda")
    for call, status in ((lambda: g.linear_cross_entropy(x[:, :60], w[:, :60], targets), 2),
                         (lambda: g.linear_cross_entropy(x, e16(0, 64), targets), 1),
                         (lambda: g.linear_cross_entropy(e16(4, 0), e16(100, 0), targets), 1)):
        with pytest.raises(g.GemmError) as e:
            call()
        assert e.value.status == status


def test_xent_stuck_waits_end(g):
    """A k-block that is never loaded, in either pass: the kernels give up and report."""
    ops = g.Ops(0)
    x, w, targets, dloss = make(300, 256, 5000, torch.float16)
    lse = g.linear_cross_entropy(x, w, targets, save=True)[1]
    ops.set_watchdog(timeout_ns=50_000_000, skip_k_block=1)
    for call in (lambda: ops.linear_cross_entropy(x, w, targets),
                 lambda: ops.linear_cross_entropy(x[:5], w[:200], targets[:5].clamp(0, 199)),
                 lambda: ops.linear_cross_entropy_backward(dloss, x, w, targets, lse)):
        call()
        with pytest.raises(g.GemmError) as e:
            ops.check_error()
        assert e.value.status == 5
    ops.set_watchdog()
    assert torch.equal(ops.linear_cross_entropy(x, w, targets), g.linear_cross_entropy(x, w, targets))
    ops.check_error()
    ops.close()
