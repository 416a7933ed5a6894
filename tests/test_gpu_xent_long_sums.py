"""The products of the vocabulary's loss over sums of many terms: dx, dW, logits of wide rows.

The tensor cores truncate a sum, always towards zero, at each step of 16 products, by at
most 2^-23 of what it has come to.  Sums of at most 8192 products stand in one accumulator
(512 steps), of logits at most 512; such parts are added in fp32.  For dx and dW logits are
all 0, so that every probability is a power of two and dz is exact in 16 bits, and the sums
come to large values on the way to small results: what truncation loses is seen whole, where
the rounding of an ordinary result would cover it."""
import math

import pytest
import torch

from test_gpu_xent import make, run

pytestmark = pytest.mark.gpu

F64 = torch.float64
PART, STEP = 8192, 16
U16 = 2.0 ** -11


@pytest.fixture(scope="module")
def g():
    import dense_fp16_gemm_04_gb300 as m
    m.build()
    return m


def near_one(gen, *shape):
    """fp16 within 2^-6 of 1."""
    t = torch.empty(*shape, dtype=torch.float16, device="cuda")
    for part in t.split(max(1, 2 ** 27 // shape[1])):
        part.copy_(1 + (torch.rand(part.shape, generator=gen, device="cuda") - 0.5) / 32)
    return t


# (T, D, V): pairs of CTAs; clusters of two pairs, of two, four and eight CTAs; shares of the
# vocabulary by lone CTAs and by pairs; pieces of it.
@pytest.mark.parametrize("T,D,V", [(1024, 4096, 2 ** 18), (333, 4096, 2 ** 15), (100, 8192, 2 ** 15), (3, 4096, 2 ** 16),
                                   (128, 1024, 2 ** 13), (40, 256, 2 ** 18), (300, 2056, 2 ** 18), (1000, 520, 2 ** 17),
                                   (5000, 512, 2 ** 17), (20000, 136, 2 ** 16)])
def test_dx_over_a_long_vocabulary(g, T, D, V):
    """dz is 1 / V, and -1 for the target (1 / V - 1 rounded): dx is the sum of the other rows
    of W over V, less the target's."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    w = near_one(gen, V, D)
    x = torch.zeros(T, D, dtype=torch.float16, device="cuda")
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda")
    targets[0] = 0
    loss, lse = g.linear_cross_entropy(x, w, targets, save=True)
    assert (lse.to(F64) - math.log(V)).abs().max() <= 2 ** -20
    dx, dw = g.linear_cross_entropy_backward(torch.ones(T, device="cuda"), x, w, targets, lse)
    g.default_ops().check_error()
    assert not dw.any()
    ref = sum(p.to(F64).sum(0) for p in w.split(2 ** 14)) / V - (1 + 1 / V) * w[targets].to(F64)
    # The target's part stands at 1 or less (and 1/64) throughout; the others, V / 8192 of
    # them, grow to 8192 / V: half of that on average.  Sums of at most 256 parts or shares.
    steps = PART / STEP
    err = 1.02 * (steps * 2.0 ** -23 * (1 + 0.5) + 256 * 2.0 ** -24)
    worst = ((dx.to(F64) - ref).abs() - U16 * (ref.abs() + err)).max().item()
    assert worst <= err, f"off by {worst:.3g}, allowed {err:.3g}"


@pytest.mark.parametrize("T,D,V", [(2 ** 17, 64, 2), (2 ** 17, 2048, 8192), (2 ** 18 + 77, 136, 512)])
def test_dw_of_many_tokens(g, T, D, V):
    """x is near 1 for one half of the tokens and near -1 for the other, W is 0, and entry 0
    is every target: row 0 of dW is (1 / V - 1) sum x, the others are sum x / V."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = near_one(gen, T, D)
    x[T // 2:] *= -1
    w = torch.zeros(V, D, dtype=torch.float16, device="cuda")
    targets = torch.zeros(T, dtype=torch.int64, device="cuda")
    _, lse = g.linear_cross_entropy(x, w, targets, save=True)
    dx, dw = g.linear_cross_entropy_backward(torch.ones(T, device="cuda"), x, w, targets, lse)
    g.default_ops().check_error()
    assert not dx.any()
    total = sum(p.to(F64).sum(0) for p in x.split(2 ** 14))
    first = float(torch.tensor(1 / V - 1).half())  # -1 of 8192 entries
    for row, scale in ((0, abs(first)), (1, 1 / V), (V - 1, 1 / V)):
        ref = (first if row == 0 else 1 / V) * total
        # Each part grows to 8192 scale: half of that on average.  The parts' sums come to
        # T / 2 scale at most.
        parts = T / PART + 1
        err = 1.02 * scale * (parts * PART / STEP * 2.0 ** -23 * PART / 2 + parts * 2.0 ** -24 * T / 2)
        worst = ((dw[row].to(F64) - ref).abs() - U16 * (ref.abs() + err) - 2.0 ** -25).max().item()
        assert worst <= err, f"row {row}: off by {worst:.3g}, allowed {err:.3g}"


@pytest.mark.parametrize("D,V,ctas", [(2 ** 20, 1000, 8), (2 ** 18, 4000, 4), (2 ** 18, 9000, 2)])
def test_logits_of_very_wide_rows(g, D, V, ctas):
    """One token, all products near 1, so that logits grow to D: clusters of CTAs share the
    rows, each a k-range."""
    gen = torch.Generator(device="cuda").manual_seed(D)
    x, w = near_one(gen, 1, D), near_one(gen, V, D)
    _, lse = g.linear_cross_entropy(x, w, torch.zeros(1, dtype=torch.int64, device="cuda"), save=True)
    g.default_ops().check_error()
    z = torch.cat([p.to(F64) @ x[0].to(F64) for p in w.split(2 ** 26 // D)])
    ref = torch.logsumexp(z, 0)
    # Parts of 512 products grow to 528: half of that on average.  A CTA's parts are added up
    # to its share of D, the CTAs' sums to D.  The lse itself is rounded a few times.
    top, share, part = 1.04 * D, 1.04 * D / ctas, 512
    err = (D / part * (part / STEP) * 2.0 ** -23 * 528 / 2 + D / part * 2.0 ** -24 * share / 2
           + ctas * 2.0 ** -24 * top + 4 * 2.0 ** -24 * top)
    off = (lse[0].to(F64) - ref).abs().item()
    assert off <= 1.02 * err, f"off by {off:.3g}, allowed {1.02 * err:.3g}"


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T,D,V", [(3, 8200, 5000), (1, 16392, 4000), (20, 65536, 700), (130, 8328, 4099)])
def test_wide_rows(g, T, D, V, dt):
    x, w, targets, dloss = make(T, D, V, dt, seed=D)
    run(g, x, w, targets, dloss, 0.3 * dloss)


@pytest.mark.parametrize("T,D,V", [(600, 4096, 16384), (9000, 128, 256), (5, 16392, 4000)])
def test_stuck_waits_of_long_sums_end(g, T, D, V):
    """A k-block that is never loaded, in products of long sums: the kernels give up and
    report, and the next call is right."""
    ops = g.Ops(0)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, D, generator=gen, device="cuda").half()
    w = (torch.randn(V, D, generator=gen, device="cuda") * D ** -0.5).half()
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda")
    dloss = torch.ones(T, device="cuda")
    _, lse = g.linear_cross_entropy(x, w, targets, save=True)
    ops.set_watchdog(timeout_ns=50_000_000, skip_k_block=1)
    for call in (lambda: ops.linear_cross_entropy_backward(dloss, x, w, targets, lse),
                 lambda: ops.linear_cross_entropy(x, w, targets)):
        call()
        with pytest.raises(g.GemmError) as e:
            ops.check_error()
        assert e.value.status == 5
    ops.set_watchdog()
    assert torch.equal(ops.linear_cross_entropy(x, w, targets, save=True)[1], lse)
    got = ops.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    ops.check_error()
    want = g.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(got, want))
    ops.close()
