"""The loss's gradients at the ends of their ranges: dz of more than 2^31 elements, and the
smallest entries that fp16's dz holds."""
import pytest
import torch

from test_gpu_xent import backward_ref, check, make, sum_eps

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(scope="module")
def g():
    import dense_fp16_gemm_04_gb300 as m
    m.build()
    return m


def test_dz_of_more_than_2_to_31_elements(g):
    """Tokens with a gradient are packed side by side, so that only those reach far: their dz
    alone has 2.29e9 elements, of which rows 524288 and on start past 2^31 and 2^32 bytes."""
    T, D, V = 700_000, 64, 4096
    x, w, targets, dloss = make(T, D, V, torch.bfloat16, seed=11)
    dloss = dloss * T
    live = torch.nonzero(targets >= 0)[:, 0]
    assert len(live) * V > 2 ** 31
    _, lse = g.linear_cross_entropy(x, w, targets, save=True)
    dx, dw = g.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    g.default_ops().check_error()
    # Packed rows around 2^31 elements, around 2^32 bytes (the same row), and the last ones.
    pick = torch.cat((live[:200], live[524_188:524_388], live[-300:], live[torch.randint(524_288, len(live), (1000,), device="cuda")]))
    rx, _ = backward_ref(dloss[pick], None, x[pick], w, targets[pick], lse[pick], x.dtype)
    check(dx[pick], *rx, "dx")
    assert not dx[targets < 0].any()
    ref, err = torch.zeros(V, D, dtype=F64, device="cuda"), torch.zeros(V, D, dtype=F64, device="cuda")
    part = 30_000
    for a in range(0, T, part):
        b = slice(a, a + part)
        _, (r, e) = backward_ref(dloss[b], None, x[b], w, targets[b], lse[b], x.dtype)
        ref += r
        err += e
    # (each part's bound has sum_eps of its own tokens; the sums of all of them pass on as many times more)
    check(dw, ref, err + sum_eps(T) / sum_eps(part) * err, "dw")


@pytest.mark.parametrize("top", [1.0, 1.99])
def test_fp16_dz_reaches_to_2_to_minus_38_of_the_largest(g, top):
    """Beside a token with the largest dloss, others 2^-30 to 2^-38 of it: dz of their targets
    is off by at most 2^-38 of the largest, and none above that is lost."""
    D = V = 64
    dt = torch.float16
    scale = 2.0 ** 14 * top
    ratios = torch.tensor([1.0] + [2.0 ** -k for k in range(30, 38)] + [1.0625 * 2.0 ** -38], device="cuda")
    T = len(ratios)
    w = torch.eye(V, D, device="cuda").to(dt)
    x = torch.zeros(T, D, device="cuda", dtype=dt)
    x[:, D - 1] = -16.0  # the last entry's probability is 1e-9, the others' 1 / 63
    targets = torch.arange(T, device="cuda")
    _, lse = g.linear_cross_entropy(x, w, targets, save=True)
    dx, _ = g.linear_cross_entropy_backward(scale * ratios, x, w, targets, lse)
    # W is the identity: dx is dz, of the target -(1 - 1 / 63) dloss.
    got = dx[targets, targets].to(F64)
    want = -(1 - 1 / 63) * scale * ratios.to(F64)
    half = 2.0 ** -25 + 2.0 ** -11 * want.abs()  # of dx's own rounding
    assert ((got - want).abs() <= 1.01 * (2.0 ** -38 * scale + 2.0 ** -11 * want.abs() + half)).all()
    assert (got < 0).all()
