"""The loss's gradients at the ends of their ranges: the smallest entries that
fp16's dz holds."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(scope="module")
def g():
    import dense_fp16_gemm_04_gb300 as m
    m.build()
    return m


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
