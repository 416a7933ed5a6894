"""The operators at the limits of their arguments: empty sums, infinities and
values near the types' largest, the longest rows, and what is refused there.
Bounds as in test_gpu_ops.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import dense_fp16_gemm_04_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("T", [1, 5, 40])
def test_ffn_of_empty_rows_keeps_zeros(g, T):
    """D = 0: g and u are empty sums, whatever their memory held before."""
    dt, F = torch.float16, 128
    junk = torch.full((T, 2 * F), float("nan"), dtype=dt, device="cuda")
    del junk  # the next allocation of this size gets its memory
    y, gu = g.gated_ffn(torch.empty(T, 0, dtype=dt, device="cuda"), torch.empty(2 * F, 0, dtype=dt, device="cuda"),
                        torch.empty(0, F, dtype=dt, device="cuda"), save=True)
    assert y.shape == (T, 0) and gu.shape == (T, 2 * F) and not gu.any()
    assert g.gated_ffn(torch.empty(T, 0, dtype=dt, device="cuda"), torch.empty(0, 0, dtype=dt, device="cuda"),
                       torch.empty(0, 0, dtype=dt, device="cuda"), save=True)[1].shape == (T, 0)
