"""Host-side checks of the norms and the loss: functions without a handle, tensors off the GPU
or of a graph, and objects that are no tensors are refused.  No kernel is launched."""
import ctypes

import pytest
import torch

import dense_fp16_gemm_04_gb300 as g
from test_ops_host import Unbound, workspace


@pytest.fixture(scope="module")
def lib():
    g.build()
    return g.load()


def h(*s):
    return torch.zeros(*s, dtype=torch.float16)


def f(*s):
    return torch.zeros(*s)


def test_null_handles_are_refused(lib):
    p, l, i, e, z = ctypes.c_void_p(), ctypes.c_int64(8), ctypes.c_int(0), ctypes.c_float(1e-5), ctypes.c_size_t(0)
    assert lib.gemm_layer_norm(p, p, l, p, p, p, l, p, l, l, e, i, i, p) == 1
    assert lib.gemm_rms_norm(p, p, l, p, p, l, p, l, l, e, i, i, p) == 1
    assert lib.gemm_layer_norm_backward(p, p, l, p, l, p, p, p, l, p, p, p, z, l, l, i, i, p) == 1
    assert lib.gemm_rms_norm_backward(p, p, l, p, l, p, p, p, l, p, p, z, l, l, i, i, p) == 1
    assert lib.gemm_linear_cross_entropy(p, p, l, p, l, p, p, p, p, z, l, l, l, l, i, p) == 1
    assert lib.gemm_linear_cross_entropy_backward(p, p, l, p, l, p, l, p, l, p, p, p, l, p, p, z, l, l, l, l, i, p) == 1
    for name, n in (("gemm_norm_backward_workspace", 2), ("gemm_linear_cross_entropy_workspace", 3),
                    ("gemm_linear_cross_entropy_backward_workspace", 3)):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_size_t
        assert fn(p, *[l] * n) == 0


def test_norm_workspaces(lib):
    """fp32 sums of the weight's and the bias's gradients for each block of rows; none
    for refused lengths."""
    top = 2 ** 31 - 4096
    for T, D in ((1, 1), (1, 8192), (16384, 64), (8192, 16384), (top, 8), (1, top)):
        n = workspace("gemm_norm_backward_workspace", T, D)
        assert n >= 8 * D and n % (8 * D) == 0 and n <= 8 * D * min(T, 4096)
    for sizes in ((0, 8), (8, 0), (top + 1, 8), (8, top + 1), (2 ** 62, 2 ** 62)):
        assert workspace("gemm_norm_backward_workspace", *sizes) == 0


def test_loss_workspaces(lib):
    """Forward: a maximum and a sum of each token for every 64 entries at least, of as
    many tokens as 512 MB hold (256 at least).  Backward: 16-bit dz of the whole
    vocabulary or of a piece, a copy of x, and fp32 sums of dx where dz is in pieces."""
    top = 2 ** 31 - 4096
    fwd = lambda *s: workspace("gemm_linear_cross_entropy_workspace", *s)
    bwd = lambda *s: workspace("gemm_linear_cross_entropy_backward_workspace", *s)
    for T, V in ((1, 1), (1, 32000), (300, 5000), (4096, 131072), (10 ** 6, 131072), (top, 2 ** 28)):
        n = min(T, 16384)
        assert fwd(T, 64, V) >= 8 * -(-V // 128) * min(n, 256)
        assert fwd(T, 64, V) <= max(2 ** 29, 32 * (V + 64) * 256) + 8 * 1216 * n + 4 * n + 1024
    for T, D, V in ((1, 8, 1), (300, 64, 5000), (4096, 4096, 131072), (10 ** 6, 64, 10 ** 5), (top, 2 ** 24, 2 ** 28)):
        piece = min(V, 4096)
        assert bwd(T, D, V) >= 2 * T * (D + piece)
        assert bwd(T, D, V) <= 2 * T * (D + 64 + min(V + 256, max(4096, 2 ** 28 // T) + 256)) + 4 * T * D + 20 * T + 2 ** 25
    assert fwd(300, 136, 9000) - fwd(300, 128, 9000) == 300 * 192 * 2  # a copy of x in whole lines
    for sizes in ((0, 8, 8), (8, 0, 8), (8, 8, 0), (top + 1, 8, 8), (8, 2 ** 24 + 1, 8), (8, 8, 2 ** 28 + 1), (2 ** 62,) * 3):
        assert fwd(*sizes) == 0 and bwd(*sizes) == 0


def calls(x, o):
    return (lambda: o.layer_norm(x, h(64), h(64)), lambda: o.rms_norm(x),
            lambda: o.layer_norm_backward(h(4, 64), x, h(64), f(4, 2)),
            lambda: o.rms_norm_backward(h(4, 64), x, h(64), f(4, 1)),
            lambda: o.linear_cross_entropy(x, h(100, 64), torch.zeros(4, dtype=torch.int64)),
            lambda: o.linear_cross_entropy_backward(f(4), x, h(100, 64), torch.zeros(4, dtype=torch.int64), f(4)))


def test_cpu_tensors_are_refused(lib):
    for o in (g, Unbound()):
        for call in calls(h(4, 64), o):
            with pytest.raises(ValueError, match="CUDA"):
                call()


def test_tensors_that_ask_for_a_graph_are_refused(lib):
    import torch.autograd.forward_ad as fw
    o = Unbound()
    for call in calls(torch.nn.Parameter(h(4, 64)), o):
        with pytest.raises(RuntimeError, match="requires grad"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call()
    with fw.dual_level():
        for call in calls(fw.make_dual(h(4, 64), h(4, 64)), o):
            with pytest.raises(RuntimeError, match="tangent"):
                call()


@pytest.mark.parametrize("other", [None, [1.0, 2.0], 3])
def test_operands_that_are_not_tensors_are_refused(lib, other):
    for o in (g, Unbound()):
        for call in calls(other, o):
            with pytest.raises(TypeError):
                call()


def test_other_types_are_refused(lib):
    o = Unbound()
    for call in calls(torch.zeros(4, 64, dtype=torch.float64), o):
        with pytest.raises(TypeError):
            call()
