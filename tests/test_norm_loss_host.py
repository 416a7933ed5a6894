"""Host-side checks of the norms: functions without a handle, tensors off the GPU
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
    fn = lib.gemm_norm_backward_workspace
    fn.restype = ctypes.c_size_t
    assert fn(p, l, l) == 0


def test_norm_workspaces(lib):
    """fp32 sums of the weight's and the bias's gradients for each block of rows; none
    for refused lengths."""
    top = 2 ** 31 - 4096
    for T, D in ((1, 1), (1, 8192), (16384, 64), (8192, 16384), (top, 8), (1, top)):
        n = workspace("gemm_norm_backward_workspace", T, D)
        assert n >= 8 * D and n % (8 * D) == 0 and n <= 8 * D * min(T, 4096)
    for sizes in ((0, 8), (8, 0), (top + 1, 8), (8, top + 1), (2 ** 62, 2 ** 62)):
        assert workspace("gemm_norm_backward_workspace", *sizes) == 0


def calls(x, o):
    return (lambda: o.layer_norm(x, h(64), h(64)), lambda: o.rms_norm(x),
            lambda: o.layer_norm_backward(h(4, 64), x, h(64), f(4, 2)),
            lambda: o.rms_norm_backward(h(4, 64), x, h(64), f(4, 1)))


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
