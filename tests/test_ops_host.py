"""Host-side checks of the operators: the header compiles as C99 and every
function it declares is exported, null handles and tensors off the GPU are
refused, and quantised codes decode to the nearest levels.  No kernel is
launched."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import dense_fp16_gemm_04_gb300 as g

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_ops.h")


@pytest.fixture(scope="module")
def lib():
    g.build()
    return g.load()


def declared():
    return re.findall(r"GEMM_API\s+[\w\s\*]+?\b(gemm_\w+)\s*\(", open(HEADER).read())


def test_header_compiles_as_c99(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "gemm_ops.h"\nint main(void) { return (int)GEMM_ACT_SILU; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                    os.path.join(ROOT, "include"), "-c", str(src), "-o", str(tmp_path / "h.o")], check=True)


def test_every_declared_function_is_exported(lib):
    names = declared()
    assert {"gemm_ops_create", "gemm_gated_ffn", "gemm_gated_ffn_backward", "gemm_w4_linear",
            "gemm_w4_gated", "gemm_orthogonalize"} <= set(names)
    raw = ctypes.CDLL(g.LIB_PATH)
    assert [n for n in names if not hasattr(raw, n)] == []


def test_null_handles_are_refused(lib):
    vp = ctypes.c_void_p
    assert lib.gemm_ops_create(None, 0) == 1
    assert lib.gemm_ops_destroy(None) == 0
    assert lib.gemm_ops_check_error(None) == 1
    assert lib.gemm_ops_set_watchdog(None, 0, -1) == 1
    assert lib.gemm_ops_launch_count(None) == 0
    i64, z = ctypes.c_int64, ctypes.c_size_t
    for name, n_sizes in (("gemm_gated_ffn_workspace", 3), ("gemm_gated_ffn_backward_workspace", 3),
                          ("gemm_orthogonalize_workspace", 3)):
        fn = getattr(lib, name)
        fn.restype = z
        assert fn(vp(), *[i64(8)] * n_sizes) == 0
    p, l, s, i = vp(), i64(8), z(0), ctypes.c_int(0)
    assert lib.gemm_gated_ffn(p, p, l, p, l, p, l, p, l, p, p, s, l, l, l, i, i, p) == 1
    assert lib.gemm_gated_ffn_backward(p, p, l, p, l, p, l, p, l, p, p, l, p, p, p, s, l, l, l, i, i, p) == 1
    assert lib.gemm_w4_linear(p, p, l, p, p, p, p, l, p, s, l, l, l, i64(32), i, p) == 1
    assert lib.gemm_w4_gated(p, p, l, p, p, p, p, l, p, s, l, l, l, i64(32), i, i, p) == 1


def test_cpu_tensors_are_refused(lib):
    x = torch.zeros(4, 64, dtype=torch.float16)
    w_in, w_down = torch.zeros(256, 64, dtype=torch.float16), torch.zeros(64, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        g.gated_ffn(x, w_in, w_down)
    with pytest.raises(ValueError):
        g.gated_ffn_backward(x, x, w_in, w_down, torch.zeros(4, 256, dtype=torch.float16))
    with pytest.raises(ValueError):
        g.w4_linear(x, torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.float16))
    with pytest.raises(ValueError):
        g.orthogonalize(torch.zeros(4, 4))


@pytest.mark.parametrize("zero_point", [False, True])
@pytest.mark.parametrize("group", [32, 64, 256])
def test_quantised_codes_are_the_nearest_levels(group, zero_point):
    """Every code is the best of the sixteen for its group's scale and zero point
    (among equally near ones, any), and a group's ends are reached."""
    gen = torch.Generator().manual_seed(group)
    w = torch.randn(6, 512, generator=gen).to(torch.float16)
    codes, scales, zeros = g.w4_quantize(w, group, zero_point)
    assert codes.shape == (6, 256) and codes.dtype == torch.uint8
    assert scales.shape == (6, 512 // group) and scales.dtype == w.dtype
    assert (zeros is None) == (not zero_point)
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(1).double()
    z = (zeros.double() if zero_point else torch.full_like(scales, 8).double()).repeat_interleave(group, 1)
    s = scales.double().repeat_interleave(group, 1)
    err = ((q - z) * s - w.double()).abs()
    levels = ((torch.arange(16).double().view(16, 1, 1) - z) * s - w.double()).abs().amin(0)
    # Dividing by the scale in fp32 may take either of two levels a rounding apart.
    assert (err <= levels + 16 * s * 2.0 ** -23).all()


def test_quantise_refusals():
    w = torch.zeros(4, 96, dtype=torch.float16)
    for group in (16, 48, 64):
        with pytest.raises(ValueError):
            g.w4_quantize(w, group)
    codes, scales, _ = g.w4_quantize(w, 32)
    assert (codes == 0x88).all() and (scales == 0).all()


# Sizes of workspaces depend on the handle's number of SMs alone (its second
# word): a stand-in for a handle does where there is no device.
SIZES = """
import ctypes, sys
import dense_fp16_gemm_04_gb300 as g
h = (ctypes.c_int32 * 256)(0, 152)
fn = getattr(g.load(), sys.argv[1])
fn.restype = ctypes.c_size_t
print(fn(h, *map(ctypes.c_int64, map(int, sys.argv[2:]))))
"""


def workspace(name, *sizes):
    """The size that a function returns, in a process of its own: what it does
    wrong may end the process."""
    r = subprocess.run([sys.executable, "-c", SIZES, name, *map(str, sizes)], cwd=ROOT, capture_output=True, text=True,
                       timeout=60)
    assert r.returncode == 0, (name, sizes, r.returncode, r.stderr)
    return int(r.stdout)


@pytest.mark.parametrize("K", [1, 31, 33, 4095])
def test_w4_workspace_of_rows_without_whole_groups(lib, K):
    """No group divides K: the product refuses it, and its workspace is 0 bytes
    (rows of K = 1 have no bytes to divide by)."""
    for gated in (0, 1):
        assert workspace("gemm_w4_workspace", 1, 8, K, gated) == 0
        assert workspace("gemm_w4_workspace", 16, 8, 32 * 512, gated) > 0


def test_workspaces_of_refused_lengths(lib):
    """Lengths past the limits: 0 bytes at once, not a plan for them."""
    top = 2 ** 31 - 4096
    for name in ("gemm_gated_ffn_workspace", "gemm_gated_ffn_backward_workspace"):
        assert workspace(name, 1, 8, 8) > 0 and workspace(name, 1, top, 8) > 0
        for sizes in ((1, 2 ** 40, 8), (1, top + 1, 8), (2 ** 62, 8, 8), (16, 8, 2 ** 30), (16, 2 ** 62, 2 ** 62)):
            assert workspace(name, *sizes) == 0, (name, sizes)
    for sizes in ((8 * 65535 + 1, 1, 4096, 0), (2 ** 62, 1, 4096, 1), (16, 1, 2 ** 40, 0)):
        assert workspace("gemm_w4_workspace", *sizes) == 0, sizes


@pytest.mark.parametrize("T", [1, 8, 16])
def test_w4_longest_rows_fit_a_grid(lib, T):
    """K is cut into as many slices as a grid's second dimension holds, at most:
    their sums' workspace is 4 bytes per slice, token and column."""
    for K in (2 ** 28, 2 ** 28 - 32, 2 ** 27, 3 * 2 ** 25):
        for gated in (0, 1):
            assert workspace("gemm_w4_workspace", T, 1, K, gated) <= 65535 * T * 4 * (1 + gated)


class Unbound:
    """The operators' methods on no handle: what the binding refuses before it needs one."""
    def __init__(self):
        from dense_fp16_gemm_04_gb300 import ops
        self._b, self._addr, self.index, self._ops = ops._load_binding(), 0, 0, ops.Ops

    def __getattr__(self, name):
        return getattr(self._ops, name).__get__(self)


def test_tensors_that_ask_for_a_graph_are_refused(lib):
    """Not answered without one; under no_grad they go on to the next check (the
    device)."""
    import torch.autograd.forward_ad as fw
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)
    o, codes = Unbound(), torch.zeros(8, 32, dtype=torch.uint8)
    calls = (lambda x: o.gated_ffn(x, h(256, 64), h(64, 128)),
             lambda x: o.gated_ffn_backward(h(4, 64), x, h(256, 64), h(64, 128), h(4, 256)),
             lambda x: o.w4_linear(x, codes, h(8, 2)), lambda x: o.w4_gated(x, codes, h(8, 2)))
    for call in calls:
        with pytest.raises(RuntimeError, match="requires grad"):
            call(torch.nn.Parameter(h(4, 64)))
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call(torch.nn.Parameter(h(4, 64)))
        with fw.dual_level(), pytest.raises(RuntimeError, match="tangent"):
            call(fw.make_dual(h(4, 64), h(4, 64)))
    with pytest.raises(RuntimeError, match="requires grad"):
        o.orthogonalize(torch.zeros(4, 4, requires_grad=True))


def test_quantised_weights_leave_the_graph():
    codes, scales, zeros = g.w4_quantize(torch.nn.Parameter(torch.ones(4, 64)), 32, zero_point=True)
    assert not (codes.requires_grad or scales.requires_grad or zeros.requires_grad)


@pytest.mark.parametrize("other", [None, [1.0, 2.0], 3])
def test_operands_that_are_not_tensors_are_refused(lib, other):
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)
    codes = torch.zeros(8, 32, dtype=torch.uint8)
    o = Unbound()
    for call in (lambda: g.gated_ffn(other, h(256, 64), h(64, 128)), lambda: g.w4_linear(other, codes, h(8, 2)),
                 lambda: g.w4_gated(other, codes, h(8, 2)), lambda: g.orthogonalize(other),
                 lambda: g.gated_ffn_backward(h(4, 64), other, h(256, 64), h(64, 128), h(4, 256)),
                 lambda: o.gated_ffn(other, h(256, 64), h(64, 128)), lambda: o.orthogonalize(other)):
        with pytest.raises(TypeError):
            call()
