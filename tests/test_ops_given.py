"""An object given as `ops` takes every call, the norms' among them: a subclass or a
wrapper sees all operators alike.  No kernel is launched."""
import pytest
import torch

import dense_fp16_gemm_04_gb300 as g

X, W = torch.zeros(4, 64), torch.zeros(64)
# Function, its arguments, what the method gets.
CALLS = {
    "gated_ffn": ((X, W, W), (X, W, W, "silu", False, None, None)),
    "gated_ffn_backward": ((X, X, W, W, X), (X, X, W, W, X, "silu", None)),
    "w4_linear": ((X, W, W), (X, W, W, None, None, None)),
    "w4_gated": ((X, W, W), (X, W, W, None, "silu", None, None)),
    "orthogonalize": ((X,), (X, 5, g.NEWTON_SCHULZ, 1e-7, None, None, None)),
    "layer_norm": ((X, W, W), (X, W, W, 1e-5, False, None, None)),
    "layer_norm_backward": ((X, X, W, X), (X, X, W, X, True, None)),
    "rms_norm": ((X, W), (X, W, 1e-6, False, None, None)),
    "rms_norm_backward": ((X, X, W, X), (X, X, W, X, None)),
    "linear_cross_entropy": ((X, X, W), (X, X, W, -100, False, None, None)),
    "linear_cross_entropy_backward": ((W, X, X, W, W), (W, X, X, W, W, -100, None, None)),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_given_handle_takes_the_call(name):
    class Seen:
        def __getattr__(self, method):
            return lambda *args: (method, args)

    args, want = CALLS[name]
    method, got = getattr(g, name)(*args, ops=Seen())
    assert method == name and len(got) == len(want)
    assert all(a is b or a == b for a, b in zip(got, want))
    # The order of the method's own parameters is the one that the function passes on.
    code = getattr(g.Ops, name).__code__
    assert code.co_argcount - 1 == len(want)
