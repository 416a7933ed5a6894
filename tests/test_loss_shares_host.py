"""When dx of the vocabulary's loss is summed in shares: read from the size of the
workspace, which holds T x D fp32 sums of each.  No kernel is launched."""
import subprocess
import sys

import pytest

import dense_fp16_gemm_04_gb300 as g
from test_ops_host import ROOT

# A stand-in for a handle: device, SMs, clusters of pairs, of two pairs and of 1, 2, 4 and 8
# CTAs that fit at once.
SIZE = """
import ctypes, sys
import dense_fp16_gemm_04_gb300 as g
h = (ctypes.c_int32 * 256)(0, 152, 76, 36, 152, 76, 36, 15)
fn = g.load().gemm_linear_cross_entropy_backward_workspace
fn.restype = ctypes.c_size_t
print(fn(h, *map(ctypes.c_int64, map(int, sys.argv[1:]))))
"""


def up(v, m):
    return -(-v // m) * m


def shares(T, D, V):
    r = subprocess.run([sys.executable, "-c", SIZE, str(T), str(D), str(V)], cwd=ROOT, capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    rest = up(16 * T, 256) + 256 + up(4 * T, 256) + up(2 * T * up(D, 64), 256) + up(2 * T * up(V, 64), 256)
    n, left = divmod(int(r.stdout) - rest, 4 * T * D)
    assert left < 256
    return n


@pytest.mark.parametrize("T,D,V,want", [
    (4, 1288, 66557, 13),       # 11 tiles of a lone CTA: 152 SMs hold 13 of each
    (128, 1032, 8191, 16),      # nine tiles, shares of eight k-blocks
    (128, 1024, 8000, 0),       # eight tiles: clusters of eight CTAs take no longer
    (100, 512, 6000, 0),
    (1, 4096, 32000, 0),        # clusters of four
    (1000, 1032, 20011, 3),     # 20 tiles of a pair of CTAs: three of each run at once
    (1024, 4096, 131072, 0),    # tiles enough
])
def test_dx_in_shares_where_that_takes_the_least_time(T, D, V, want):
    g.build()
    assert shares(T, D, V) == want
