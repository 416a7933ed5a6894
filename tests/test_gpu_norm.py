"""Layer norm, RMS norm and their gradients against their definitions in 64 bits.

Tolerances are bounds, computed per element.  A value rounded to type t is off by
at most u = eps(t) / 2 of itself (fp16 below its normal range: 2^-25).  An fp32 sum
is off by at most 2^-24 of the sum of its terms' magnitudes for every addition that
a term goes through: over a row, n / 256 in its thread, then shuffles and warps
(at most 64); over T rows at most T and then as many blocks as there are (at most
T + 64 in all)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F64 = torch.float64
TYPES = [(torch.float16, torch.float16), (torch.float16, torch.float32), (torch.bfloat16, torch.bfloat16),
         (torch.bfloat16, torch.float32), (torch.float32, torch.float32)]
IDS = ["f16", "f16_f32", "bf16", "bf16_f32", "f32"]
E = 2.0 ** -24


@pytest.fixture(scope="module")
def g():
    import dense_fp16_gemm_04_gb300 as m
    m.build()
    return m


def u(dt):
    return torch.finfo(dt).eps / 2


def row_eps(n):
    return (n / 256 + 64) * E


def check(got, ref, err, what):
    dt = got.dtype
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
    bound = 1.01 * (err + u(dt) * (ref.abs() + err)) + tiny + 1e-37
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = ((got.to(F64) - ref).abs() / bound).max().item() if got.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"


def make(T, D, dt, wt, seed=0, offset=0.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    def r(*s):
        return torch.randn(*s, generator=gen, device="cuda")
    x = (r(T, D) * torch.exp(r(T, 1)) + offset * r(1, D)).to(dt)
    return x, (1 + 0.3 * r(D)).to(wt), (0.5 * r(D)).to(wt), r(T, D).to(dt)


def forward_ref(x, weight, bias, eps, rms):
    """y, its error, the statistics and theirs."""
    x = x.to(F64)
    n = x.shape[1]
    en = row_eps(n)
    m = torch.zeros_like(x[:, :1]) if rms else x.mean(1, keepdim=True)
    c = x - m
    var = c.square().mean(1, keepdim=True)
    r = 1 / (var + eps).sqrt()
    # The first pass's mean is off by e1; the second takes all but its own error back.
    e1 = torch.zeros_like(m) if rms else en * x.abs().mean(1, keepdim=True)
    off = c.abs().mean(1, keepdim=True) + e1
    ec = torch.zeros_like(m) if rms else (en + 2 * E) * off
    ev = 2 * E * (c.abs() + e1) + ec
    er = r * (0.5 * ((en + 4 * E) * (var + e1 ** 2) + 4 * (e1 + ec) * ec) / (var + eps) + 4 * E)
    h = c * r
    eh = r * ev + c.abs() * er + 2 * E * h.abs()
    w = weight.to(F64) if weight is not None else torch.ones(n, dtype=F64, device="cuda")
    b = bias.to(F64) if bias is not None else torch.zeros(n, dtype=F64, device="cuda")
    y = h * w + b
    return y, eh * w.abs() + 2 * E * ((h * w).abs() + b.abs()), (m, ec + E * e1, r, er)


def check_stats(stats, ref, rms):
    m, em, r, er = ref
    if not rms:
        check(stats[:, :1], m, em, "mean")
    check(stats[:, -1:], r, er, "reciprocal deviation")


def backward_ref(dy, x, weight, stats, rms):
    x, dy, stats = x.to(F64), dy.to(F64), stats.to(F64)
    T, n = x.shape
    en = row_eps(n)
    r = stats[:, -1:]
    h = (x - (0 if rms else stats[:, :1])) * r
    w = weight.to(F64) if weight is not None else torch.ones(n, dtype=F64, device="cuda")
    q = dy * w
    c1 = torch.zeros_like(r) if rms else q.mean(1, keepdim=True)
    c2 = (q * h).mean(1, keepdim=True)
    e1 = 0 if rms else (en + 2 * E) * q.abs().mean(1, keepdim=True)
    e2 = (en + 6 * E) * (q * h).abs().mean(1, keepdim=True)
    dx = r * (q - c1 - h * c2)
    edx = r * (4 * E * (q.abs() + c1.abs()) + 6 * E * (h * c2).abs() + e1 + h.abs() * e2) + 4 * E * dx.abs()
    rows = (T + 64) * E
    dw, edw = (dy * h).sum(0), (rows + 4 * E) * (dy * h).abs().sum(0)
    return (dx, edx), (dw, edw), (dy.sum(0), rows * dy.abs().sum(0))


def run(g, x, weight, bias, eps, rms, out=None):
    if rms:
        return g.rms_norm(x, weight, eps=eps, save=True, out=out)
    return g.layer_norm(x, weight, bias, eps=eps, save=True, out=out)


def back(g, dy, x, weight, stats, rms):
    if rms:
        return g.rms_norm_backward(dy, x, weight, stats)
    return g.layer_norm_backward(dy, x, weight, stats)


# Rows of one element, of less than a warp, around a load of 8 and a row's threads,
# off every vector, and longer than registers or shared memory hold.
SHAPES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 31), (1, 33), (9, 64), (17, 100), (33, 255), (2, 256), (6, 264),
          (130, 520), (64, 1000), (3, 1003), (7, 1024), (40, 1032), (5, 2048), (300, 2056), (2, 4096), (19, 4100),
          (1, 8192), (6, 8200), (700, 96), (1025, 1280), (2, 16384), (3, 16392), (2, 20001), (1, 65536), (2, 70008),
          (1, 300001), (50, 130), (9, 1002), (40, 4098), (3, 8190), (7, 12346), (2, 16386), (300, 66)]


@pytest.mark.parametrize("rms", [False, True], ids=["ln", "rms"])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)), ids=[f"{t}x{d}" for t, d in SHAPES])
def test_norm(g, i, shape, types, rms):
    T, D = shape
    x, weight, bias, dy = make(T, D, *types, seed=i)
    eps = 1e-5 if D > 2 else 1e-2
    if i % 4 == 1:
        weight = bias = None
    elif i % 4 == 3:
        bias = None
    out = torch.full((T, D), float("nan"), dtype=x.dtype, device="cuda")
    y, stats = run(g, x, weight, bias, eps, rms, out)
    assert y.data_ptr() == out.data_ptr()
    ref, err, sref = forward_ref(x, weight, None if rms else bias, eps, rms)
    check(y, ref, err, "y")
    assert stats.shape == (T, 1 if rms else 2) and stats.dtype == torch.float32
    check_stats(stats, sref, rms)
    kw = {} if rms else {"bias": bias}
    assert torch.equal((g.rms_norm if rms else g.layer_norm)(x, weight, eps=eps, **kw), y)
    got = back(g, dy, x, weight, stats, rms)
    refs = backward_ref(dy, x, weight, stats, rms)
    check(got[0], *refs[0], "dx")
    if weight is None:
        assert got[1] is None
    else:
        assert got[1].dtype == weight.dtype
        check(got[1], *refs[1], "dweight")
    if not rms:
        check(got[2], *refs[2], "dbias")
        assert g.layer_norm_backward(dy, x, weight, stats, bias=False)[2] is None
    for a, b in zip(got, back(g, dy, x, weight, stats, rms)):
        assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("rms", [False, True], ids=["ln", "rms"])
@pytest.mark.parametrize("D", [50, 1024, 3001, 5000])
def test_norm_against_differences(g, D, rms):
    """<gradient, v> against central differences of the 64-bit loss, along the
    gradient itself; the gradient is fp32 and off by far less than 1e-4 of itself
    (its bound above is), the differences by eps^2 of a smooth function."""
    x, weight, bias, dy = make(11, D, torch.float32, torch.float32, seed=D)
    _, stats = run(g, x, weight, bias, 1e-5, rms)
    grads = back(g, dy, x, weight, stats, rms)
    base = [t.to(F64) for t in ((x, weight) if rms else (x, weight, bias))]
    def loss(xx, ww, bb=0.0):
        c = xx if rms else xx - xx.mean(1, keepdim=True)
        return ((c / (c.square().mean(1, keepdim=True) + 1e-5).sqrt() * ww + bb) * dy.to(F64)).sum()
    for i, gr in enumerate(grads):
        v = gr.to(F64) / gr.to(F64).norm()
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + 1e-4 * v, base[i] - 1e-4 * v
        num, ana = (loss(*hi) - loss(*lo)) / 2e-4, (gr.to(F64) * v).sum()
        assert abs(num - ana) <= 1e-4 * ana.abs(), (i, num.item(), ana.item())


@pytest.mark.parametrize("rms", [False, True], ids=["ln", "rms"])
@pytest.mark.parametrize("D", [40, 1000, 1024, 1026, 4104, 33000])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_norm_strided_rows_from_any_element(g, types, D, rms):
    T = 6
    x, weight, bias, dy = make(T, D, *types, seed=1)
    y0, stats = run(g, x, weight, bias, 1e-5, rms)
    want = back(g, dy, x, weight, stats, rms)
    ref, err, _ = forward_ref(x, weight, None if rms else bias, 1e-5, rms)
    refs = backward_ref(dy, x, weight, stats, rms)
    for start, extra in ((8, 16), (1, 2), (3, 8), (8, 13), (2, 4)):
        def pad(t):
            big = torch.full((T, D + start + extra), float("nan"), dtype=t.dtype, device="cuda")
            v = big[:, start:start + D]
            v.copy_(t)
            return v
        def moved(t):
            b = torch.empty(D + start, dtype=t.dtype, device="cuda")
            b[start:] = t
            return b[start:]
        big = torch.full((T, D + start + extra), 7.0, dtype=x.dtype, device="cuda")
        y, st = run(g, pad(x), moved(weight), moved(bias), 1e-5, rms, big[:, start:start + D])
        assert (big[:, :start] == 7).all() and (big[:, start + D:] == 7).all()
        check(y, ref, err, "y")  # whatever path the alignment takes
        got = back(g, pad(dy), pad(x), moved(weight), stats, rms)
        for a, r in zip(got, refs):
            check(a, *r, "gradient")
    assert torch.isfinite(want[0]).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.float16])
def test_layer_norm_far_from_zero(g, dt):
    """A mean a thousand times the deviation: the second pass keeps the result to
    the bound, which does not grow with the mean's own rounding."""
    for D in (64, 1000, 4096, 40000):
        x, weight, bias, _ = make(5, D, torch.float32, torch.float32, seed=D, offset=0.0)
        x = (x / x.std(1, keepdim=True) + 1000.0).to(dt)
        y, stats = g.layer_norm(x, weight.to(dt), bias.to(dt), save=True)
        ref, err, sref = forward_ref(x, weight.to(dt), bias.to(dt), 1e-5, False)
        check(y, ref, err, "y")
        check_stats(stats, sref, False)
        assert (err / (ref.abs() + 1)).median() < 1e-4


@pytest.mark.parametrize("rms", [False, True], ids=["ln", "rms"])
def test_norm_constant_and_zero_rows(g, rms):
    x = torch.zeros(4, 1000, dtype=torch.bfloat16, device="cuda")
    x[1] = 3.0
    x[2, 17] = 1e30
    x[3] = 1e-30
    weight = torch.full((1000,), 2.0, dtype=torch.bfloat16, device="cuda")
    y, stats = run(g, x, weight, None, 1e-5, rms)
    ref, err, _ = forward_ref(x[[0, 1, 3]], weight, None, 1e-5, rms)
    check(y[[0, 1, 3]], ref, err + 2 * E * 3.0, "y")
    assert not y[0].any()
    if not rms:
        assert not y[1].any()
    dx = back(g, torch.ones_like(x), x, weight, stats, rms)[0]
    assert torch.isfinite(dx[[0, 1, 3]]).all()


@pytest.mark.parametrize("rms", [False, True], ids=["ln", "rms"])
@pytest.mark.parametrize("D", [100, 1024, 4096, 20001])
def test_norm_non_finite_rows_stay_in_their_rows(g, D, rms):
    x, weight, bias, dy = make(9, D, torch.float16, torch.float16)
    y0, stats0 = run(g, x, weight, bias, 1e-5, rms)
    x2 = x.clone()
    x2[3, D // 2], x2[5, 1] = float("nan"), float("inf")
    y, stats = run(g, x2, weight, bias, 1e-5, rms)
    keep = torch.tensor([0, 1, 2, 4, 6, 7, 8], device="cuda")
    assert torch.equal(y[keep], y0[keep]) and torch.equal(stats[keep], stats0[keep])
    assert torch.isnan(y[3]).all() and torch.isnan(y[5, 1]) and (rms or torch.isnan(y[5]).all())
    dx, dx0 = back(g, dy, x2, weight, stats, rms)[0], back(g, dy, x, weight, stats0, rms)[0]
    assert torch.equal(dx[keep], dx0[keep])


def test_norm_empty(g):
    x = torch.empty(0, 48, dtype=torch.float16, device="cuda")
    w = torch.ones(48, dtype=torch.float16, device="cuda")
    y, stats = g.layer_norm(x, w, w, save=True)
    assert y.shape == (0, 48) and stats.shape == (0, 2)
    dx, dw, db = g.layer_norm_backward(x, x, w, stats)
    assert dx.shape == (0, 48) and not dw.any() and not db.any() and dw.shape == db.shape == (48,)
    with pytest.raises(g.GemmError) as e:
        g.rms_norm(torch.empty(4, 0, dtype=torch.float16, device="cuda"))
    assert e.value.status == 1


@pytest.mark.parametrize("shape", [(66000, 40), (140000, 16), (20000, 264)])
def test_norm_many_rows(g, shape):
    T, D = shape
    x, weight, bias, dy = make(T, D, torch.bfloat16, torch.float32, seed=3)
    y, stats = g.layer_norm(x, weight, bias, save=True)
    ref, err, sref = forward_ref(x, weight, bias, 1e-5, False)
    check(y, ref, err, "y")
    check_stats(stats, sref, False)
    for a, r in zip(g.layer_norm_backward(dy, x, weight, stats), backward_ref(dy, x, weight, stats, False)):
        check(a, *r, "gradient")


def test_norm_past_two_gigaelements(g):
    """Rows whose offsets pass 32 bits, through the distance between them."""
    T, D = 5, 264
    big = torch.zeros(T, 2 ** 29 + 8, dtype=torch.float16, device="cuda")
    x, weight, bias, dy = make(T, D, torch.float16, torch.float16)
    v = big[:, 8:8 + D]
    v.copy_(x)
    y, stats = g.layer_norm(v, weight, bias, save=True)
    y0, stats0 = g.layer_norm(x, weight, bias, save=True)
    assert torch.equal(y, y0) and torch.equal(stats, stats0)
    for a, b in zip(g.layer_norm_backward(dy, v, weight, stats), g.layer_norm_backward(dy, x, weight, stats)):
        assert torch.equal(a, b)


def test_norm_of_more_than_two_gigaelements(g):
    T, D = 300_000, 8192
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    for part in x.split(30_000):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
    weight = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
    y, stats = g.rms_norm(x, weight, save=True)
    pick = torch.cat((torch.arange(100, device="cuda"), torch.arange(262_100, 262_200, device="cuda"),
                      torch.arange(T - 100, T, device="cuda")))
    ref, err, sref = forward_ref(x[pick], weight, None, 1e-6, True)
    check(y[pick], ref, err, "y")
    check_stats(stats[pick], sref, True)
    dx, dw = g.rms_norm_backward(y, x, weight, stats)
    check(dx[pick], *backward_ref(y[pick], x[pick], weight, stats[pick], True)[0], "dx")
    ref, err = torch.zeros(D, dtype=F64, device="cuda"), torch.zeros(D, dtype=F64, device="cuda")
    for a in range(0, T, 15_000):
        b = slice(a, a + 15_000)
        h = x[b].to(F64) * stats[b].to(F64)
        ref += (y[b].to(F64) * h).sum(0)
        err += (T + 64) * E * (y[b].to(F64) * h).abs().sum(0)
    check(dw, ref, err, "dweight")


# ------------------------------------------------------------ streams, graphs --
def test_norm_streams_and_graphs(g):
    x, weight, bias, dy = make(300, 1032, torch.bfloat16, torch.float32)
    def all_(stream=None):
        y, stats = g.layer_norm(x, weight, bias, save=True, stream=stream)
        z, st = g.rms_norm(x, weight, save=True, stream=stream)
        return (y, stats, z, st, *g.layer_norm_backward(dy, x, weight, stats, stream=stream),
                *g.rms_norm_backward(dy, x, weight, st, stream=stream))
    want = [t.clone() for t in all_()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = all_(stream)
        trash = [torch.full((n,), float("nan"), device="cuda") for n in (1 << k for k in range(6, 22)) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del trash
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_()
    for t in got:
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_norm_refusals(g):
    x, weight, bias, dy = make(4, 64, torch.float16, torch.float16)
    _, stats = g.layer_norm(x, weight, bias, save=True)
    for call in (lambda: g.layer_norm(x, weight[:32]), lambda: g.layer_norm(x, None, bias),
                 lambda: g.layer_norm(x, weight, bias[:1]), lambda: g.layer_norm(x[0], weight),
                 lambda: g.layer_norm(x, weight.cpu()), lambda: g.layer_norm(x.t(), weight),
                 lambda: g.layer_norm(x, torch.ones(128, device="cuda")[::2]),
                 lambda: g.layer_norm(x, weight, out=torch.empty(4, 63, dtype=x.dtype, device="cuda")),
                 lambda: g.layer_norm_backward(dy[:3], x, weight, stats),
                 lambda: g.layer_norm_backward(dy, x, weight, stats[:, :1]),
                 lambda: g.rms_norm_backward(dy, x, weight, stats)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: g.layer_norm(x.double()), lambda: g.layer_norm(x, weight.bfloat16()),
                 lambda: g.layer_norm(x, weight, bias.float()), lambda: g.rms_norm(x, 1.0),
                 lambda: g.layer_norm_backward(dy.float(), x, weight, stats),
                 lambda: g.layer_norm_backward(dy, x, weight, stats.double()),
                 lambda: g.layer_norm(x, eps="a")):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: g.layer_norm(x, weight, out=x), lambda: g.layer_norm(x, eps=-1.0),
                 lambda: g.layer_norm(x, eps=float("nan"))):
        with pytest.raises(g.GemmError) as e:
            call()
        assert e.value.status == 1
