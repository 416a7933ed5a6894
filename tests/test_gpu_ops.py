"""The operators beside the GEMM against their definitions in 64 bits: the
gated block, its backward pass, the 4-bit products and the orthogonalised
update, at the sizes and layouts where each can go wrong.

Tolerances are bounds, computed per element from the operands: a value rounded
to 16 bits is off by at most u = 2^-11 (fp16) or 2^-8 (bf16) of itself, and an
fp32 sum of K products by at most K 2^-23 of the sum of their magnitudes (the
tensor cores may truncate where IEEE addition rounds).  fp16 results below the
normal range are off by up to 2^-25 instead."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
F64 = torch.float64
DTYPES = [torch.float16, torch.bfloat16]
ACTS = ["silu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module")
def g():
    import dense_fp16_gemm_04_gb300 as m
    m.build()
    return m


def sum_eps(K):
    return (K + 16) * 2.0 ** -23


def act_ref(act, v):
    """act(v), act'(v) and how far fast exponentials may put them off."""
    if act == "relu":
        return v.clamp_min(0), (v > 0).to(v.dtype), torch.zeros_like(v)
    k = math.sqrt(2 / math.pi)
    p = v if act == "silu" else 2 * k * (v + 0.044715 * v ** 3)
    dp = torch.ones_like(v) if act == "silu" else 2 * k * (1 + 3 * 0.044715 * v ** 2)
    s = torch.sigmoid(p)
    # exp's argument is off by 2^-23 |p|, the quotient by a few ulps.
    return v * s, s + v * dp * s * (1 - s), (p.abs() + 8) * 2.0 ** -22


def gated_ref(x, w_in, act, dt):
    """h, its error before rounding, and g, u with theirs."""
    F, K = w_in.shape[0] // 2, x.shape[1]
    p = x.to(F64) @ w_in.to(F64).t()
    e = sum_eps(K) * (x.to(F64).abs() @ w_in.to(F64).abs().t())
    gv, uv, eg, eu = p[:, :F], p[:, F:], e[:, :F], e[:, F:]
    a, da, ea = act_ref(act, gv)
    # |act'| and its change are below 2 on every branch.
    err_a = 2 * eg + a.abs() * ea
    return a * uv, err_a * (uv.abs() + eu) + a.abs() * eu, p, e


def check(got, ref, err, dt, what):
    d = (got.to(F64) - ref).abs()
    bound = 1.01 * (err + U[dt] * (ref.abs() + err)) + TINY[dt] + 1e-30
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = (d / bound).max().item() if d.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"


def make_ffn(T, D, F, dt, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    def r(*s):
        return torch.randn(*s, generator=gen, device="cuda")
    return (r(T, D).to(dt), (r(2 * F, D) * D ** -0.5).to(dt), (r(D, F) * F ** -0.5).to(dt), r(T, D).to(dt))


def run_ffn(g, x, w_in, w_down, act, dt, save=True):
    ops = g.default_ops()
    out = torch.full((x.shape[0], x.shape[1]), float("nan"), dtype=dt, device="cuda")
    y = g.gated_ffn(x, w_in, w_down, act=act, save=save, out=out)
    y, gu = y if save else (y, None)
    ops.check_error()
    assert y.data_ptr() == out.data_ptr()
    h, eh, p, ep = gated_ref(x, w_in, act, dt)
    if save:
        check(gu, p, ep, dt, "gu")
    wd = w_down.to(F64)
    eh = eh + U[dt] * (h.abs() + eh) + TINY[dt]
    err = eh @ wd.abs().t() + sum_eps(h.shape[1]) * ((h.abs() + eh) @ wd.abs().t())
    check(y, h @ wd.t(), err, dt, "y")
    return y, gu


# Tokens around the streaming kernels' tiles of 8 and 16, the split tiles of
# 128 rows and the pair's 256; dimensions off every tile.
FFN_SHAPES = [(1, 8, 8), (1, 256, 512), (3, 136, 264), (8, 1024, 1000), (9, 520, 72), (16, 64, 2048),
              (17, 512, 1024), (33, 1000, 520), (127, 264, 640), (129, 1032, 392), (200, 2048, 1536),
              (257, 136, 4096), (700, 328, 1048), (1030, 1024, 2056), (2500, 520, 3080)]


@pytest.mark.parametrize("dt", DTYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("i,shape", list(enumerate(FFN_SHAPES)), ids=[f"{t}x{d}x{f}" for t, d, f in FFN_SHAPES])
def test_ffn(g, i, shape, dt):
    x, w_in, w_down, _ = make_ffn(*shape, dt, seed=i)
    run_ffn(g, x, w_in, w_down, ACTS[i % 3], dt)


@pytest.mark.parametrize("T", [1, 12, 40, 300])
def test_ffn_without_saving_is_the_same(g, T):
    x, w_in, w_down, _ = make_ffn(T, 520, 776, torch.float16)
    a, _ = g.gated_ffn(x, w_in, w_down, save=True)
    b = g.gated_ffn(x, w_in, w_down)
    assert torch.equal(a, b)


@pytest.mark.parametrize("T", [2, 24, 600])
def test_ffn_strided_rows(g, T):
    D, F, dt = 264, 392, torch.float16
    x, w_in, w_down, dy = make_ffn(T, D, F, dt)
    def pad(t, extra):
        big = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device="cuda")
        v = big[:, 8:8 + t.shape[1]]
        v.copy_(t)
        return v
    y, gu = run_ffn(g, pad(x, 24), pad(w_in, 16), pad(w_down, 40), "silu", dt)
    y0, gu0 = g.gated_ffn(x, w_in, w_down, save=True)
    assert torch.equal(y, y0) and torch.equal(gu, gu0)
    out = torch.full((T, D + 16), 7.0, dtype=dt, device="cuda")
    g.gated_ffn(x, w_in, w_down, out=out[:, 8:8 + D])
    assert torch.equal(out[:, 8:8 + D], y0)
    assert (out[:, :8] == 7).all() and (out[:, 8 + D:] == 7).all()
    for a, b in zip(g.gated_ffn_backward(pad(dy, 8), pad(x, 24), pad(w_in, 16), pad(w_down, 40), gu),
                    g.gated_ffn_backward(dy, x, w_in, w_down, gu)):
        assert torch.equal(a, b)


def ffn_backward_ref(dy, x, w_in, w_down, gu, act, dt):
    F = w_down.shape[1]
    T, D = x.shape
    d, wd, wi, xd = dy.to(F64), w_down.to(F64), w_in.to(F64), x.to(F64)
    gv, uv = gu[:, :F].to(F64), gu[:, F:].to(F64)
    a, da, ea = act_ref(act, gv)
    dh = d @ wd
    edh = sum_eps(D) * (d.abs() @ wd.abs())
    dgu = torch.cat((dh * uv * da, dh * a), 1)
    # The slope is a sum of terms up to 1 + |a p'|: fast exponentials put it off by ea of those.
    k = 1.6
    eda = ea * (1 + a.abs() * (1 if act == "silu" else k * (1 + 0.14 * gv ** 2)))
    edgu = torch.cat((edh * (uv * da).abs() + (dh.abs() + edh) * uv.abs() * eda,
                      edh * a.abs() + (dh.abs() + edh) * a.abs() * ea), 1) + 2.0 ** -21 * dgu.abs()
    edgu = edgu + U[dt] * (dgu.abs() + edgu) + TINY[dt]
    h = a * uv
    eh = h.abs() * (ea + 2.0 ** -21 + U[dt]) * 1.01 + TINY[dt]
    def prod(p, ep, q, K):
        return p @ q, ep @ q.abs() + sum_eps(K) * ((p.abs() + ep) @ q.abs())
    dx = prod(dgu, edgu, wi, 2 * F)
    dwi = prod(dgu.t(), edgu.t(), xd, T)
    dwd_t = prod(h.t(), eh.t(), d, T)
    return dx, dwi, (dwd_t[0].t(), dwd_t[1].t())


@pytest.mark.parametrize("dt", DTYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("i,shape", list(enumerate(FFN_SHAPES)), ids=[f"{t}x{d}x{f}" for t, d, f in FFN_SHAPES])
def test_ffn_backward(g, i, shape, dt):
    x, w_in, w_down, dy = make_ffn(*shape, dt, seed=100 + i)
    act = ACTS[(i + 1) % 3]
    gu = (x @ w_in.t())
    got = g.gated_ffn_backward(dy, x, w_in, w_down, gu, act=act)
    g.default_ops().check_error()
    for name, o, (ref, err) in zip(("dx", "dw_in", "dw_down"), got,
                                   ffn_backward_ref(dy, x, w_in, w_down, gu, act, dt)):
        check(o, ref, err, dt, name)


@pytest.mark.parametrize("act", ACTS)
def test_ffn_backward_against_differences(g, act):
    """<grad, v> against central differences of the 64-bit loss along v.  16-bit
    rounding of dg, du, h and the result: a few u of the gradient's own size,
    which a direction along the gradient itself does not magnify."""
    dt = torch.float16
    x, w_in, w_down, dy = make_ffn(60, 136, 200, dt, seed=5)
    _, gu = g.gated_ffn(x, w_in, w_down, act=act, save=True)
    grads = g.gated_ffn_backward(dy, x, w_in, w_down, gu, act=act)
    def loss(xx, wi, wd):
        p = xx @ wi.t()
        a = act_ref(act, p[:, :200])[0]
        return ((a * p[:, 200:]) @ wd.t() * dy.to(F64)).sum()
    base = [x.to(F64), w_in.to(F64), w_down.to(F64)]
    for i, gr in enumerate(grads):
        v = gr.to(F64) / gr.to(F64).norm()
        eps = 1e-4
        hi, lo = [list(base) for _ in range(2)]
        hi[i], lo[i] = base[i] + eps * v, base[i] - eps * v
        num = (loss(*hi) - loss(*lo)) / (2 * eps)
        ana = (gr.to(F64) * v).sum()
        assert abs(num - ana) <= 8 * U[dt] * ana.abs(), (act, i, num.item(), ana.item())


def test_ffn_empty(g):
    dt = torch.float16
    x, w_in, w_down, dy = make_ffn(0, 64, 128, dt)
    y, gu = g.gated_ffn(x, w_in, w_down, save=True)
    assert y.shape == (0, 64) and gu.shape == (0, 256)
    dx, dwi, dwd = g.gated_ffn_backward(dy, x, w_in, w_down, gu)
    assert dx.shape == (0, 64) and not dwi.any() and not dwd.any()
    x, w_in, w_down, dy = (torch.randn(5, 64, device="cuda").to(dt), torch.empty(0, 64, dtype=dt, device="cuda"),
                           torch.empty(64, 0, dtype=dt, device="cuda"), torch.randn(5, 64, device="cuda").to(dt))
    assert not g.gated_ffn(x, w_in, w_down).any()
    assert not g.gated_ffn_backward(dy, x, w_in, w_down, torch.empty(5, 0, dtype=dt, device="cuda"))[0].any()


@pytest.mark.parametrize("T", [4, 50, 400])
def test_ffn_non_finite_rows_stay_in_their_rows(g, T):
    dt = torch.float16
    x, w_in, w_down, _ = make_ffn(T, 264, 520, dt)
    y0 = g.gated_ffn(x, w_in, w_down)
    x2 = x.clone()
    x2[T // 2, 3] = float("nan")
    x2[T - 1, 5] = float("inf")
    y = g.gated_ffn(x2, w_in, w_down)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[T // 2] = keep[T - 1] = False
    assert torch.equal(y[keep], y0[keep])
    assert torch.isnan(y[T // 2]).all() and not torch.isfinite(y[T - 1]).any()


# ------------------------------------------------------------ 4-bit weights --
def make_w4(T, rows, K, group, zeros, dt, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, K, generator=gen, device="cuda").to(dt)
    codes = torch.randint(0, 256, (rows, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = (torch.randn(rows, K // group, generator=gen, device="cuda") * K ** -0.5).to(dt)
    z = torch.randint(0, 16, (rows, K // group), generator=gen, device="cuda", dtype=torch.uint8) if zeros else None
    return x, codes, scales, z


def w4_ref(codes, scales, zeros):
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(1).to(F64)
    G = q.shape[1] // scales.shape[1]
    z = zeros.to(F64).repeat_interleave(G, 1) if zeros is not None else 8.0
    return (q - z) * scales.to(F64).repeat_interleave(G, 1)


W4_SHAPES = [(1, 1, 32, 32), (1, 16, 128, 128), (1, 17, 96, 32), (2, 100, 320, 64), (5, 33, 1024, 128),
             (8, 257, 2048, 64), (9, 48, 4096, 256), (16, 1000, 160, 32), (17, 64, 512, 128),
             (50, 40, 1984, 64), (1, 5000, 256, 256), (3, 31, 8192, 8192)]


@pytest.mark.parametrize("dt", DTYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("i,shape", list(enumerate(W4_SHAPES)), ids=["x".join(map(str, s)) for s in W4_SHAPES])
def test_w4(g, i, shape, gated, dt):
    T, N, K, G = shape
    x, codes, scales, z = make_w4(T, 2 * N if gated else N, K, G, i % 2 == 1, dt, seed=i)
    w = w4_ref(codes, scales, z)
    out = torch.full((T, N + 3), float("nan"), dtype=dt, device="cuda")[:, 1:1 + N]
    if not gated:
        got = g.w4_linear(x, codes, scales, z, out=out)
        check(got, x.to(F64) @ w.t(), sum_eps(K) * (x.to(F64).abs() @ w.abs().t()), dt, "y")
        return
    act = ACTS[i % 3]
    got = g.w4_gated(x, codes, scales, z, act=act, out=out)
    h, eh, _, _ = gated_ref(x, w, act, dt)
    check(got, h, eh, dt, "h")


def test_w4_columns_are_exact(g):
    """One-hot x picks single weights: exact products, one rounding."""
    K, N = 256, 48
    _, codes, scales, z = make_w4(1, N, K, 32, True, torch.float16)
    x = torch.eye(K, device="cuda", dtype=torch.float16)
    got = g.w4_linear(x, codes, scales, z)
    assert torch.equal(got, w4_ref(codes, scales, z).t().to(torch.float16))


def test_w4_strided_x_and_empty(g):
    x, codes, scales, z = make_w4(3, 40, 256, 64, True, torch.float16)
    big = torch.full((3, 256 + 24), float("nan"), dtype=torch.float16, device="cuda")
    big[:, 8:264] = x
    assert torch.equal(g.w4_linear(big[:, 8:264], codes, scales, z), g.w4_linear(x, codes, scales, z))
    assert g.w4_linear(x[:0], codes, scales, z).shape == (0, 40)
    e = torch.empty(3, 0, dtype=torch.float16, device="cuda")
    y = g.w4_linear(e, torch.empty(40, 0, dtype=torch.uint8, device="cuda"), torch.empty(40, 0, dtype=torch.float16, device="cuda"))
    assert y.shape == (3, 40) and not y.any()


@pytest.mark.parametrize("zero_point", [False, True])
def test_w4_quantize(g, zero_point):
    """Rounding to the nearest of a group's levels: off by at most half a step,
    plus what rounding the scale to 16 bits moves the outermost level by."""
    w = torch.randn(70, 512, device="cuda").to(torch.float16)
    w[3] = 0
    codes, scales, zeros = g.w4_quantize(w, 64, zero_point)
    d = (w4_ref(codes, scales, zeros) - w.to(F64)).abs().reshape(70, 8, 64)
    s = scales.to(F64).unsqueeze(-1)
    assert (d <= (1.0 if zero_point else 0.5) * s * 1.001 + 16 * s * U[torch.float16]).all()
    assert torch.isfinite(scales).all()


# ------------------------------------------------------ orthogonalised update --
COEFFS = (3.4445, -4.7750, 2.0315)


def ns_ref(m, steps, coeffs, eps):
    a, b, c = coeffs
    x = m.to(F64)
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    norms = [x.square().sum((-2, -1)).sqrt()]
    for _ in range(steps):
        if x.shape[-2] <= x.shape[-1]:
            p = x @ x.mT
            x = a * x + (b * p + c * p @ p) @ x
        else:
            p = x.mT @ x
            x = a * x + x @ (b * p + c * p @ p)
        norms.append(x.square().sum((-2, -1)).sqrt())
    # A step leaves X off by at most about 2^-18 of its norm: two parts keep 22
    # bits, dropping low times low costs 2^-22, the sums about 2^-20, each three
    # times over and weighed by |b| s + |c| s^3 <= 4.  Later steps magnify that
    # by at most a.
    err = sum(2.0 ** -18 * n * a ** (steps - i) for i, n in enumerate(norms))
    return x, err


NS_SHAPES = [(1, 1), (1, 7), (9, 1), (5, 3), (64, 64), (100, 40), (128, 256), (129, 257), (300, 1000),
             (1000, 300), (513, 511), (1024, 1024), (2100, 1100)]


@pytest.mark.parametrize("i,shape", list(enumerate(NS_SHAPES)), ids=[f"{m}x{n}" for m, n in NS_SHAPES])
@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
def test_orthogonalize(g, i, shape, src):
    gen = torch.Generator(device="cuda").manual_seed(i)
    M, N = shape
    m = (torch.randn(M, N, generator=gen, device="cuda") * 10.0 ** (i % 5 - 2)).to(src)
    ref, err = ns_ref(m, 5, COEFFS, 1e-7)
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        o = g.orthogonalize(m, dtype=dt)
        g.default_ops().check_error()
        assert o.dtype == dt and torch.isfinite(o).all()
        d = (o.to(F64) - ref).norm()
        bound = err + (U[dt] if dt in U else 0) * ref.norm()
        assert d <= bound, (dt, d.item(), bound.item())


@pytest.mark.parametrize("shape", [(3, 40, 72), (4, 200, 136), (2, 600, 600)])
def test_orthogonalize_batch_is_each_matrix(g, shape):
    m = torch.randn(*shape, device="cuda")
    m[1] = 0
    o = g.orthogonalize(m)
    assert not o[1].any()
    for b in range(shape[0]):
        assert torch.equal(o[b], g.orthogonalize(m[b]))


def test_orthogonalize_strided_transposed_sizes(g):
    big = torch.randn(200, 331, device="cuda")
    v = big[3:103, 5:182]
    a = g.orthogonalize(v.contiguous())
    out = torch.full((100, 190), 5.0, device="cuda")
    g.orthogonalize(v, out=out[:, 7:184])
    assert torch.equal(out[:, 7:184], a)
    assert (out[:, :7] == 5).all() and (out[:, 184:] == 5).all()
    # The transposed matrix has the transposed result.
    t = g.orthogonalize(v.t().contiguous())
    assert (t.t() - a).norm() <= 2 * ns_ref(v, 5, COEFFS, 1e-7)[1]


def test_orthogonalize_steps_and_empty(g):
    m = torch.randn(30, 50, device="cuda")
    x0 = g.orthogonalize(m, steps=0)
    assert (x0 - m / (m.norm() + 1e-7)).abs().max() <= 2.0 ** -20
    ref, err = ns_ref(m, 3, (1.5, -0.5, 0.0), 0.0)
    assert (g.orthogonalize(m, steps=3, coeffs=(1.5, -0.5, 0.0), eps=0.0).to(F64) - ref).norm() <= err
    assert g.orthogonalize(m[:0]).shape == (0, 50)
    assert g.orthogonalize(torch.empty(0, 3, 4, device="cuda")).shape == (0, 3, 4)


# ------------------------------------------------------------ streams, refusals --
def test_ops_follow_the_current_stream(g):
    x, w_in, w_down, dy = make_ffn(300, 256, 512, torch.float16)
    want = g.gated_ffn(x, w_in, w_down)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x2 = torch.zeros_like(x)
        torch.cuda._sleep(20_000_000)
        x2.copy_(x)
        y = g.gated_ffn(x2, w_in, w_down)
    s.synchronize()
    assert torch.equal(y, want)
    assert torch.equal(g.gated_ffn(x, w_in, w_down, stream=s).cpu() if s.synchronize() is None else None,
                       want.cpu())


def test_ops_in_a_graph(g):
    x, w_in, w_down, dy = make_ffn(40, 256, 512, torch.float16)
    xm, codes, scales, z = make_w4(2, 64, 256, 64, True, torch.float16)
    m = torch.randn(100, 60, device="cuda")
    def all_():
        y, gu = g.gated_ffn(x, w_in, w_down, save=True)
        return (y, *g.gated_ffn_backward(dy, x, w_in, w_down, gu), g.w4_linear(xm, codes, scales, z),
                g.orthogonalize(m))
    want = [t.clone() for t in all_()]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = all_()
    for t in got:
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_ops_are_deterministic(g):
    x, w_in, w_down, dy = make_ffn(100, 2048, 4096, torch.bfloat16)
    y, gu = g.gated_ffn(x, w_in, w_down, save=True)
    first = (y, gu, *g.gated_ffn_backward(dy, x, w_in, w_down, gu))
    for _ in range(3):
        y, gu = g.gated_ffn(x, w_in, w_down, save=True)
        for a, b in zip(first, (y, gu, *g.gated_ffn_backward(dy, x, w_in, w_down, gu))):
            assert torch.equal(a, b)


def test_watchdog_ends_a_stuck_wait(g):
    """A k-block that is never loaded: the kernel gives up, reports and leaves
    the context usable."""
    ops = g.Ops(0)
    x, w_in, w_down, _ = make_ffn(300, 256, 512, torch.float16)
    ops.set_watchdog(timeout_ns=50_000_000, skip_k_block=1)
    ops.gated_ffn(x, w_in, w_down)
    with pytest.raises(g.GemmError) as e:
        ops.check_error()
    assert e.value.status == 5 and ops.last_error_detail()[0] == 5
    ops.set_watchdog()
    assert torch.equal(ops.gated_ffn(x, w_in, w_down), g.gated_ffn(x, w_in, w_down))
    ops.check_error()
    ops.close()


def test_refusals(g):
    dt = torch.float16
    x, w_in, w_down, dy = make_ffn(4, 64, 128, dt)
    _, gu = g.gated_ffn(x, w_in, w_down, save=True)
    with pytest.raises(ValueError):
        g.gated_ffn(x, w_in, w_down, act="tanh")
    with pytest.raises(ValueError):
        g.gated_ffn(x, w_in[:128], w_down)
    with pytest.raises(ValueError):
        g.gated_ffn(x, w_in.cpu(), w_down)
    with pytest.raises(ValueError):
        g.gated_ffn(x.cpu(), w_in, w_down)
    with pytest.raises(ValueError):
        g.gated_ffn(x.t().contiguous().t(), w_in, w_down)
    with pytest.raises(TypeError):
        g.gated_ffn(x.float(), w_in, w_down)
    with pytest.raises(TypeError):
        g.gated_ffn(x, w_in.bfloat16(), w_down)
    with pytest.raises(g.GemmError) as e:  # D = 60
        g.gated_ffn(x[:, :60], w_in[:, :60], w_down[:60])
    assert e.value.status == 2
    with pytest.raises(g.GemmError) as e:  # the output over the input
        g.gated_ffn(x, w_in, w_down, out=x)
    assert e.value.status == 1
    with pytest.raises(ValueError):
        g.gated_ffn_backward(dy, x, w_in, w_down, gu[:, :-8])
    xm, codes, scales, z = make_w4(2, 64, 256, 64, True, dt)
    with pytest.raises(ValueError):
        g.w4_linear(xm[:, :128], codes, scales, z)
    with pytest.raises(g.GemmError) as e:  # a group of 16
        g.w4_linear(xm, codes, torch.zeros(64, 16, dtype=dt, device="cuda"))
    assert e.value.status == 1
    with pytest.raises(ValueError):
        g.w4_gated(xm, codes[:63], scales[:63])
    with pytest.raises(TypeError):
        g.w4_linear(xm, codes.int(), scales)
    with pytest.raises(ValueError):
        g.orthogonalize(torch.zeros(3, device="cuda"))
    with pytest.raises(TypeError):
        g.orthogonalize(torch.zeros(3, 3, device="cuda", dtype=torch.int32))
    with pytest.raises(ValueError):
        g.orthogonalize(torch.zeros(3, 4, device="cuda").t())


# ---------------------------------------------- shared tiles, batches, long offsets --
# 256 x 256 tiles just past a round of 76 pairs: their k-blocks are shared out.
@pytest.mark.parametrize("shape", [(2817, 1096, 2104), (1300, 4104, 2056)])
def test_ffn_shared_tiles(g, shape):
    T, D, F = shape
    dt = torch.float16
    x, w_in, w_down, dy = make_ffn(T, D, F, dt, seed=7)
    y, gu = run_ffn(g, x, w_in, w_down, "silu", dt)
    for _ in range(2):
        y2, gu2 = g.gated_ffn(x, w_in, w_down, save=True)
        assert torch.equal(y, y2) and torch.equal(gu, gu2)
    got = g.gated_ffn_backward(dy, x, w_in, w_down, gu)
    g.default_ops().check_error()
    for name, o, (ref, err) in zip(("dx", "dw_in", "dw_down"), got,
                                   ffn_backward_ref(dy, x, w_in, w_down, gu, "silu", dt)):
        check(o, ref, err, dt, name)
    for a, b in zip(got, g.gated_ffn_backward(dy, x, w_in, w_down, gu)):
        assert torch.equal(a, b)


def test_orthogonalize_shared_tiles(g):
    m = torch.randn(3000, 3010, device="cuda")
    ref, err = ns_ref(m, 2, COEFFS, 1e-7)
    o = g.orthogonalize(m, steps=2)
    g.default_ops().check_error()
    assert (o.to(F64) - ref).norm() <= err
    both = g.orthogonalize(torch.stack((m, 2 * m)), steps=2)
    assert torch.equal(both[0], o) and torch.equal(both[0], both[1])  # twice m is the same after scaling


@pytest.mark.parametrize("shape", [(7, 130, 300), (20, 64, 64), (5, 900, 1000), (3, 1200, 500), (40, 128, 70)])
def test_orthogonalize_larger_batches(g, shape):
    m = torch.randn(*shape, device="cuda")
    o = g.orthogonalize(m)
    for b in (0, 1, shape[0] - 1):
        assert torch.equal(o[b], g.orthogonalize(m[b]))
        ref, err = ns_ref(m[b], 5, COEFFS, 1e-7)
        assert (o[b].to(F64) - ref).norm() <= err


def test_w4_scales_off_a_word(g):
    """Scales and zero points that start on any element of their allocation."""
    for group in (32, 64, 128):
        x, codes, scales, z = make_w4(3, 50, 256, group, True, torch.float16)
        want = g.w4_linear(x, codes, scales, z)
        for shift in (1, 2, 3):
            def moved(t):
                b = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
                b[shift:] = t.flatten()
                return b[shift:].view(t.shape)
            assert torch.equal(g.w4_linear(x, codes, moved(scales), moved(z)), want)
            assert torch.equal(g.w4_linear(x, codes, moved(scales)), g.w4_linear(x, codes, scales))


@pytest.mark.parametrize("gated", [False, True])
def test_w4_past_four_gigabytes(g, gated):
    """Codes of 5.1 GB: rows past the 32-bit byte offsets of one launch."""
    T, N, K, G = 2, 40000, 262144, 128
    if gated:
        N //= 2
    rows = 2 * N if gated else N
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, K, generator=gen, device="cuda").to(torch.float16)
    codes = torch.randint(0, 256, (rows, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(rows, K // G, generator=gen, device="cuda") * K ** -0.5).to(torch.float16)
    got = g.w4_gated(x, codes, scales) if gated else g.w4_linear(x, codes, scales)
    pick = torch.tensor([0, 1, N // 2, 32767 % N, 32768 % N, N - 2, N - 1], device="cuda")
    if gated:
        sel = torch.cat((pick, pick + N))
        h, eh, _, _ = gated_ref(x, w4_ref(codes[sel], scales[sel], None), "silu", torch.float16)
        check(got[:, pick], h, eh, torch.float16, "h")
    else:
        w = w4_ref(codes[pick], scales[pick], None)
        check(got[:, pick], x.to(F64) @ w.t(), sum_eps(K) * (x.to(F64).abs() @ w.abs().t()), torch.float16, "y")


def test_ffn_past_two_gigaelements(g):
    """gu of 2.3e9 elements: token offsets past 32 bits."""
    T, D, F = 70000, 64, 16640
    x, w_in, w_down, dy = make_ffn(T, D, F, torch.float16)
    y, gu = g.gated_ffn(x, w_in, w_down, save=True)
    pick = torch.tensor([0, 1, 64528, 64529, T - 130, T - 1], device="cuda")
    h, eh, p, ep = gated_ref(x[pick], w_in, "silu", torch.float16)
    check(gu[pick], p, ep, torch.float16, "gu")
    wd = w_down.to(F64)
    eh = eh + U[torch.float16] * (h.abs() + eh) + TINY[torch.float16]
    check(y[pick], h @ wd.t(), eh @ wd.abs().t() + sum_eps(F) * ((h.abs() + eh) @ wd.abs().t()), torch.float16, "y")
    dx, _, _ = g.gated_ffn_backward(dy, x, w_in, w_down, gu)
    ref, err = ffn_backward_ref(dy[pick], x[pick], w_in, w_down, gu[pick], "silu", torch.float16)[0]
    check(dx[pick], ref, err, torch.float16, "dx")


def test_dependent_calls_back_to_back(g):
    """Each call reads what the one before wrote, with nothing waiting between."""
    dt = torch.float16
    x, w_in, w_down, _ = make_ffn(20, 256, 512, dt)
    _, codes, scales, z = make_w4(1, 256, 256, 64, True, dt)
    def chain(sync):
        v = x
        for i in range(20):
            v = g.gated_ffn(v[:4] if i % 3 == 0 else v, w_in, w_down)
            if sync:
                torch.cuda.synchronize()
            v = g.w4_linear(v, codes, scales, z)
            if sync:
                torch.cuda.synchronize()
            v = (v / v.float().norm().to(dt)).repeat(5 if v.shape[0] == 4 else 1, 1)
        return v
    want = chain(True)
    for _ in range(3):
        assert torch.equal(chain(False), want)


def test_example_trains_and_serves(g):
    """examples/gated_block.py: the loss falls, and the 4-bit block answers like
    the 16-bit one but for the rounding of its weights."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_block.py")
    spec = importlib.util.spec_from_file_location("gated_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, w_in, w_down = ex.train(steps=40, tokens=512, dim=128, hidden=256)
    assert torch.isfinite(losses).all() and losses[-1] < 0.5 * losses[0]
    x = torch.randn(3, 128, device="cuda").to(w_in.dtype)
    served = ex.W4Block(w_in, w_down)
    h, eh, _, _ = gated_ref(x, w4_ref(*served.w_in), "silu", torch.float16)
    eh = eh + U[torch.float16] * (h.abs() + eh) + TINY[torch.float16]
    wd = w4_ref(*served.w_down)
    check(served(x), h @ wd.t(), eh @ wd.abs().t() + sum_eps(256) * ((h.abs() + eh) @ wd.abs().t()),
          torch.float16, "served")


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 16, 20])
def test_w4_small_groups_at_every_count(g, T, group, zeros):
    """Small groups are kept apart in one way for a token or two, in another for
    more; an odd number of groups, and even ones that end inside a block of 128
    or with it."""
    for K in (7 * group, 30 * group):
        for dt in DTYPES:
            x, codes, scales, z = make_w4(T, 70, K, group, zeros, dt, seed=T)
            w = w4_ref(codes, scales, z)
            check(g.w4_linear(x, codes, scales, z), x.to(F64) @ w.t(), sum_eps(K) * (x.to(F64).abs() @ w.abs().t()),
                  dt, "y")
            h, eh, _, _ = gated_ref(x, w, "silu", dt)
            check(g.w4_gated(x, codes, scales, z), h, eh, dt, "h")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 4, 7, 16])
def test_w4_single_weights_are_exact(g, T, group):
    """One-hot x, T columns at a time: every code meets its own scale and zero point."""
    K, N = 384, 40
    _, codes, scales, z = make_w4(1, N, K, group, True, torch.bfloat16, seed=T)
    want = w4_ref(codes, scales, z).t().to(torch.bfloat16)
    for x, y in zip(torch.eye(K, device="cuda", dtype=torch.bfloat16).split(T), want.split(T)):
        assert torch.equal(g.w4_linear(x, codes, scales, z), y)


@pytest.mark.parametrize("T", [2, 20])
def test_ffn_infinite_weights_at_the_end_of_rows(g, T):
    """Rows that end inside a block of 32: an infinite weight there gives
    infinity, and does not meet the zeros beyond."""
    D = F = 40
    x = torch.ones(T, D, device="cuda", dtype=torch.float16)
    w_in = torch.full((2 * F, D), 0.01, device="cuda", dtype=torch.float16)
    w_down = torch.full((D, F), 0.01, device="cuda", dtype=torch.float16)
    w_down[5, F - 1] = float("inf")
    y = g.gated_ffn(x, w_in, w_down)
    assert torch.isposinf(y[:, 5]).all() and torch.isfinite(y[:, :5]).all() and torch.isfinite(y[:, 6:]).all()
    w_in[F + 3, D - 1] = float("inf")
    _, gu = g.gated_ffn(x, w_in, w_down, save=True)
    assert torch.isposinf(gu[:, F + 3]).all() and torch.isfinite(gu[:, :F + 3]).all() and torch.isfinite(gu[:, F + 4:]).all()


@pytest.mark.parametrize("act", ACTS)
def test_ffn_backward_of_large_gates(g, act):
    """Gates as large as the type holds: slopes 0 and 1, not NaN."""
    T, D, F = 3, 8, 8
    one = torch.ones(T, D, device="cuda", dtype=torch.bfloat16)
    gu = torch.ones(T, 2 * F, device="cuda", dtype=torch.bfloat16)
    gu[0, :F], gu[1, :F], gu[2, :F] = 1e30, -1e30, -3e38
    w_in = torch.zeros(2 * F, D, device="cuda", dtype=torch.bfloat16)
    w_in[:F] = 1
    w_down = torch.eye(D, F, device="cuda", dtype=torch.bfloat16)
    dx, _, _ = g.gated_ffn_backward(one, one, w_in, w_down, gu, act=act)
    assert torch.equal(dx.float(), torch.tensor([[8.0], [0.0], [0.0]], device="cuda").expand(T, D))


def test_another_stream_owns_what_it_uses(g):
    """With ``stream`` given, workspaces and results come from that stream's
    memory: the current stream does not get them back while they are in use."""
    dt = torch.float16
    x, w_in, w_down, dy = make_ffn(300, 512, 1024, dt, seed=5)
    xm, codes, scales, z = make_w4(2, 64, 16384, 64, True, dt)
    m = torch.randn(300, 400, device="cuda")
    y, gu = g.gated_ffn(x, w_in, w_down, save=True)
    want = (y, *g.gated_ffn_backward(dy, x, w_in, w_down, gu), g.w4_linear(xm, codes, scales, z), g.orthogonalize(m))
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for call, ref in ((lambda: g.gated_ffn(x, w_in, w_down, stream=stream), want[:1]),
                          (lambda: g.gated_ffn_backward(dy, x, w_in, w_down, gu, stream=stream), want[1:4]),
                          (lambda: g.w4_linear(xm, codes, scales, z, stream=stream), want[4:5]),
                          (lambda: g.orthogonalize(m, stream=stream), want[5:])):
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)  # about 10 ms, so that the call is still to run below
            got = call()
            trash = [torch.full((n,), float("nan"), device="cuda") for n in (1 << k for k in range(6, 22)) for _ in range(3)]
            torch.cuda.synchronize()
            got = got if isinstance(got, tuple) else (got,)
            assert len(got) == len(ref) and all(torch.equal(a, b) for a, b in zip(got, ref))
            del trash


def test_wrong_objects_are_refused(g):
    x, w_in, w_down, _ = make_ffn(2, 16, 16, torch.float16)
    with pytest.raises(TypeError):
        g.default_ops().gated_ffn([1, 2], w_in, w_down)
    with pytest.raises(TypeError):
        g.gated_ffn(x, None, w_down)
    with pytest.raises(ValueError):
        g.gated_ffn(x, w_in, w_down, out=torch.empty(2, 16, dtype=torch.float16))
