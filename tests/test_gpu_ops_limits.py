"""The operators at the limits of their arguments: empty sums, infinities and
values near the types' largest, the longest rows, and what is refused there.
Bounds as in test_gpu_ops.py."""
import random

import pytest
import torch

from test_gpu_ops import F64, check, make_ffn, make_w4, sum_eps, w4_ref

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


# ------------------------------------------------------------ 4-bit products --
def same_specials(got, ref):
    return (torch.equal(got.isnan(), ref.isnan()) and torch.equal(got.isposinf(), ref.isposinf()) and
            torch.equal(got.isneginf(), ref.isneginf()))


def w4_product(x, w):
    """x W^T in 64 bits, product by product: infinities as the formula has them."""
    return (x.to(F64).unsqueeze(1) * w).sum(-1)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 3, 5, 9, 17])
def test_w4_infinite_x(g, T, group, dt):
    """An infinite x makes each of its token's sums a signed infinity, or NaN where
    its weight is zero or infinities of both signs meet; other tokens are as before."""
    for K, zeros in ((512, True), (352 // group * group, False), (9 * group, True)):
        x, codes, scales, z = make_w4(T, 50, K, group, zeros, dt, seed=T)
        w = w4_ref(codes, scales, z)
        before = g.w4_linear(x, codes, scales, z)
        x[0, 77] = float("inf")
        x[T // 2, 30] = float("-inf")
        x[T - 1, K - 1] = float("inf")
        got, ref = g.w4_linear(x, codes, scales, z), w4_product(x, w)
        assert same_specials(got, ref)
        rest = [t for t in range(T) if t not in (0, T // 2, T - 1)]
        assert torch.equal(got[rest], before[rest])
        x[0, 5] = float("nan")
        assert g.w4_linear(x, codes, scales, z)[0].isnan().all()
        x[0, 5] = 1.0
        p = w4_product(x, w)
        for act, ref in (("relu", p[:, :25].clamp_min(0) * p[:, 25:]), ("silu", p[:, :25] * torch.sigmoid(p[:, :25]) * p[:, 25:])):
            assert same_specials(g.w4_gated(x, codes, scales, z, act=act), ref)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 4, 11])
def test_w4_very_large_x(g, T, group):
    """x up to the type's largest: its products with the codes' offset overflow,
    its products with the weights do not."""
    K, dt = 640, torch.bfloat16
    x, codes, scales, z = make_w4(T, 40, K, group, True, dt, seed=T)
    x[0, 77], x[T - 1, 300] = 2.0 ** 126, -3e38
    scales *= 2.0 ** -8
    w = w4_ref(codes, scales, z)
    check(g.w4_linear(x, codes, scales, z), w4_product(x, w), sum_eps(K) * (x.to(F64).abs() @ w.abs().t()), dt, "y")


def test_w4_infinite_x_over_slices(g):
    """K cut over CTAs: the slice that meets the infinity sums its own part."""
    K, dt = 16384, torch.float16
    x, codes, scales, z = make_w4(3, 33, K, 64, True, dt)
    for at in (0, 8191, K - 1):
        y = x.clone()
        y[1, at] = float("-inf")
        assert same_specials(g.w4_linear(y, codes, scales, z), w4_product(y, w4_ref(codes, scales, z)))


def test_w4_infinite_scale(g):
    """An infinite scale in the last group of rows that end inside a block."""
    for group in (32, 64):
        K = 3 * group
        x, codes, scales, z = make_w4(2, 20, K, group, False, torch.float16)
        x = x.abs()
        codes[7, K // 2 - group // 2:] = 0xff  # weights of one sign: 7 times the scale
        scales[7, 2] = float("inf")
        got = g.w4_linear(x, codes, scales, z)
        assert torch.isposinf(got[:, 7]).all()
        keep = torch.arange(20, device="cuda") != 7
        assert torch.isfinite(got[:, keep]).all()


# ------------------------------------------------------ orthogonalised update --
LONGEST = 2 ** 31 - 4096


def test_orthogonalize_longest_rows(g):
    """The kernels' 32-bit counters step past the end of a row: the longest they
    can is taken and right to its end, a longer one refused before any launch."""
    lib, h = g.default_ops()._lib, g.default_ops()._h
    for M, N in ((1, LONGEST), (LONGEST, 1)):
        assert lib.gemm_orthogonalize_workspace(h, 1, M, N) > 0
    for batch, M, N in ((1, 1, LONGEST + 1), (1, LONGEST + 1, 1), (1, 1, 2 ** 31 - 1), (1, 2 ** 62, 2 ** 62), (65536, 1, 1)):
        assert lib.gemm_orthogonalize_workspace(h, batch, M, N) == 0
    m = torch.zeros(1, 2 ** 31 - 100, dtype=torch.float16, device="cuda")
    with pytest.raises(g.GemmError) as e:
        g.orthogonalize(m)
    assert e.value.status == 1
    at = [0, 255, 2 ** 30 + 7, LONGEST - 1]
    m[0, at] = 3.0
    o = g.orthogonalize(m[:, :LONGEST], steps=0, eps=0.0)
    g.default_ops().check_error()
    assert (o[0, at] == 0.5).all()
    assert int((o != 0).sum()) == len(at)


def test_w4_longest_rows(g):
    """Rows of 2^28 codes for 16 tokens: K cut into more slices than 16 warps a CTA
    would leave within a grid.  A few ones in x pick weights from every part."""
    T, N, K, dt = 16, 2, 2 ** 28, torch.float16
    gen = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.full((N, K // 128), 0.25, dtype=dt, device="cuda")
    x = torch.zeros(T, K, dtype=dt, device="cuda")
    at = torch.cat((torch.tensor([0, 1, K // 2 - 1, K - 1], device="cuda"), torch.randint(0, K, (28,), generator=gen, device="cuda")))
    on = torch.randint(0, 2, (T, at.numel()), generator=gen, device="cuda").to(dt)
    x[:, at] = on
    on = x[:, at].to(F64)  # what stands there where two positions are one
    first = (at.unsqueeze(0) == at.unsqueeze(1)).int().argmax(1) == torch.arange(at.numel(), device="cuda")
    q = (codes[:, at // 2] >> (4 * (at % 2)).to(torch.uint8) & 15).to(F64)
    want = (on * first) @ ((q - 8) * 0.25).t()
    got = g.w4_linear(x, codes, scales)
    g.default_ops().check_error()
    assert torch.equal(got.to(F64), want)


# --------------------------------------------------------------------- autograd --
def test_tensors_that_ask_for_a_graph_are_refused(g):
    """Whichever tensor it is, the output among them, while gradients are recorded;
    without, the call is the one on plain tensors."""
    dt = torch.float16
    x, w_in, w_down, dy = make_ffn(4, 64, 128, dt)
    gu = torch.randn(4, 256, device="cuda").to(dt)
    xm, codes, scales, z = make_w4(4, 64, 256, 64, True, dt)
    m = torch.randn(40, 30, device="cuda")
    def empty(*s):
        return torch.empty(*s, dtype=dt, device="cuda")
    n = 0
    for fn, args, out in ((g.gated_ffn, (x, w_in, w_down), empty(4, 64)), (g.gated_ffn_backward, (dy, x, w_in, w_down, gu), None),
                          (g.w4_linear, (xm, codes, scales, z), empty(4, 64)), (g.w4_gated, (xm, codes, scales, z), empty(4, 32)),
                          (g.orthogonalize, (m,), torch.empty_like(m))):
        want = fn(*args)
        for i, a in enumerate(args):
            if not a.is_floating_point():
                continue
            other = list(args)
            other[i] = torch.nn.Parameter(a.clone())
            with pytest.raises(RuntimeError, match="requires grad"):
                fn(*other)
            for mode in (torch.no_grad, torch.inference_mode):
                with mode():
                    got = fn(*other)
                assert all(torch.equal(p, q) for p, q in zip(*((t if isinstance(t, tuple) else (t,)) for t in (got, want))))
            n += 1
        if out is not None:
            with pytest.raises(RuntimeError, match="requires grad"):
                fn(*args, out=out.requires_grad_())
            with torch.no_grad():
                assert torch.equal(fn(*args, out=out), want)
    assert n == 13


# ----------------------------------------------------------------- host threads --
def test_calls_from_threads_that_have_not_used_cuda(g):
    """Such a thread has no context until its first CUDA call; each operator makes
    that call itself."""
    import threading
    dt = torch.float16
    x, w_in, w_down, dy = make_ffn(40, 64, 128, dt)
    xm, codes, scales, z = make_w4(4, 64, 256, 64, True, dt)
    m = torch.randn(40, 30, device="cuda")
    _, gu = g.gated_ffn(x, w_in, w_down, save=True)
    for fn, args in ((g.gated_ffn, (x, w_in, w_down)), (g.gated_ffn, (x[:2], w_in, w_down)),
                     (g.gated_ffn_backward, (dy, x, w_in, w_down, gu)), (g.w4_linear, (xm, codes, scales, z)),
                     (g.w4_gated, (xm, codes, scales, z)), (g.orthogonalize, (m,))):
        want, got = fn(*args), []
        def body():
            try:
                got.append(fn(*args))
            except Exception as e:
                got.append(e)
        t = threading.Thread(target=body)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not isinstance(got[0], Exception), (fn.__name__, got[0])
        assert all(torch.equal(p, q) for p, q in zip(*((v if isinstance(v, tuple) else (v,)) for v in (got[0], want))))


def test_gated_block_as_an_autograd_function(g):
    """The two passes as the methods of a Function: gradients reach the weights."""
    class Block(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w_in, w_down):
            y, gu = g.gated_ffn(x, w_in, w_down, save=True)
            ctx.save_for_backward(x, w_in, w_down, gu)
            return y

        @staticmethod
        def backward(ctx, dy):
            return g.gated_ffn_backward(dy, *ctx.saved_tensors)

    x, w_in, w_down, dy = make_ffn(40, 64, 128, torch.float16)
    params = [torch.nn.Parameter(t.clone()) for t in (x, w_in, w_down)]
    Block.apply(*params).backward(dy)
    _, gu = g.gated_ffn(x, w_in, w_down, save=True)
    for p, want in zip(params, g.gated_ffn_backward(dy, x, w_in, w_down, gu)):
        assert torch.equal(p.grad, want)


def test_outputs_count_as_written(g):
    """`out` raises the tensor's version: autograd sees that a value it saved has
    been overwritten.  Tensors of inference mode, which have none, are written too."""
    dt = torch.float16
    x, w_in, w_down, _ = make_ffn(4, 64, 128, dt)
    xm, codes, scales, z = make_w4(4, 64, 256, 64, True, dt)
    m = torch.randn(4, 64, device="cuda")
    for fn, args in ((g.gated_ffn, (x, w_in, w_down)), (g.w4_linear, (xm, codes, scales, z)),
                     (lambda *a, out: g.w4_gated(*a, out=out[:, :32]), (xm, codes, scales, z)),
                     (lambda *a, out: g.orthogonalize(*a, out=out, dtype=dt), (m,))):
        out = torch.ones(4, 64, device="cuda", dtype=dt)
        leaf = torch.ones(4, 64, device="cuda", dtype=dt, requires_grad=True)
        y = leaf * out  # saves out
        before = out._version
        fn(*args, out=out)
        assert out._version == before + 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
        with torch.inference_mode():
            frozen = torch.ones(4, 64, device="cuda", dtype=dt)
        assert torch.equal(fn(*args, out=frozen), fn(*args, out=out))


# -------------------------------------------------------------- views of one buffer --
def test_outputs_beside_inputs_in_one_matrix(g):
    """An output in other columns, or other matrices, of the buffer that holds an
    input shares no element with it: taken, and nothing else is written."""
    dt = torch.float16
    for T in (1, 5, 40, 300):
        x, w_in, w_down, _ = make_ffn(T, 64, 128, dt)
        both = torch.cat((x, torch.full_like(x, 7.0), x), 1)
        g.gated_ffn(both[:, :64], w_in, w_down, out=both[:, 64:128])
        assert torch.equal(both[:, 64:128], g.gated_ffn(x, w_in, w_down))
        assert torch.equal(both[:, :64], x) and torch.equal(both[:, 128:], x)
        xm, codes, scales, z = make_w4(T, 40, 64, 32, True, dt)
        both = torch.cat((torch.full((T, 41), 7.0, device="cuda", dtype=dt)[:, :40], xm), 1)
        g.w4_linear(both[:, 40:], codes, scales, z, out=both[:, :40])
        assert torch.equal(both[:, :40], g.w4_linear(xm, codes, scales, z)) and torch.equal(both[:, 40:], xm)
    m = torch.randn(3, 20, 30, device="cuda")
    want = g.orthogonalize(m)
    beside = torch.cat((m, m), 2)
    assert torch.equal(g.orthogonalize(beside[..., 30:], out=beside[..., :30]), want)
    assert torch.equal(beside[..., 30:], m)
    below = torch.cat((m, m), 1)
    assert torch.equal(g.orthogonalize(below[:, :20], out=below[:, 20:]), want) and torch.equal(below[:, :20], m)
    turns = m.repeat_interleave(2, 0)
    assert torch.equal(g.orthogonalize(turns[0::2], out=turns[1::2]), want) and torch.equal(turns[0::2], m)
    assert torch.equal(g.orthogonalize(m[:1].expand(3, 20, 30))[2], want[0])


def test_outputs_are_refused_where_they_share_elements(g):
    """Random views of one buffer: refused exactly where an element is in both."""
    rng = random.Random(0)
    refused = 0
    for _ in range(400):
        B, M, N = rng.randint(1, 4), rng.randint(1, 6), rng.randint(2, 12)
        buf = torch.randn(B, M, N, device="cuda")
        where = torch.arange(buf.numel()).view(B, M, N)
        b, r, c = rng.randint(1, B), rng.randint(1, M), rng.randint(1, N - 1)
        def view(step=rng.choice((1, 2))):
            i = rng.randint(0, B - b) if step == 1 else rng.randint(0, 1)
            r0, c0 = rng.randint(0, M - r), rng.randint(0, N - c)
            cut = (slice(i, i + b) if step == 1 else slice(i, None, 2), slice(r0, r0 + r), slice(c0, c0 + c))
            return buf[cut], set(where[cut].flatten().tolist())
        (v, at), (w, on) = view(), view()
        if v.shape != w.shape or not at:
            continue
        want = g.orthogonalize(v.contiguous())
        if at & on:
            refused += 1
            before = buf.clone()
            with pytest.raises(g.GemmError) as e:
                g.orthogonalize(v, out=w)
            assert e.value.status == 1 and torch.equal(buf, before)
        else:
            assert torch.equal(g.orthogonalize(v, out=w), want)
    assert 50 < refused < 350
    dt = torch.float16
    x, w_in, w_down, _ = make_ffn(5, 64, 128, dt)
    both = torch.cat((x, x), 1)
    for first in (0, 8, 56):
        with pytest.raises(g.GemmError):
            g.gated_ffn(both[:, :64], w_in, w_down, out=both[:, first:first + 64])
    flat = torch.zeros(2000, device="cuda", dtype=dt)  # rows of two pitches in one range: refused, whether or not they meet
    with pytest.raises(g.GemmError):
        g.gated_ffn(flat.as_strided((5, 64), (128, 1)), w_in, w_down, out=flat.as_strided((5, 64), (192, 1), 64))


# --------------------------------------------------------------------- watchdog --
# A form of the products each (the cost model's choice on 152 SMs), for the gated
# product and the one after it: pairs; two pairs on a tile, then pairs; pairs, then
# two pairs; clusters of four.
@pytest.mark.parametrize("shape", [(1536, 4096, 1536), (1536, 4096, 768), (4096, 512, 2048), (17, 512, 512)],
                         ids=["pairs", "two_pairs_first", "two_pairs_second", "clusters"])
def test_watchdog_ends_a_stuck_wait_in_every_form(g, shape):
    """A k-block that is never loaded: every role of the unit gives up after the
    limit, in the CTAs that share its tile too; the next call is right."""
    ops = g.Ops(0)
    x, w_in, w_down, _ = make_ffn(*shape, torch.float16)
    ops.set_watchdog(timeout_ns=50_000_000, skip_k_block=1)
    ops.gated_ffn(x, w_in, w_down)
    with pytest.raises(g.GemmError) as e:
        ops.check_error()
    assert e.value.status == 5 and ops.last_error_detail()[0] == 5
    ops.set_watchdog()
    assert torch.equal(ops.gated_ffn(x, w_in, w_down), g.gated_ffn(x, w_in, w_down))
    ops.check_error()
    ops.close()


# The update's: k-ranges side by side in one CTA; lone CTAs, then pairs; two pairs.
@pytest.mark.parametrize("shape", [(5, 900, 1000), (1, 3000, 3010), (1, 2048, 2048)], ids=["parts", "lone", "two_pairs"])
def test_watchdog_ends_a_stuck_wait_of_an_update(g, shape):
    ops = g.Ops(0)
    m = torch.randn(*shape, device="cuda")
    ops.set_watchdog(timeout_ns=50_000_000, skip_k_block=1)
    ops.orthogonalize(m, steps=1)
    with pytest.raises(g.GemmError) as e:
        ops.check_error()
    assert e.value.status == 5 and ops.last_error_detail()[0] == 5
    ops.set_watchdog()
    assert torch.equal(ops.orthogonalize(m, steps=1), g.orthogonalize(m, steps=1))
    ops.check_error()
    ops.close()


# ---------------------------------------------------------------------- streams --
@pytest.mark.parametrize("stream", [0, 1, 2], ids=["null", "legacy", "per_thread"])
def test_streams_by_their_handles(g, stream):
    """CUDA's own handles: the null stream, the legacy default stream and the
    thread's default stream."""
    dt = torch.float16
    x, w_in, w_down, dy = make_ffn(40, 64, 128, dt)
    xm, codes, scales, z = make_w4(4, 64, 256, 64, True, dt)
    m = torch.randn(40, 30, device="cuda")
    _, gu = g.gated_ffn(x, w_in, w_down, save=True)
    for fn, args in ((g.gated_ffn, (x, w_in, w_down)), (g.gated_ffn_backward, (dy, x, w_in, w_down, gu)),
                     (g.w4_linear, (xm, codes, scales, z)), (g.w4_gated, (xm, codes, scales, z)), (g.orthogonalize, (m,))):
        want = fn(*args)
        torch.cuda.synchronize()
        got = fn(*args, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(*((v if isinstance(v, tuple) else (v,)) for v in (got, want))))
