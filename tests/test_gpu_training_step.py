"""The operators together, as a training step uses them: a norm before the gated
block, one before the head, the loss, and back through all of them to the update.
Every stage is held to its own bound from what it was given (the bounds of the other
files), in eager mode, from one graph, and through torch's autograd."""
import pytest
import torch

import test_gpu_norm as tn
import test_gpu_ops as to
import test_gpu_xent as tx

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(scope="module")
def g():
    import dense_fp16_gemm_04_gb300 as m
    m.build()
    return m


def make(T, D, F, V, dt, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    def r(*s):
        return torch.randn(*s, generator=gen, device="cuda")
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda")
    targets[: T // 4] = -100
    return dict(x=r(T, D).to(dt), n1=(1 + 0.1 * r(D)), n2=(1 + 0.1 * r(D)).to(dt), b2=(0.1 * r(D)).to(dt),
                w_in=(r(2 * F, D) * D ** -0.5).to(dt), w_down=(r(D, F) * F ** -0.5).to(dt),
                head=(r(V, D) * D ** -0.5).to(dt), targets=targets)


def step(g, p, scale):
    """Forward, backward and the update of the block's matrices; every tensor on the way."""
    t = {}
    t["a"], t["s1"] = g.rms_norm(p["x"], p["n1"], save=True)
    t["y"], t["gu"] = g.gated_ffn(t["a"], p["w_in"], p["w_down"], save=True)
    t["r"] = p["x"] + t["y"]
    t["z"], t["s2"] = g.layer_norm(t["r"], p["n2"], p["b2"], save=True)
    t["loss"], t["lse"] = g.linear_cross_entropy(t["z"], p["head"], p["targets"], save=True)
    dloss = torch.full((1,), scale, device="cuda").expand(len(p["targets"]))
    t["dz"], t["dhead"] = g.linear_cross_entropy_backward(dloss, t["z"], p["head"], p["targets"], t["lse"])
    t["dr"], t["dn2"], t["db2"] = g.layer_norm_backward(t["dz"], t["r"], p["n2"], t["s2"])
    t["da"], t["dw_in"], t["dw_down"] = g.gated_ffn_backward(t["dr"], t["a"], p["w_in"], p["w_down"], t["gu"])
    t["dx1"], t["dn1"] = g.rms_norm_backward(t["da"], p["x"], p["n1"], t["s1"])
    t["dx"] = t["dr"] + t["dx1"]
    t["u_in"], t["u_down"] = g.orthogonalize(t["dw_in"]), g.orthogonalize(t["dw_down"])
    return t


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 64, 128, 500), (37, 136, 264, 1003), (600, 520, 1032, 6007)],
                         ids=lambda s: "x".join(map(str, s)))
def test_step(g, shape, dt):
    p = make(*shape, dt)
    if shape[0] == 1:
        p["targets"][:] = 3
    scale = 256.0 / shape[0]
    t = step(g, p, scale)
    g.default_ops().check_error()
    T = shape[0]
    # forward
    y, err, st = tn.forward_ref(p["x"], p["n1"], None, 1e-6, True)
    tn.check(t["a"], y, err, "a")
    tn.check_stats(t["s1"], st, True)
    h, eh, pr, ep = to.gated_ref(t["a"], p["w_in"], "silu", dt)
    to.check(t["gu"], pr, ep, dt, "gu")
    wd = p["w_down"].to(F64)
    eh = eh + to.U[dt] * (h.abs() + eh) + to.TINY[dt]
    to.check(t["y"], h @ wd.t(), eh @ wd.abs().t() + to.sum_eps(shape[2]) * ((h.abs() + eh) @ wd.abs().t()), dt, "y")
    y, err, st = tn.forward_ref(t["r"], p["n2"], p["b2"], 1e-5, False)
    tn.check(t["z"], y, err, "z")
    tn.check_stats(t["s2"], st, False)
    rl, rz = tx.forward_ref(t["z"], p["head"], p["targets"])
    tx.check(t["loss"], *rl, "loss")
    tx.check(t["lse"], *rz, "lse")
    # backward
    dloss = torch.full((T,), scale, device="cuda")
    rx, rw = tx.backward_ref(dloss, None, t["z"], p["head"], p["targets"], t["lse"], dt)
    tx.check(t["dz"], *rx, "dz")
    tx.check(t["dhead"], *rw, "dhead")
    for name, r in zip(("dr", "dn2", "db2"), tn.backward_ref(t["dz"], t["r"], p["n2"], t["s2"], False)):
        tn.check(t[name], *r, name)
    refs = to.ffn_backward_ref(t["dr"], t["a"], p["w_in"], p["w_down"], t["gu"], "silu", dt)
    for name, r in zip(("da", "dw_in", "dw_down"), refs):
        to.check(t[name], *r, dt, name)
    for name, r in zip(("dx1", "dn1"), tn.backward_ref(t["da"], p["x"], p["n1"], t["s1"], True)):
        tn.check(t[name], *r, name)
    for name, m in (("u_in", t["dw_in"]), ("u_down", t["dw_down"])):
        ref, e = to.ns_ref(m, 5, to.COEFFS, 1e-7)
        assert (t[name].to(F64) - ref).norm() <= e + to.U[dt] * ref.norm(), name


def test_step_in_a_graph_and_twice_at_once(g):
    """One captured step, replayed on new inputs, and two graphs with workspaces of one
    pool replayed in turn, give what the eager step gives."""
    p = make(300, 264, 520, 4001, torch.bfloat16)
    other = make(300, 264, 520, 4001, torch.bfloat16, seed=1)
    want, want2 = step(g, p, 0.01), step(g, other, 0.01)
    held = {k: v.clone() for k, v in p.items()}
    torch.cuda.synchronize()
    pool = torch.cuda.graph_pool_handle()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    got = []
    for graph in graphs:
        with torch.cuda.graph(graph, pool=pool):
            got.append(step(g, held, 0.01))
    for graph, out in zip(graphs, got):
        for inputs, ref in ((p, want), (other, want2)):
            for k, v in inputs.items():
                held[k].copy_(v)
            graph.replay()
            torch.cuda.synchronize()
            for k in ref:
                assert torch.equal(out[k], ref[k]), k


def test_steps_on_two_streams(g):
    """Two steps at once, each on its own stream and from its own thread."""
    import threading
    ps = [make(200, 264, 520, 4001, torch.float16, seed=s) for s in range(2)]
    want = [step(g, p, 0.01) for p in ps]
    torch.cuda.synchronize()
    bad = []
    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = step(g, ps[i], 0.01)
                s.synchronize()
                bad.extend(k for k in got if not torch.equal(got[k], want[i][k]))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_gradients_through_autograd(g):
    """The forward and backward operators as torch.autograd.Functions (whose backward
    runs on a thread of autograd's) give the step's gradients."""
    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            y, st = g.layer_norm(x, w, b, save=True)
            ctx.save_for_backward(x, w, st)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, w, st = ctx.saved_tensors
            return g.layer_norm_backward(dy.contiguous(), x, w, st)

    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, t):
            loss, lse = g.linear_cross_entropy(x, w, t, save=True)
            ctx.save_for_backward(x, w, t, lse)
            return loss, lse

        @staticmethod
        def backward(ctx, dloss, dlse):
            x, w, t, lse = ctx.saved_tensors
            return (*g.linear_cross_entropy_backward(dloss, x, w, t, lse, dlse=dlse), None)

    p = make(100, 136, 8, 1003, torch.bfloat16)
    leaves = [p[k].clone().requires_grad_() for k in ("x", "n2", "b2", "head")]
    x, n2, b2, head = leaves
    loss, lse = Loss.apply(Norm.apply(x, n2, b2), head, p["targets"])
    (loss.sum() * 0.02 + 1e-3 * lse.square().sum()).backward()
    z, st = g.layer_norm(p["x"], p["n2"], p["b2"], save=True)
    dlse = 1e-3 * 2 * lse.detach()
    dz, dhead = g.linear_cross_entropy_backward(torch.full((100,), 0.02, device="cuda"), z, p["head"], p["targets"],
                                                lse.detach(), dlse=dlse)
    want = (*g.layer_norm_backward(dz, p["x"], p["n2"], st), dhead)
    for leaf, w in zip(leaves, want):
        assert torch.equal(leaf.grad, w)
    with pytest.raises(RuntimeError, match="requires grad"):
        g.layer_norm(x, n2, b2)
    with pytest.raises(RuntimeError, match="requires grad"):
        g.linear_cross_entropy(z, head, p["targets"])
