"""The decoder block's operators run together on cuda:0, as a decoder block uses them.

Serving: norm -> Mamba layer -> (residual add and norm in one call) -> mixture of experts
with the residual stream added.  Training: norm -> linear with SiLU -> linear with the
residual stream, and back.  Each stage is held against its formula in float64 from the
values the stage before it stored, with the tolerances of the stage's own test; the chain,
enqueued without a wait or captured into a graph, gives the bits of the same calls with a
synchronisation after each.
"""
import pytest

import test_gpu_linear as lin
import test_gpu_moe as moe
import test_gpu_norm as norm

pytestmark = pytest.mark.gpu


def block(tokens, d_model=256, d_inner=512, d_ff=392, experts=4, seed=0):
    """Weights and a residual stream of one block."""
    import torch
    from mamba_selective_scan_jamba_b200 import devio, synth
    g = torch.Generator().manual_seed(seed)

    def rn(*s, std=1.0, mean=0.0):
        return (torch.randn(*s, generator=g) * std + mean).to(torch.bfloat16).cuda()
    w = synth.Workload("block", 1, tokens, d_inner, 32, "bf16", seed=seed + 1, extra=True)
    m = moe.make(tokens, d_model, d_ff, experts, seed=seed + 2)
    return dict(w=w, W=devio.weights_to_device(synth.make_weights(w)), m=m,
                stream=rn(tokens, d_model), n1=rn(d_model, std=0.1, mean=1.0),
                n2=rn(d_model, std=0.1, mean=1.0),
                inp=rn(2 * d_inner, d_model, std=d_model ** -0.5),
                outp=rn(d_model, d_inner, std=d_inner ** -0.5))


class Serving:
    """The block's buffers and its calls, in order."""

    def __init__(self, b):
        import torch
        from mamba_selective_scan_jamba_b200 import devio, jmix
        self.b, self.jm = b, jmix
        t, d = b["stream"].shape
        e, f = b["m"]["wg"].shape[:2]
        self.nd = jmix.norm_dims(t, d)
        self.ld = devio.dims_of(b["w"])
        self.md = jmix.moe_dims(t, d, f, e, 2, router=jmix.JM_ROUTE_SOFTMAX_TOPK)
        self.n_layer = jmix.jm_layer_fwd_workspace_size(self.ld, d)
        self.n_moe = jmix.jm_moe_fwd_workspace_size(self.md)
        # one workspace for both, as a program whose calls follow one another keeps it
        self.ws = devio.workspace(max(self.n_layer, self.n_moe))
        z = torch.zeros_like
        self.h, self.mix, self.sum, self.y, self.out = (z(b["stream"]) for _ in range(5))
        self.state = torch.zeros((1, b["w"].d_inner, 16), device="cuda")

    def calls(self):
        b, jm = self.b, self.jm
        return [
            lambda s: jm.jm_norm_fwd(self.nd, b["stream"], b["n1"], self.h, stream=s),
            lambda s: jm.jm_layer_fwd(self.ld, b["stream"].shape[1], self.h, b["inp"], b["W"],
                                      b["outp"], self.mix, self.state, self.ws, self.n_layer,
                                      stream=s),
            lambda s: jm.jm_norm_fwd(self.nd, self.mix, b["n2"], self.y, residual=b["stream"],
                                     sum_out=self.sum, stream=s),
            lambda s: jm.jm_moe_fwd(self.md, self.y, b["m"]["wr"], b["m"]["wg"], b["m"]["wu"],
                                    b["m"]["wd"], self.out, self.ws, self.n_moe,
                                    residual=self.sum, stream=s),
        ]

    def run(self, stream=None, wait=False):
        import torch
        for c in self.calls():
            c(stream)
            if wait:
                torch.cuda.synchronize()

    def results(self):
        return [v.clone() for v in (self.h, self.mix, self.sum, self.y, self.out, self.state)]


@pytest.mark.parametrize("tokens", [1, 37, 200])
def test_serving_block(tokens):
    import torch
    b = block(tokens, seed=tokens)
    s = Serving(b)
    s.run(wait=True)
    want = s.results()
    assert s.jm.jm_poll_error(s.ws) == s.jm.JM_OK
    # stage by stage: the norms, and the experts on what the second norm stored
    _, _, _, _, ref = norm.ref_fwd(b["stream"], None, b["n1"], None, 0, 1e-6)
    w = b["n1"].double().abs()
    assert ((s.h.double() - ref).abs() <= norm.half("bf16") * ref.abs() + 64 * norm.E32 * (ref.abs() + w)).all()
    total, _, _, _, ref = norm.ref_fwd(s.mix, b["stream"], b["n2"], None, 0, 1e-6)
    assert torch.equal(s.sum, total)
    w = b["n2"].double().abs()
    assert ((s.y.double() - ref).abs() <= norm.half("bf16") * ref.abs() + 64 * norm.E32 * (ref.abs() + w)).all()
    out, _, _ = moe.check(dict(b["m"], x=s.y.clone(), r=s.sum.clone()), 2, moe.TOPK, residual=True)
    assert torch.equal(out, s.out)
    # without waits between, and the layer's output from its own test's path stays the same
    for v in (s.h, s.mix, s.sum, s.y, s.out):
        v.fill_(float("nan"))
    s.run()
    torch.cuda.synchronize()
    for a, e in zip(s.results(), want):
        assert torch.equal(a, e)


def test_serving_block_in_two_graphs_that_share_a_workspace():
    """Two blocks captured into two graphs, replayed in turn on one stream, with one
    workspace between them; the second's input is the first's output."""
    import torch
    b1, b2 = block(24, seed=5), block(24, seed=6)
    s1, s2 = Serving(b1), Serving(b2)
    s2.ws = s1.ws
    b2["stream"] = s1.out
    s1.run(wait=True)
    s2.run(wait=True)
    graphs = []
    for s in (s1, s2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run(torch.cuda.current_stream())
        graphs.append(g)
    x0 = b1["stream"].clone()
    for k in (1.0, -0.5, 2.0):
        b1["stream"].copy_(x0 * k)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert s1.jm.jm_poll_error(s1.ws) == s1.jm.JM_OK
        got = s1.results() + s2.results()
        s1.run(wait=True)
        s2.run(wait=True)
        for a, e in zip(got, s1.results() + s2.results()):
            assert torch.equal(a, e)


class Training:
    """h = norm(x); p = h w1^T + b1, u = silu(p); out = u w2^T + x; and the gradients of
    sum(out g)."""

    def __init__(self, rows, d, f, seed):
        import torch
        from mamba_selective_scan_jamba_b200 import devio, jmix
        self.jm = jmix
        g = torch.Generator().manual_seed(seed)

        def rn(*s, std=1.0, mean=0.0):
            return (torch.randn(*s, generator=g) * std + mean).to(torch.bfloat16).cuda()
        self.x, self.g = rn(rows, d, std=2.0, mean=0.3), rn(rows, d)
        self.wn, self.bn = rn(d, std=0.1, mean=1.0), rn(d, std=0.1)
        self.w1, self.b1 = rn(f, d, std=d ** -0.5), rn(f)
        self.w2 = rn(d, f, std=f ** -0.5)
        self.nd = jmix.norm_dims(rows, d, kind=jmix.JM_NORM_LAYER)
        self.d1 = jmix.linear_dims(rows, d, f, act=jmix.JM_ACT_SILU)
        self.d2 = jmix.linear_dims(rows, f, d)
        self.n = [jmix.jm_linear_fwd_workspace_size(self.d1),
                  jmix.jm_linear_fwd_workspace_size(self.d2),
                  jmix.jm_linear_bwd_workspace_size(self.d2),
                  jmix.jm_linear_bwd_workspace_size(self.d1),
                  jmix.jm_norm_bwd_workspace_size(self.nd)]
        self.ws = devio.workspace(max(self.n))
        z = torch.zeros_like
        self.h, self.out, self.gh, self.gx = z(self.x), z(self.x), z(self.x), z(self.x)
        self.stats = torch.zeros(rows, 2, device="cuda")
        self.p = torch.zeros(rows, f, device="cuda", dtype=torch.bfloat16)
        self.u, self.gu = z(self.p), z(self.p)
        self.gw1, self.gb1, self.gw2 = z(self.w1), z(self.b1), z(self.w2)
        self.gwn, self.gbn = z(self.wn), z(self.bn)

    def run(self, stream=None, wait=False):
        import torch
        jm, n, ws = self.jm, self.n, self.ws
        for c in (
            lambda s: jm.jm_norm_fwd(self.nd, self.x, self.wn, self.h, bias=self.bn,
                                     stats=self.stats, stream=s),
            lambda s: jm.jm_linear_fwd(self.d1, self.h, self.w1, self.u, ws, n[0], bias=self.b1,
                                       pre=self.p, stream=s),
            lambda s: jm.jm_linear_fwd(self.d2, self.u, self.w2, self.out, ws, n[1],
                                       residual=self.x, stream=s),
            lambda s: jm.jm_linear_bwd(self.d2, self.g, self.u, self.w2, ws, n[2], g_x=self.gu,
                                       g_w=self.gw2, stream=s),
            lambda s: jm.jm_linear_bwd(self.d1, self.gu, self.h, self.w1, ws, n[3], pre=self.p,
                                       g_x=self.gh, g_w=self.gw1, g_bias=self.gb1, stream=s),
            lambda s: jm.jm_norm_bwd(self.nd, self.gh, self.x, self.wn, self.stats, self.gx, ws,
                                     n[4], g_sum=self.g, g_weight=self.gwn, g_bias=self.gbn,
                                     stream=s),
        ):
            c(stream)
            if wait:
                torch.cuda.synchronize()

    def results(self):
        return [v.clone() for v in (self.h, self.p, self.u, self.out, self.gu, self.gw2, self.gh,
                                    self.gw1, self.gb1, self.gx, self.gwn, self.gbn, self.stats)]


@pytest.mark.parametrize("rows,d,f", [(3, 64, 136), (150, 256, 520), (700, 520, 1032)])
def test_training_block(rows, d, f):
    import torch
    t = Training(rows, d, f, seed=rows)
    t.run(wait=True)
    want = t.results()
    assert t.jm.jm_poll_error(t.ws) == t.jm.JM_OK
    # the products and their backward from the values that were stored
    a = dict(x=t.h, w=t.w1, b=t.b1, r=t.x, g=t.gu)
    out, pre = lin.check_fwd(a, "silu", bias=True, residual=False)
    assert torch.equal(out, t.u) and torch.equal(pre, t.p)
    o = lin.check_bwd(a, "silu", t.p)
    assert torch.equal(o["g_x"], t.gh) and torch.equal(o["g_w"], t.gw1)
    assert torch.equal(o["g_bias"], t.gb1)
    # the whole chain against float64 autograd: six roundings to bf16 lie between the inputs
    # and a gradient (h, p or u, g_u, g_p, g_h, the gradient itself), each within half a step
    # relative to its value; in root mean square over a gradient their effects add to no more
    # than their sum, 6 half
    v = {k: getattr(t, k).double().requires_grad_(True) for k in ("x", "wn", "bn", "w1", "b1", "w2")}
    m = v["x"].mean(1, keepdim=True)
    h = (v["x"] - m) * (((v["x"] - m) ** 2).mean(1, keepdim=True) + 1e-6) ** -0.5 * v["wn"] + v["bn"]
    p = h @ v["w1"].t() + v["b1"]
    y = (p * torch.sigmoid(p)) @ v["w2"].t() + v["x"]
    (y * t.g.double()).sum().backward()
    for name, got in (("x", t.gx), ("wn", t.gwn), ("bn", t.gbn), ("w1", t.gw1), ("b1", t.gb1),
                      ("w2", t.gw2)):
        ref = v[name].grad
        rms = ref.square().mean().sqrt()
        err = (got.double() - ref).square().mean().sqrt()
        assert err <= 6 * lin.HALF * rms, name
    # without waits between, and replayed from a graph
    t.run()
    torch.cuda.synchronize()
    for a, e in zip(t.results(), want):
        assert torch.equal(a, e)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.run(torch.cuda.current_stream())
    x0 = t.x.clone()
    for k in (0.5, 1.0):
        t.x.copy_(x0 * k)
        graph.replay()
        torch.cuda.synchronize()
    for a, e in zip(t.results(), want):
        assert torch.equal(a, e)


def test_many_calls_share_one_workspace():
    """Calls of every operator follow one another without a wait, with one workspace between
    them all: the bits of the same calls with a synchronisation after each."""
    import random

    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    calls, outs, need = [], [], 256

    def buf(*like):
        new = [torch.zeros_like(v) for v in like]
        outs.extend(new)
        return new

    for m, k, n, a in ((1003, 264, 520, "relu"), (40, 512, 1024, "silu"), (4100, 72, 88, "gelu"),
                       (300, 1024, 264, "none"), (1, 2048, 512, "silu"), (120, 1544, 392, "gelu")):
        t = lin.make(m, k, n, seed=m)
        d = jmix.linear_dims(m, k, n, act=lin.ACTS.index(a))
        nf, nb = jmix.jm_linear_fwd_workspace_size(d), jmix.jm_linear_bwd_workspace_size(d)
        need = max(need, nf, nb)
        out, pre, gx, gw, gb = buf(t["r"], t["r"], t["x"], t["w"], t["b"])
        calls.append(lambda w, t=t, d=d, n=nf, out=out, pre=pre: jmix.jm_linear_fwd(
            d, t["x"], t["w"], out, w, n, bias=t["b"], residual=t["r"], pre=pre))
        calls.append(lambda w, t=t, d=d, n=nb, a=a, pre=pre, gx=gx, gw=gw, gb=gb: jmix.jm_linear_bwd(
            d, t["g"], t["x"], t["w"], w, n, pre=None if a == "none" else pre, g_x=gx, g_w=gw,
            g_bias=gb))
    for t_, d_, f_, e_ in ((1, 264, 1032, 4), (37, 512, 392, 8), (200, 64, 520, 2)):
        m = moe.make(t_, d_, f_, e_, seed=t_)
        d = jmix.moe_dims(t_, d_, f_, e_, 2, router=jmix.JM_ROUTE_SOFTMAX_TOPK)
        n = jmix.jm_moe_fwd_workspace_size(d)
        need = max(need, n)
        out, = buf(m["x"])
        calls.append(lambda w, m=m, d=d, n=n, out=out: jmix.jm_moe_fwd(
            d, m["x"], m["wr"], m["wg"], m["wu"], m["wd"], out, w, n, residual=m["r"]))
    for rows, cols, io in ((700, 1021, "f32"), (2000, 512, "bf16"), (64, 4096, "bf16")):
        t = norm.make(rows, cols, io, seed=cols)
        d = jmix.norm_dims(rows, cols, jmix.JM_BF16 if io == "bf16" else jmix.JM_F32, 1)
        n = jmix.jm_norm_bwd_workspace_size(d)
        need = max(need, n)
        y, gx, gw, gb = buf(t["x"], t["x"], t["w"], t["w"])
        st = torch.zeros(rows, 2, device="cuda")
        calls.append(lambda w, t=t, d=d, n=n, y=y, st=st, gx=gx, gw=gw, gb=gb: (
            jmix.jm_norm_fwd(d, t["x"], t["w"], y, bias=t["b"], stats=st),
            jmix.jm_norm_bwd(d, t["gy"], t["x"], t["w"], st, gx, w, n, g_sum=t["gs"], g_weight=gw,
                             g_bias=gb)))
    ws = devio.workspace(need)
    for c in calls:
        c(ws)
        torch.cuda.synchronize()
        assert jmix.jm_poll_error(ws) == jmix.JM_OK
    want = [v.clone() for v in outs]
    rng = random.Random(2)
    for _ in range(6):
        # (pre holds the same values from the first pass on, so any order will do)
        order = list(range(len(calls)))
        rng.shuffle(order)
        for i in order:
            calls[i](ws)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
