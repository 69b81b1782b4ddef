"""jm_moe_fwd on cuda:0 against the formulas in float64.

Tolerances, from the arithmetic (half = 2^-8, bf16's half step; eps32 = 2^-24).  A product
of bf16 values is exact in float32; a sum of n of them is within 2 n eps32 of sum|a b| in
any order, rounded or truncated, partial tiles included (2 n + 300):
  gate, up   eg = (2 D + 300) eps32 sum|x w|, and eu alike
  silu       ea = 1.13 eg + 32 eps32 |silu| + 4 eps32 (1 + |gate|)   (its slope is below 1.13)
  h          eh = |up| ea + |silu| eu + ea eu, then half of |h| + eh for its rounding to bf16
  product    ey = eh |Wdown| + (2 F + 300) eps32 |h| |Wdown|
  weights    logits carry 16 eps32 sum|x wr| (8 terms in float32, the rest in float64) and
             one rounding of their difference; exp, sum and division 64 eps32:
             ew = w eps32 (64 + 2 max|l - top| + 32 max sum|x wr|)
  out        half |out| + (1 + half) (sum w ey + ew |y|) + (K + 2) eps32 (sum w |y| + |residual|)
"""
import pytest

pytestmark = pytest.mark.gpu

E32, HALF = 2.0 ** -24, 2.0 ** -8
ALL, TOPK = 0, 1


def make(t, d, f, e, seed, skew=0.0):
    import torch
    g = torch.Generator().manual_seed(seed)

    def rn(*s, std=1.0):
        return (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()
    m = dict(x=rn(t, d), wr=rn(e, d, std=d ** -0.5), wg=rn(e, f, d, std=d ** -0.5),
             wu=rn(e, f, d, std=d ** -0.5), wd=rn(e, d, f, std=f ** -0.5), r=rn(t, d))
    if skew:   # every token close to the last expert's row
        m["x"] = (m["x"].float() + skew * m["wr"][-1].float() * d ** 0.5).to(torch.bfloat16)
    return m


def run(m, k, router, residual=True, out=None, stream=None, ws=None, lists=True):
    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    (t, d), (e, f) = m["x"].shape, m["wg"].shape[:2]
    dm = jmix.moe_dims(t, d, f, e, k, router=router)
    n = jmix.jm_moe_fwd_workspace_size(dm)
    if ws is None:
        ws = devio.workspace(n)
        ws.fill_(0xFF)   # NaN: a read of stale scratch would show
    o = torch.full_like(m["x"], float("nan")) if out is None else out
    idx = torch.full((t, k), -1, device="cuda", dtype=torch.int32) if lists else None
    w = torch.full((t, k), float("nan"), device="cuda") if lists else None
    res = {True: m["r"], False: None}[residual] if isinstance(residual, bool) else residual
    jmix.jm_moe_fwd(dm, m["x"], m["wr"], m["wg"], m["wu"], m["wd"], o, ws, n, residual=res,
                    topk_idx=idx, topk_w=w, stream=stream)
    if stream is None:
        assert jmix.jm_poll_error(ws) == jmix.JM_OK, jmix.jm_last_error()
    return o, idx, w


def check(m, k, router, residual=True):
    import torch
    out, idx, w = run(m, k, router, residual)
    x = m["x"].double()
    t = x.shape[0]
    logits = x @ m["wr"].double().t()
    mag = (x.abs() @ m["wr"].double().abs().t()).amax(1, keepdim=True) if t else logits
    val, want = torch.sort(logits, dim=1, descending=True, stable=True)
    # where neighbours are further apart than their error the choice is certain
    near = val[:, :k + 1]
    sure = (near[:, :-1] - near[:, 1:] > 64 * E32 * mag).all(1)
    if near.shape[1] == 1:
        sure = torch.ones(t, dtype=torch.bool, device="cuda")
    assert torch.equal(idx[sure].long(), want[sure, :k])
    pick = idx.long()
    assert (pick >= 0).all() and (pick < logits.shape[1]).all()
    if k > 1:
        s = pick.sort(1).values
        assert (s[:, 1:] != s[:, :-1]).all()
    lp = logits.gather(1, pick)
    w64 = (torch.softmax(lp, 1) if router == TOPK else torch.softmax(logits, 1).gather(1, pick))
    spread = (logits - logits.amax(1, keepdim=True)).abs().amax(1, keepdim=True) if t else lp
    ew = w64 * E32 * (64 + 2 * spread + 32 * mag)
    assert ((w.double() - w64).abs() <= ew).all()
    ref = torch.zeros_like(x)
    err = torch.zeros_like(x)
    size = m["r"].double().abs() if residual else torch.zeros_like(x)
    for e in torch.unique(pick).tolist():
        rows, col = torch.nonzero(pick == e, as_tuple=True)
        wg, wu, wd = (m[q][e].double() for q in ("wg", "wu", "wd"))
        d, f = wg.shape[1], wg.shape[0]
        xr = x[rows]
        g, u = xr @ wg.t(), xr @ wu.t()
        eg = (2 * d + 300) * E32 * (xr.abs() @ wg.abs().t())
        eu = (2 * d + 300) * E32 * (xr.abs() @ wu.abs().t())
        a = g * torch.sigmoid(g)
        ea = 1.13 * eg + 32 * E32 * a.abs() + 4 * E32 * (1 + g.abs())
        h = a * u
        eh = u.abs() * ea + a.abs() * eu + ea * eu
        eh = eh + HALF * (h.abs() + eh)
        y = h @ wd.t()
        ey = eh @ wd.abs().t() + (2 * f + 300) * E32 * ((h.abs() + eh) @ wd.abs().t())
        we, ee = w64[rows, col][:, None], ew[rows, col][:, None]
        ref.index_add_(0, rows, we * y)
        err.index_add_(0, rows, we * ey + ee * (y.abs() + ey))
        size.index_add_(0, rows, we * y.abs())
    if residual:
        ref = ref + m["r"].double()
    tol = HALF * ref.abs() + (1 + HALF) * err + (k + 2) * E32 * size
    assert ((out.double() - ref).abs() <= tol).all()
    return out, idx, w


# tokens, D, F, experts, top_k: one token to the most, widths below one tile and one K
# step, ragged ones, more CTAs than steps, ranges that cut units, every expert or few in use
SHAPES = [(1, 8, 8, 1, 1), (1, 64, 64, 2, 2), (1, 4096, 1024, 16, 2), (1, 1024, 4104, 8, 2),
          (2, 512, 1416, 8, 2), (5, 72, 136, 4, 3), (13, 512, 1416, 8, 2), (16, 264, 520, 7, 2),
          (17, 200, 1000, 5, 1), (33, 256, 264, 24, 8), (64, 1024, 2056, 16, 2),
          (100, 2048, 1032, 16, 2), (200, 64, 64, 2, 2), (255, 1032, 520, 3, 1),
          (256, 128, 136, 256, 8), (256, 256, 512, 1, 1), (256, 2048, 4096, 16, 2)]


@pytest.mark.parametrize("router", [ALL, TOPK])
@pytest.mark.parametrize("t,d,f,e,k", SHAPES)
def test_moe_matches_float64(t, d, f, e, k, router):
    check(make(t, d, f, e, seed=t + d + f + e), k, router, residual=(t + router) % 2 == 0)


@pytest.mark.parametrize("t,e,k", [(40, 16, 1), (256, 16, 2), (256, 64, 1), (130, 4, 2)])
def test_moe_uneven_router(t, e, k):
    """Nearly every token chooses one expert: more rows than a block holds."""
    import torch
    m = make(t, 256, 392, e, seed=t + e, skew=3.0)
    _, idx, _ = check(m, k, TOPK)
    assert torch.bincount(idx.flatten(), minlength=e).max() >= 0.9 * t


def test_moe_ties_go_to_the_lower_index():
    import torch
    m = make(9, 128, 128, 6, seed=3)
    m["wr"][4] = m["wr"][1]
    m["wr"][5] = m["wr"][1]
    _, idx, w = check(m, 3, TOPK)
    for r in range(9):
        got = [i for i in idx[r].tolist() if i in (1, 4, 5)]
        assert got == sorted(got) and got == [1, 4, 5][:len(got)]
    m["wr"].zero_()
    _, idx, w = run(m, 2, ALL)
    assert (idx == torch.tensor([0, 1], device="cuda")).all() and ((w - 1 / 6).abs() <= 4 * E32).all()


def test_moe_nonfinite_tokens_stay_in_their_rows():
    import torch
    m = make(21, 256, 264, 8, seed=4)
    ref, ridx, _ = run(m, 2, TOPK)
    m["x"][3, 100] = float("nan")
    m["x"][7, 9] = float("inf")
    out, idx, w = run(m, 2, TOPK)
    keep = [i for i in range(21) if i not in (3, 7)]
    assert torch.equal(out[keep], ref[keep]) and torch.equal(idx[keep], ridx[keep])
    assert torch.isnan(out[3]).all() and not torch.isfinite(out[7]).any()
    assert (idx[3] == torch.tensor([0, 1], device="cuda")).all()


def test_moe_no_tokens_and_optional_outputs():
    import torch
    m = make(0, 64, 128, 4, seed=1)
    out, _, _ = run(m, 2, ALL)
    assert out.shape[0] == 0
    m = make(30, 512, 768, 8, seed=2)
    out, idx, w = run(m, 2, ALL)
    o2, _, _ = run(m, 2, ALL, lists=False)
    assert torch.equal(out, o2)
    over = m["r"].clone()
    run(m, 2, ALL, residual=over, out=over)
    assert torch.equal(over, out)
    again, idx2, w2 = run(m, 2, ALL)
    assert torch.equal(again, out) and torch.equal(idx2, idx) and torch.equal(w2, w)


@pytest.mark.parametrize("t", [1, 29])
def test_moe_writes_only_its_rows(t):
    import torch
    m = make(t, 256, 264, 8, seed=6)
    ref, _, _ = run(m, 2, TOPK)
    wide = torch.full((t + 8, 256), 5.0, device="cuda", dtype=torch.bfloat16)
    run(m, 2, TOPK, out=wide[4:t + 4])
    assert torch.equal(wide[4:t + 4], ref)
    assert (wide[:4] == 5.0).all() and (wide[t + 4:] == 5.0).all()


@pytest.mark.parametrize("t", [1, 48])
def test_moe_on_another_stream_and_captured(t):
    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    m = make(t, 512, 1024, 8, seed=7)
    ref, _, _ = run(m, 2, TOPK)
    ws = devio.workspace(jmix.jm_moe_fwd_workspace_size(jmix.moe_dims(t, 512, 1024, 8, 2)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(ref)
    run(m, 2, TOPK, out=out, stream=side, ws=ws, lists=False)
    side.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(m, 2, TOPK, out=out, stream=torch.cuda.current_stream(), ws=ws, lists=False)
    x0 = m["x"].clone()
    for s in (1.0, -2.0, 0.5):   # other experts are chosen on replay
        m["x"].copy_(x0 * s)
        graph.replay()
        torch.cuda.synchronize()
        assert jmix.jm_poll_error(ws) == jmix.JM_OK
        assert torch.equal(out, run(m, 2, TOPK)[0])


def test_moe_two_calls_on_two_streams():
    """Two calls at once, each with its own workspace."""
    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    ms = [make(20, 512, 1024, 8, seed=30 + i) for i in range(2)]
    refs = [run(m, 2, TOPK)[0] for m in ms]
    streams = [torch.cuda.Stream() for _ in ms]
    n = jmix.jm_moe_fwd_workspace_size(jmix.moe_dims(20, 512, 1024, 8, 2))
    wss, outs = [devio.workspace(n) for _ in ms], [torch.zeros_like(r) for r in refs]
    torch.cuda.synchronize()
    for _ in range(20):
        for m, s, w, o in zip(ms, streams, wss, outs):
            run(m, 2, TOPK, out=o, stream=s, ws=w, lists=False)
    torch.cuda.synchronize()
    for o, r, w in zip(outs, refs, wss):
        assert torch.equal(o, r)
        assert jmix.jm_poll_error(w) == jmix.JM_OK


# Logits are float64 sums of exact products: within d + 16 roundings of E64 of sum|x w|.  (The
# bound of 16 eps32 at the top of this file was for sums of 8 of them in float32; it holds.)
E64 = 2.0 ** -53


@pytest.mark.parametrize("t,d,e,k", [(1, 4096, 16, 2), (40, 1024, 9, 3), (256, 4096, 16, 2),
                                     (64, 264, 250, 8)])
def test_moe_close_logits_keep_their_order(t, d, e, k):
    """Logits that differ by less than a float32 sum of eight products resolves (a channel of
    x is 30000 times the others) are put in order as float64 sums of d exact products, within
    d + 16 roundings of sum|x w| here and d in the reference, tell them apart."""
    import torch
    m = make(t, d, 64, e, seed=t + e)
    g = torch.Generator().manual_seed(e)
    m["x"][:, 5] = 30000.0
    m["wr"][:] = m["wr"][0]
    m["wr"][:, 5] = 0.0078125
    near = torch.randn(e, 8, generator=g) * 2.0 ** -10    # beside the large channel
    near[:, 5] = 0.0078125
    m["wr"][:, :8] = near.to(torch.bfloat16).cuda()
    x = m["x"].double()
    logits = x @ m["wr"].double().t()
    mag = x.abs() @ m["wr"].double().abs().t().amax(1, keepdim=True)
    val, want = torch.sort(logits, dim=1, descending=True, stable=True)
    gap = val[:, :k] - val[:, 1:k + 1]
    sure = (gap > (2 * d + 32) * E64 * mag).all(1)
    assert sure.float().mean() >= 0.9 and (gap < 64 * E32 * mag).float().mean() >= 0.5
    _, idx, w = run(m, k, TOPK)
    assert torch.equal(idx[sure].long(), want[sure, :k])
    w64 = torch.softmax(val[:, :k], 1)
    # one rounding of each logit's distance from the largest, exp, sum and division
    spread = val[:, :1] - val[:, k - 1:k]
    assert ((w.double() - w64).abs() <= w64 * (E32 * (64 + 2 * spread) + 4 * d * E64 * mag)).all()


@pytest.mark.parametrize("t", [1, 40])
@pytest.mark.parametrize("e", [2, 3, 9, 17, 250])
def test_moe_equal_experts_tie(t, e):
    """Rows of the router that are alike give the same bits whichever CTA sums them, with
    products of very different sizes, whose sum depends on its order."""
    import torch
    m = make(t, 4096, 64, e, seed=e)
    size = torch.exp2(torch.randint(-40, 40, (4096,), generator=torch.Generator().manual_seed(e)))
    m["x"] = (m["x"].float() * size.cuda()).to(torch.bfloat16)
    m["wr"][:] = m["wr"][0]
    k = min(e, 8)
    _, idx, w = run(m, k, TOPK)
    assert (idx == torch.arange(k, device="cuda")).all()
    assert ((w - 1 / k).abs() <= 4 * E32).all()
