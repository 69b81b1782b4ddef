"""jm_linear_fwd / jm_linear_bwd on cuda:0 against the formulas in float64.

Tolerances, from the arithmetic (half = 2^-8, bf16's half step; eps32 = 2^-24).  A
product of K bf16 pairs is exact in float32 and its sum of K terms, whatever the
order, is within K eps32 of sum|a b| when every addition rounds to nearest, and
within twice that when the tensor core truncates:
  pre   half |p| + (2 K + 8) eps32 (sum|x w| + |bias|)
  out   half |out| + 2 * (the product's error) + eps_act + eps32 |residual|: the
        activations' slopes are below 1.13, and their own error (erfc, exp, division)
        is below 32 eps32 |act(p)| plus 4 eps32 (1 + |p|) of argument rounding;
  g_p   is rounded to bf16 before the products, so g_x and g_w carry half (1 + half)
        of sum|g_p w| beside the sum's error; act' itself is within 64 eps32 (1 + |p|)
        of its value, at most 64 eps32 (1 + |p|) |g_out| per term;
  g_bias sums unrounded g_out act' over the rows: (rows + 64 (1 + max|p|)) eps32 sum|g_out|.
"""
import pytest

pytestmark = pytest.mark.gpu

E32, HALF = 2.0 ** -24, 2.0 ** -8
ACTS = ["none", "relu", "gelu", "silu"]


def make(m, k, n, seed):
    import torch
    g = torch.Generator().manual_seed(seed)

    def rn(*s, std=1.0):
        return (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()
    return dict(x=rn(m, k), w=rn(n, k, std=k ** -0.5), b=rn(n), r=rn(m, n), g=rn(m, n))


def act(v, a):
    import torch
    if a == "relu":
        return torch.clamp(v, min=0)
    if a == "gelu":
        return v * torch.special.ndtr(v)
    if a == "silu":
        return v * torch.sigmoid(v)
    return v


def act_grad(v, a):
    import torch
    if a == "relu":
        return (v > 0).double()
    if a == "gelu":
        return torch.special.ndtr(v) + v * torch.exp(-v * v / 2) / (2 * torch.pi) ** 0.5
    if a == "silu":
        s = torch.sigmoid(v)
        return s * (1 + v * (1 - s))
    return torch.ones_like(v)


def run_fwd(t, a, bias=True, residual=True, pre=True, out=None, stream=None, ws=None):
    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    m, k, n = t["x"].shape[0], t["x"].shape[1], t["w"].shape[0]
    d = jmix.linear_dims(m, k, n, act=ACTS.index(a))
    nb = jmix.jm_linear_fwd_workspace_size(d)
    if ws is None:
        ws = devio.workspace(nb)
        ws.fill_(0xFF)   # NaN: a read of stale scratch would show
    o = torch.full((m, n), float("nan"), device="cuda", dtype=torch.bfloat16) if out is None else out
    p = torch.full_like(o, float("nan")) if pre else None
    res = {True: t["r"], False: None}[residual] if isinstance(residual, bool) else residual
    jmix.jm_linear_fwd(d, t["x"], t["w"], o, ws, nb, bias=t["b"] if bias else None,
                       residual=res, pre=p, stream=stream)
    if stream is None:
        assert jmix.jm_poll_error(ws) == jmix.JM_OK, jmix.jm_last_error()
    return o, p


def check_fwd(t, a, bias=True, residual=True):
    out, pre = run_fwd(t, a, bias, residual)
    x, w = t["x"].double(), t["w"].double()
    b = t["b"].double() if bias else 0.0 * t["b"].double()
    p = x @ w.t() + b
    e = (2 * x.shape[1] + 8) * E32 * (x.abs() @ w.abs().t() + b.abs())
    assert ((pre.double() - p).abs() <= HALF * p.abs() + e).all()
    y = act(p, a)
    ref = y + (t["r"].double() if residual else 0)
    tol = (HALF * ref.abs() + 2 * e + 32 * E32 * y.abs() + 4 * E32 * (1 + p.abs())
           + (E32 * t["r"].double().abs() if residual else 0))
    assert ((out.double() - ref).abs() <= tol).all()
    return out, pre


def run_bwd(t, a, pre, want=("g_x", "g_w", "g_bias")):
    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    m, k, n = t["x"].shape[0], t["x"].shape[1], t["w"].shape[0]
    d = jmix.linear_dims(m, k, n, act=ACTS.index(a))
    nb = jmix.jm_linear_bwd_workspace_size(d)
    ws = devio.workspace(nb)
    ws.fill_(0xFF)
    o = dict(g_x=torch.full_like(t["x"], float("nan")), g_w=torch.full_like(t["w"], float("nan")),
             g_bias=torch.full_like(t["b"], float("nan")))
    o = {q: v for q, v in o.items() if q in want}
    jmix.jm_linear_bwd(d, t["g"], t["x"] if "g_w" in o else None, t["w"] if "g_x" in o else None,
                       ws, nb, pre=None if a == "none" else pre, **o)
    assert jmix.jm_poll_error(ws) == jmix.JM_OK, jmix.jm_last_error()
    return o


def check_bwd(t, a, pre):
    o = run_bwd(t, a, pre)
    m, k = t["x"].shape
    n = t["w"].shape[0]
    x, w, g, p = t["x"].double(), t["w"].double(), t["g"].double(), pre.double()
    gp = g * act_grad(p, a)
    rnd = 0.0 if a == "none" else HALF * (1 + HALF)
    dg = rnd * gp.abs() + (0.0 if a == "none" else 64 * E32) * (1 + p.abs()) * g.abs()
    for q, ref, e in (("g_x", gp @ w, dg @ w.abs() + (2 * n + 8) * E32 * (gp.abs() @ w.abs())),
                      ("g_w", gp.t() @ x,
                       dg.t() @ x.abs() + (2 * m + 8) * E32 * (gp.abs().t() @ x.abs()))):
        assert ((o[q].double() - ref).abs() <= HALF * ref.abs() + (1 + HALF) * e).all(), q
    top = 1 + (p.abs().max() if p.numel() else 0)
    ref = gp.sum(0)
    assert ((o["g_bias"].double() - ref).abs()
            <= HALF * ref.abs() + (m + 64 * top) * E32 * g.abs().sum(0)).all()
    return o


# one row to many, row tiles that end inside a tile, widths below one tile and one K
# chunk, both tile widths, K splits, and more work items than CTA pairs
SHAPES = [(1, 8, 8), (1, 64, 64), (3, 72, 136), (16, 264, 520), (17, 4096, 1024), (64, 1032, 2056),
          (128, 512, 4096), (129, 520, 264), (130, 4096, 512), (255, 200, 1000), (256, 8192, 4096),
          (257, 1024, 264), (300, 64, 2048), (1003, 1032, 2056), (2048, 1024, 4096),
          (5000, 328, 328), (4100, 2048, 4104)]


@pytest.mark.parametrize("m,k,n", SHAPES)
def test_linear_matches_float64(m, k, n):
    i = (m + k + n) // 8
    a = ACTS[i % 4]
    t = make(m, k, n, seed=m + k + n)
    _, pre = check_fwd(t, a, bias=i % 3 != 0, residual=i % 2 == 0)
    check_bwd(t, a, pre)


@pytest.mark.parametrize("a", ACTS)
@pytest.mark.parametrize("m", [1, 33, 200, 700])
def test_linear_activations(a, m):
    t = make(m, 256, 512, seed=m)
    t["b"] *= 4    # both tails of the activations
    for bias in (True, False):
        for residual in (True, False):
            _, pre = check_fwd(t, a, bias, residual)
    check_bwd(t, a, pre)


@pytest.mark.parametrize("m", [5, 140, 600])
def test_linear_optional_outputs_and_in_place(m):
    import torch
    t = make(m, 512, 1024, seed=3)
    out, pre = run_fwd(t, "silu")
    o2, _ = run_fwd(t, "silu", pre=False)
    assert torch.equal(out, o2)
    over = t["r"].clone()
    run_fwd(t, "silu", residual=over, out=over)
    assert torch.equal(over, out)
    full = run_bwd(t, "silu", pre)
    for want in (("g_x",), ("g_w",), ("g_bias",), ("g_x", "g_bias"), ()):
        part = run_bwd(t, "silu", pre, want)
        for q, v in part.items():
            assert torch.equal(v, full[q]), (want, q)
    again = run_bwd(t, "silu", pre)
    for q in full:
        assert torch.equal(again[q], full[q])


def test_linear_no_rows():
    t = make(0, 64, 128, seed=1)
    out, pre = run_fwd(t, "gelu")
    o = run_bwd(t, "gelu", pre)
    assert out.shape[0] == 0 and not o["g_w"].any() and not o["g_bias"].any()


@pytest.mark.parametrize("m", [7, 300])
def test_linear_nonfinite_rows_stay_in_their_rows(m):
    import torch
    t = make(m, 256, 512, seed=5)
    ref, _ = run_fwd(t, "none")
    t["x"][2, 100] = float("inf")
    t["x"][4, 1] = float("nan")
    out, _ = run_fwd(t, "none")
    keep = [i for i in range(m) if i not in (2, 4)]
    assert torch.equal(out[keep], ref[keep])
    assert torch.isnan(out[4]).all() and not torch.isfinite(out[2]).any()


@pytest.mark.parametrize("m", [9, 300])
def test_linear_writes_only_its_rows(m):
    """Rows before and behind the outputs stay as they were."""
    import torch
    t = make(m, 256, 264, seed=6)
    wide = torch.full((m + 8, 264), 5.0, device="cuda", dtype=torch.bfloat16)
    out = wide[4:m + 4]
    ref, _ = run_fwd(t, "relu")
    run_fwd(t, "relu", out=out)
    assert torch.equal(out, ref)
    assert (wide[:4] == 5.0).all() and (wide[m + 4:] == 5.0).all()


@pytest.mark.parametrize("m", [4, 256])
def test_linear_on_another_stream_and_captured(m):
    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    t = make(m, 1024, 2048, seed=7)
    ref, _ = run_fwd(t, "gelu")
    d = jmix.linear_dims(m, 1024, 2048, act=2)
    ws = devio.workspace(jmix.jm_linear_fwd_workspace_size(d))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(ref)
    run_fwd(t, "gelu", pre=False, out=out, stream=side, ws=ws)
    side.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_fwd(t, "gelu", pre=False, out=out, stream=torch.cuda.current_stream(), ws=ws)
    x0 = t["x"].clone()
    for s in (1.0, -2.0, 0.5):
        t["x"].copy_(x0 * s)
        graph.replay()
        torch.cuda.synchronize()
        assert jmix.jm_poll_error(ws) == jmix.JM_OK
        want, _ = run_fwd(t, "gelu")
        assert torch.equal(out, want)


def test_linear_two_calls_on_two_streams():
    """Two calls at once, each with its own workspace."""
    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    ts = [make(48, 4096, 1024, seed=20 + i) for i in range(2)]
    refs = [run_fwd(t, "silu")[0] for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    wss = [devio.workspace(jmix.jm_linear_fwd_workspace_size(jmix.linear_dims(48, 4096, 1024, 3)))
           for _ in ts]
    outs = [torch.zeros_like(r) for r in refs]
    torch.cuda.synchronize()
    for _ in range(20):
        for t, s, w, o in zip(ts, streams, wss, outs):
            run_fwd(t, "silu", pre=False, out=o, stream=s, ws=w)
    torch.cuda.synchronize()
    for o, r, w in zip(outs, refs, wss):
        assert torch.equal(o, r)
        assert jmix.jm_poll_error(w) == jmix.JM_OK


def test_linear_gradient_against_differences():
    """Directional derivative of sum(out c) by central differences of the float64
    formula, against the kernel's gradients: bf16 gradients, so 2 half steps of the
    sum of magnitudes."""
    t = make(37, 128, 256, seed=11)
    for a in ACTS:
        _, pre = check_fwd(t, a)
        o = run_bwd(t, a, pre)
        import torch
        g = torch.Generator().manual_seed(1)
        dx = torch.randn(t["x"].shape, generator=g).cuda().double()
        dw = torch.randn(t["w"].shape, generator=g).cuda().double()
        db = torch.randn(t["b"].shape, generator=g).cuda().double()
        h = 1e-6

        def loss(s):
            p = ((t["x"].double() + s * h * dx) @ (t["w"].double() + s * h * dw).t()
                 + t["b"].double() + s * h * db)
            return (act(p, a) * t["g"].double()).sum()
        num = (loss(1) - loss(-1)) / (2 * h)
        parts = [(o["g_x"], dx), (o["g_w"], dw), (o["g_bias"], db)]
        ana = sum((q.double() * v).sum() for q, v in parts)
        # each entry is within about 3 half steps of its magnitude; signs are random
        mag = sum((q.double() * v).square().sum() for q, v in parts).sqrt()
        assert abs(num - ana) <= 8 * HALF * mag


# few rows over long contracted indexes, with each size of a cluster; two pairs on a tile,
# both widths, and a last row tile whose second half is empty
JOINED = [(1, 1024, 1024), (2, 16384, 136), (8, 4096, 1024), (40, 6000, 3000), (64, 520, 512),
          (100, 4104, 1000), (150, 4096, 8192), (160, 4104, 264), (192, 8192, 520),
          (300, 2048, 1304), (390, 5256, 2008), (530, 5496, 2208), (818, 4200, 1440),
          (2619, 1048, 96)]


@pytest.mark.parametrize("m,k,n", JOINED)
def test_linear_products_joined_in_shared_memory(m, k, n):
    import torch
    i = m % 4
    t = make(m, k, n, seed=m + 2 * n)
    out, pre = check_fwd(t, ACTS[i], bias=i % 2 == 0, residual=True)
    again, _ = run_fwd(t, ACTS[i], bias=i % 2 == 0, residual=True)
    assert torch.equal(out, again)
    check_fwd(t, "none", bias=False, residual=False)
    check_bwd(t, ACTS[i], pre)


# tiles a CTA pair: one to three of short and of long contracted indexes (fewer K chunks than
# ring stages, and more), a last tile with an empty half or with fewer columns
DRAINED = [(300, 64, 2048), (4096, 64, 2048), (9000, 72, 2056), (19000, 8, 520), (2305, 1032, 4104),
           (5000, 1544, 2048), (10000, 1544, 264)]


@pytest.mark.parametrize("m,k,n", DRAINED)
def test_linear_pairs_end_with_every_signal_received(m, k, n):
    """CTAs of one launch follow those of another on their SM at once: with a signal still on
    its way to a CTA that has left, the next one's barriers would count it.  Every wait at the
    kernel's end is satisfied (the error header says so) and all launches give the same bits."""
    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    t = make(m, k, n, seed=m + k)
    out, pre = run_fwd(t, "relu")
    o = run_bwd(t, "relu", pre)
    d = jmix.linear_dims(m, k, n, act=ACTS.index("relu"))
    nf, nb = jmix.jm_linear_fwd_workspace_size(d), jmix.jm_linear_bwd_workspace_size(d)
    wss = [devio.workspace(max(nf, nb)) for _ in range(16)]
    outs = [(torch.empty_like(out), torch.empty_like(o["g_x"]), torch.empty_like(o["g_w"]))
            for _ in range(2)]
    for i, ws in enumerate(wss):
        q = outs[i % 2]
        jmix.jm_linear_fwd(d, t["x"], t["w"], q[0], ws, nf, bias=t["b"], residual=t["r"])
        jmix.jm_linear_bwd(d, t["g"], t["x"], t["w"], ws, nb, pre=pre, g_x=q[1], g_w=q[2])
    torch.cuda.synchronize()
    for ws in wss:
        assert jmix.jm_poll_error(ws) == jmix.JM_OK, jmix.jm_last_error()
    for q in outs:
        assert torch.equal(q[0], out) and torch.equal(q[1], o["g_x"]) and torch.equal(q[2], o["g_w"])


@pytest.mark.parametrize("m", [16, 700])
def test_linear_gelu_tail(m):
    """GELU and its derivative keep their relative accuracy far below zero, where they are the
    normal tail: float32 values of up to 12 squared and halved carry 72 * 2 roundings into the
    exponential, 2^-16 in all, then one rounding to bf16.  The derivative is the difference
    of the two terms that the bound adds.  (The reference's tail by erfc: torch's ndtr is 0
    below -8.3 on a GPU.)"""
    import torch
    v = -torch.exp2(torch.linspace(-6, 3.58, 8 * m, dtype=torch.float64))   # to -11.96
    x = v.to(torch.bfloat16).cuda().view(m, 8)
    eye = torch.eye(8, device="cuda", dtype=torch.bfloat16)
    t = dict(x=x, w=eye, b=torch.zeros(8, device="cuda", dtype=torch.bfloat16),
             r=torch.zeros_like(x), g=torch.ones_like(x))
    out, pre = run_fwd(t, "gelu", bias=False, residual=False)
    assert torch.equal(pre, x)
    p = x.double()
    phi = 0.5 * torch.special.erfc(-p / 2 ** 0.5)
    ref = p * phi
    assert ((out.double() - ref).abs() <= (HALF + 2.0 ** -16) * ref.abs()).all()
    gx = run_bwd(t, "gelu", pre, ("g_x",))["g_x"].double()
    dens = p.abs() * torch.exp(-p * p / 2) / (2 * torch.pi) ** 0.5
    tol = HALF * (phi - dens).abs() + 2.0 ** -16 * (phi + dens)
    assert ((gx - (phi - dens)).abs() <= tol).all()
