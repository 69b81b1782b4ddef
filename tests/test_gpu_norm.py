"""jm_norm_fwd / jm_norm_bwd on cuda:0 against the formulas in float64.

Tolerances, derived from the kernels' arithmetic (float32, one rounding to the
io type at the end; eps32 = 2^-24 the half step of float32, half(io) that of the
io type, relative):
  y      half(io) |y| + eps32 (32 rstd |w| max|s| + 8 (|xh w| + |b|)): a mean or a mean
         square over n values is at most 32 additions deep (16 in a thread, 5 + 5 in the
         two shuffle trees and the last steps), and (s - m) inherits that error scaled by
         max|s|;
  g_x    half(io) |g_x| + 64 eps32 (rstd (|g| + mean|g| + |xh| mean|g xh|) + |g_sum| + c),
         c = rstd^2 (|x| + |m|) mean|g xh| for the rounding of xh before its use;
  g_w    half(io) |g_w| + (rows + 64) eps32 sum|g_y xh| (a sum of `rows` terms).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24


def half(io):
    return 2.0 ** -8 if io == "bf16" else 2.0 ** -24


def make(rows, cols, io, seed, scale=2.0, offset=0.5):
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32

    def rn(*s, std=1.0, mean=0.0):
        return (torch.randn(*s, generator=g) * std + mean).to(dt).cuda()
    return dict(x=rn(rows, cols, std=scale, mean=offset), r=rn(rows, cols), w=rn(cols, std=0.3, mean=1.0),
                b=rn(cols), gy=rn(rows, cols), gs=rn(rows, cols))


def ref_fwd(x, r, w, b, kind, eps):
    import torch
    s = x if r is None else (x.float() + r.float()).to(x.dtype)
    s64 = s.double()
    m = s64.mean(1, keepdim=True) if kind else torch.zeros_like(s64[:, :1])
    rstd = (((s64 - m) ** 2).mean(1, keepdim=True) + eps) ** -0.5
    xh = (s64 - m) * rstd
    y = xh * w.double() + (0 if b is None else b.double())
    return s, m, rstd, xh, y


def run_fwd(t, io, kind, residual, bias, x=None, eps=1e-6):
    import torch
    from mamba_selective_scan_jamba_b200 import jmix
    x = t["x"] if x is None else x
    rows, cols = x.shape
    d = jmix.norm_dims(rows, cols, jmix.JM_BF16 if io == "bf16" else jmix.JM_F32, kind, eps,
                       x_stride=x.stride(0) if rows > 1 else None)
    y = torch.full((rows, cols), float("nan"), device="cuda", dtype=x.dtype)
    s = torch.full_like(y, float("nan")) if residual else None
    st = torch.full((rows, 2), float("nan"), device="cuda")
    jmix.jm_norm_fwd(d, x, t["w"], y, bias=t["b"] if bias else None,
                     residual=t["r"] if residual else None, sum_out=s, stats=st)
    torch.cuda.synchronize()
    return d, y, s, st


def check_fwd(t, io, kind, residual, bias, x=None, eps=1e-6):
    import torch
    x = t["x"] if x is None else x
    d, y, s, st = run_fwd(t, io, kind, residual, bias, x, eps)
    rs, m, rstd, xh, yr = ref_fwd(x, t["r"] if residual else None, t["w"], t["b"] if bias else None,
                                  kind, eps)
    if residual:
        assert torch.equal(s, rs)
    w, b = t["w"].double().abs(), (t["b"].double().abs() if bias else 0.0)
    top = rs.double().abs().amax(1, keepdim=True)
    tol = half(io) * yr.abs() + E32 * (32 * rstd * w * top + 8 * (xh.abs() * w + b))
    assert ((y.double() - yr).abs() <= tol).all()
    assert ((st[:, :1].double() - m).abs() <= 32 * E32 * top).all()
    assert ((st[:, 1:].double() - rstd).abs() <= 64 * E32 * rstd * (1 + top * rstd)).all()
    return d, rs, st


def check_bwd(t, io, kind, d, x, st, g_sum, alias=False):
    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    rows, cols = x.shape
    n = jmix.jm_norm_bwd_workspace_size(d)
    ws = devio.workspace(n)
    ws.fill_(0xFF)   # NaN: a read of stale scratch would show
    gy = t["gy"].clone()
    gx = gy if alias else torch.full_like(gy, float("nan"))
    gw = torch.full_like(t["w"], float("nan"))
    gb = torch.full_like(t["w"], float("nan")) if kind else None
    jmix.jm_norm_bwd(d, gy, x, t["w"], st, gx, ws, n, g_sum=t["gs"] if g_sum else None,
                     g_weight=gw, g_bias=gb)
    assert jmix.jm_poll_error(ws) == jmix.JM_OK
    m, rstd = st[:, :1].double(), st[:, 1:].double()
    g0, w = t["gy"].double(), t["w"].double()
    xh = (x.double() - m) * rstd
    g = g0 * w
    c1 = (g * xh).mean(1, keepdim=True)
    c0 = g.mean(1, keepdim=True) if kind else torch.zeros_like(c1)
    gs = t["gs"].double() if g_sum else torch.zeros_like(g)
    gxr = rstd * (g - c0 - xh * c1) + gs
    mag = (rstd * (g.abs() + g.abs().mean(1, keepdim=True)
                   + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) + gs.abs()
           + rstd ** 2 * (x.double().abs() + m.abs()) * (g * xh).abs().mean(1, keepdim=True))
    assert ((gx.double() - gxr).abs() <= half(io) * gxr.abs() + 64 * E32 * mag).all()
    gwr = (g0 * xh).sum(0)
    mag_w = (g0 * xh).abs().sum(0) + (g0.abs() * (x.double().abs() + m.abs()) * rstd).sum(0) / max(rows, 1)
    assert ((gw.double() - gwr).abs() <= half(io) * gwr.abs() + (rows + 64) * E32 * mag_w).all()
    if kind:
        gbr = g0.sum(0)
        assert ((gb.double() - gbr).abs()
                <= half(io) * gbr.abs() + (rows + 64) * E32 * g0.abs().sum(0)).all()
    return gx, gw, gb


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 1), (3, 7), (9, 8), (1, 31), (33, 33), (1, 4096),
                                       (257, 256), (1000, 264), (2, 1021), (513, 1024), (70, 2048),
                                       (700, 4096), (40, 5120), (21, 8192), (5, 8191), (17, 16384),
                                       (3, 16383), (20011, 24)])
def test_norm_matches_float64(rows, cols, kind, io):
    t = make(rows, cols, io, seed=rows * 31 + cols)
    d, s, st = check_fwd(t, io, kind, residual=False, bias=bool(kind))
    check_bwd(t, io, kind, d, s, st, g_sum=rows % 2 == 1)
    d, s, st = check_fwd(t, io, kind, residual=True, bias=False)
    check_bwd(t, io, kind, d, s, st, g_sum=rows % 2 == 0, alias=True)


@pytest.mark.parametrize("io,stride", [("bf16", 520), ("bf16", 517), ("f32", 516), ("f32", 515)])
def test_norm_of_strided_rows(io, stride):
    """x is a slice of a wider matrix; what lies between its rows is not touched."""
    import torch
    t = make(37, 512, io, seed=4)
    wide = torch.full((37, stride), 7.0, device="cuda", dtype=t["x"].dtype)
    wide[:, :512] = t["x"]
    x = wide[:, :512]
    d, s, st = check_fwd(t, io, 1, residual=False, bias=True, x=x)
    check_bwd(t, io, 1, d, x, st, g_sum=True)
    check_fwd(t, io, 0, residual=True, bias=False, x=x)
    assert (wide[:, 512:] == 7.0).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_norm_in_place(io):
    """y and sum over x and the residual give the bits of separate buffers."""
    import torch
    from mamba_selective_scan_jamba_b200 import jmix
    for cols in (4096, 333):
        t = make(50, cols, io, seed=6)
        d, y, s, _ = run_fwd(t, io, 0, residual=True, bias=False)
        x2, r2 = t["x"].clone(), t["r"].clone()
        jmix.jm_norm_fwd(d, x2, t["w"], x2, residual=r2, sum_out=r2)
        assert torch.equal(x2, y) and torch.equal(r2, s)


def test_norm_rows_far_from_zero():
    """Rows whose mean is 500 times their spread: the variance does not cancel."""
    t = make(64, 2048, "f32", seed=8, scale=1.0, offset=500.0)
    check_fwd(t, "f32", 1, residual=False, bias=False)


def test_norm_constant_and_zero_rows():
    import torch
    t = make(4, 512, "f32", seed=9)
    t["x"][0] = 0.0
    t["x"][1] = 3.0
    d, y, s, st = run_fwd(t, "f32", 1, residual=False, bias=False)
    assert torch.isfinite(y).all() and not y[0].any()
    assert y[1].abs().max() < 1e-3


def test_norm_nonfinite_rows_stay_in_their_rows():
    import torch
    t = make(6, 1000, "bf16", seed=10)
    ref = run_fwd(t, "bf16", 1, residual=False, bias=False)[1].clone()
    t["x"][2, 17] = float("inf")
    t["x"][4, 3] = float("nan")
    y = run_fwd(t, "bf16", 1, residual=False, bias=False)[1]
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], ref[keep])
    assert torch.isnan(y[2]).any() and torch.isnan(y[4]).all()


def test_norm_no_rows():
    import torch
    t = make(0, 64, "bf16", seed=1)
    d, s, st = check_fwd(t, "bf16", 1, residual=True, bias=True)
    _, gw, gb = check_bwd(t, "bf16", 1, d, s, st, g_sum=False)
    assert not gw.any() and not gb.any()


def test_norm_bwd_same_bits_twice_and_without_sums():
    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    t = make(3000, 1024, "bf16", seed=12)
    d, s, st = check_fwd(t, "bf16", 1, residual=False, bias=True)
    a = check_bwd(t, "bf16", 1, d, s, st, g_sum=True)
    b = check_bwd(t, "bf16", 1, d, s, st, g_sum=True)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    n = jmix.jm_norm_bwd_workspace_size(d)
    gx = torch.empty_like(a[0])
    jmix.jm_norm_bwd(d, t["gy"], s, t["w"], st, gx, devio.workspace(n), n, g_sum=t["gs"])
    assert torch.equal(gx, a[0])
    assert jmix.jm_last_launch_count() == 1 and jmix.jm_last_kernel_name(0) == "k_norm_bwd"


def test_norm_gradient_against_differences():
    """float32 directional derivative of sum(y c) along a direction, by central
    differences of the float64 formula."""
    import torch
    t = make(5, 48, "f32", seed=14)
    for kind in (0, 1):
        d, s, st = check_fwd(t, "f32", kind, residual=False, bias=False)
        gx, gw, _ = check_bwd(t, "f32", kind, d, s, st, g_sum=False)
        v, u, h = t["r"].double(), t["b"].double(), 1e-5

        def loss(k):
            x = t["x"].double() + k * h * v
            w = t["w"].double() + k * h * u
            return (ref_fwd(x, None, w, None, kind, 1e-6)[4] * t["gy"].double()).sum()
        num = (loss(1) - loss(-1)) / (2 * h)
        ana = (gx.double() * v).sum() + (gw.double() * u).sum()
        assert abs(num - ana) <= 1e-4 * (1 + abs(num))


def test_norm_on_another_stream_and_captured():
    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    t = make(300, 4096, "bf16", seed=15)
    d, y0, s0, st0 = run_fwd(t, "bf16", 1, residual=True, bias=True)
    gx0, gw0, gb0 = check_bwd(t, "bf16", 1, d, s0, st0, g_sum=True)
    n = jmix.jm_norm_bwd_workspace_size(d)
    ws = devio.workspace(n)
    y, s, st = torch.zeros_like(y0), torch.zeros_like(s0), torch.zeros_like(st0)
    gx, gw, gb = torch.zeros_like(gx0), torch.zeros_like(gw0), torch.zeros_like(gb0)
    x = t["x"].clone()

    def both(stream):
        jmix.jm_norm_fwd(d, x, t["w"], y, bias=t["b"], residual=t["r"], sum_out=s, stats=st,
                         stream=stream)
        jmix.jm_norm_bwd(d, t["gy"], s, t["w"], st, gx, ws, n, g_sum=t["gs"], g_weight=gw,
                         g_bias=gb, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    side.synchronize()
    for a, b in ((y, y0), (s, s0), (st, st0), (gx, gx0), (gw, gw0), (gb, gb0)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(torch.cuda.current_stream())
    for k in range(3):   # replays with changed inputs in place
        x.copy_(t["x"] * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        d2, y2, s2, st2 = run_fwd(dict(t, x=x), "bf16", 1, residual=True, bias=True)
        assert torch.equal(y, y2) and torch.equal(s, s2) and torch.equal(st, st2)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("rows,cols", [(5000, 1), (2501, 3), (9999, 7), (20000, 131), (3001, 1021),
                                       (1301, 943), (701, 4357), (401, 8191), (307, 16383),
                                       (3000, 514), (2999, 2052)])
def test_norm_of_many_ragged_rows(rows, cols, kind, io):
    """Rows that are no multiple of 16 bytes, more than one round of the GPU's CTAs."""
    t = make(rows, cols, io, seed=rows + cols)
    d, s, st = check_fwd(t, io, kind, residual=True, bias=bool(kind))
    check_bwd(t, io, kind, d, s, st, g_sum=True)
    d, s, st = check_fwd(t, io, kind, residual=False, bias=False)
    check_bwd(t, io, kind, d, s, st, g_sum=False, alias=True)


@pytest.mark.parametrize("rows", [2000, 2007])
def test_norm_of_ragged_rows_in_place_and_in_bounds(rows):
    """y over x, sum over the residual, g_x over g_sum; the values around the tensors stay."""
    import torch
    from mamba_selective_scan_jamba_b200 import devio, jmix
    cols = 1013
    t = make(rows, cols, "bf16", seed=3)
    d, y, s, st = run_fwd(t, "bf16", 1, residual=True, bias=True)
    n = rows * cols

    def guarded(v):
        g = torch.full((n + 64,), 9.0, device="cuda", dtype=torch.bfloat16)
        g[:n] = v.flatten()
        return g, g[:n].view(rows, cols)
    xg, x = guarded(t["x"])
    rg, r = guarded(t["r"])
    jmix.jm_norm_fwd(d, x, t["w"], x, bias=t["b"], residual=r, sum_out=r)
    assert torch.equal(x, y) and torch.equal(r, s)
    nb = jmix.jm_norm_bwd_workspace_size(d)
    ws = devio.workspace(nb)
    gx = torch.empty_like(y)
    jmix.jm_norm_bwd(d, t["gy"], s, t["w"], st, gx, ws, nb, g_sum=t["gs"])
    sg, over = guarded(t["gs"])
    jmix.jm_norm_bwd(d, t["gy"], s, t["w"], st, over, ws, nb, g_sum=over)
    assert torch.equal(over, gx)
    for g in (xg, rg, sg):
        assert (g[n:] == 9.0).all()
