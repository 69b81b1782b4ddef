"""CPU checks of the decoder block's operators: the host refuses bad arguments
before any launch (no call below reaches the GPU)."""
import pytest

from mamba_selective_scan_jamba_b200 import build, jmix

F = 1 << 40        # fake, never dereferenced device addresses, far apart
G = 1 << 36
W = 1 << 45        # fake workspace


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_libjmix()
    return jmix.load()


def norm_fwd(d, **over):
    a = dict(x=F, weight=F + 2 * G, y=F + 3 * G, bias=None, residual=None, sum_out=None, stats=None)
    a.update(over)
    return jmix.jm_norm_fwd(d, **a, stream=0, check=False)


def norm_bwd(d, nbytes=None, **over):
    a = dict(g_y=F, x=F + G, weight=F + 2 * G, stats=F + 3 * G, g_x=F + 4 * G, workspace=W,
             ws_bytes=jmix.jm_norm_bwd_workspace_size(d) if nbytes is None else nbytes)
    a.update(over)
    return jmix.jm_norm_bwd(d, **a, stream=0, check=False)


@pytest.mark.parametrize("over,code,msg", [
    (dict(rows=-1), jmix.JM_ERR_INVALID_ARG, "rows"),
    (dict(cols=0), jmix.JM_ERR_INVALID_ARG, "cols"),
    (dict(x_stride=31), jmix.JM_ERR_INVALID_ARG, "x_stride"),
    (dict(cols=16385), jmix.JM_ERR_UNSUPPORTED, "16384"),
    (dict(rows=1 << 32), jmix.JM_ERR_INVALID_ARG, "large"),
    (dict(eps=-1.0), jmix.JM_ERR_INVALID_ARG, "eps"),
    (dict(eps=float("nan")), jmix.JM_ERR_INVALID_ARG, "eps"),
    (dict(io=5), jmix.JM_ERR_INVALID_ARG, "io dtype"),
    (dict(kind=2), jmix.JM_ERR_INVALID_ARG, "kind"),
])
def test_norm_rejects_bad_dims(over, code, msg):
    kw = dict(rows=4, cols=32)
    kw.update(over)
    d = jmix.norm_dims(**kw)
    assert norm_fwd(d) == code and msg in jmix.jm_last_error()
    assert norm_bwd(d, nbytes=1 << 20) == code and msg in jmix.jm_last_error()
    assert jmix.jm_norm_bwd_workspace_size(d) == 0
    d = jmix.norm_dims(4, 32)
    d.reserved = 1
    assert norm_fwd(d) == jmix.JM_ERR_INVALID_ARG and "reserved" in jmix.jm_last_error()


def test_norm_rejects_bad_pointers():
    d = jmix.norm_dims(4, 32, kind=jmix.JM_NORM_LAYER)
    bad = jmix.JM_ERR_INVALID_ARG
    for k in ("x", "weight", "y"):
        assert norm_fwd(d, **{k: None}) == bad and "NULL" in jmix.jm_last_error(), k
        assert norm_fwd(d, **{k: F + 8}) == bad and "aligned" in jmix.jm_last_error(), k
    assert norm_fwd(d, residual=F + 5 * G) == bad and "sum is NULL" in jmix.jm_last_error()
    assert norm_fwd(d, sum_out=F + 5 * G) == bad and "without a residual" in jmix.jm_last_error()
    # y over the weight, half over x, over the sum; sum half over the residual
    assert norm_fwd(d, y=F + 2 * G) == bad and "y overlaps weight" in jmix.jm_last_error()
    assert norm_fwd(d, y=F + 64) == bad and "y overlaps x" in jmix.jm_last_error()
    r = F + 5 * G
    assert norm_fwd(d, residual=r, sum_out=F + 3 * G) == bad
    assert "sum overlaps y" in jmix.jm_last_error()
    assert norm_fwd(d, residual=r, sum_out=r + 16) == bad
    assert "sum overlaps residual" in jmix.jm_last_error()
    assert norm_fwd(d, stats=F) == bad and "stats overlaps x" in jmix.jm_last_error()
    strided = jmix.norm_dims(4, 32, kind=jmix.JM_NORM_LAYER, x_stride=40)
    assert norm_fwd(strided, y=F) == bad and "y overlaps x" in jmix.jm_last_error()
    rms = jmix.norm_dims(4, 32)
    assert norm_fwd(rms, bias=F + G) == bad and "bias" in jmix.jm_last_error()


def test_norm_bwd_rejects_bad_pointers():
    d = jmix.norm_dims(4, 32)
    bad = jmix.JM_ERR_INVALID_ARG
    for k in ("g_y", "x", "weight", "stats", "g_x"):
        assert norm_bwd(d, **{k: None}) == bad and "NULL" in jmix.jm_last_error(), k
    assert norm_bwd(d, g_x=F + G) == bad and "g_x overlaps x" in jmix.jm_last_error()
    assert norm_bwd(d, g_x=F + 16) == bad and "g_x overlaps g_y" in jmix.jm_last_error()
    assert norm_bwd(d, g_weight=F + 2 * G) == bad
    assert norm_bwd(d, g_bias=F + 6 * G) == bad and "g_bias" in jmix.jm_last_error()
    n = jmix.jm_norm_bwd_workspace_size(d)
    assert norm_bwd(d, nbytes=n - 1) == jmix.JM_ERR_WORKSPACE
    assert norm_bwd(d, workspace=None) == jmix.JM_ERR_WORKSPACE
    assert norm_bwd(d, workspace=W + 16) == jmix.JM_ERR_WORKSPACE
    assert norm_bwd(d, workspace=F + G) == bad and "workspace overlaps x" in jmix.jm_last_error()


def test_norm_no_rows_needs_no_buffers():
    assert norm_fwd(jmix.norm_dims(0, 32), x=None, y=None) == jmix.JM_OK
    assert jmix.jm_last_launch_count() == 0


def test_binding_checks_tensors():
    """What an address cannot say is checked in the binding."""
    import torch
    t = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(jmix.JmixError, match="x is torch.bfloat16") as e:
        jmix.jm_norm_fwd(jmix.norm_dims(4, 32, io=jmix.JM_F32), t, F, F, stream=0)
    assert e.value.status == jmix.JM_ERR_INVALID_ARG
    with pytest.raises(jmix.JmixError, match="residual is not contiguous"):
        jmix.jm_norm_fwd(jmix.norm_dims(4, 32), F, F, F, residual=t.t(), stream=0)
    with pytest.raises(jmix.JmixError, match="stats is torch.bfloat16"):
        jmix.jm_norm_fwd(jmix.norm_dims(4, 32), F, F, F, stats=t, stream=0)
    with pytest.raises(jmix.JmixError, match="CUDA device"):
        jmix.jm_norm_fwd(jmix.norm_dims(4, 32), t, F, F, stream=0)


def rows_verdict(x, rows, cols, x_stride=None):
    """What the binding says of x before it asks for its device (these tensors have no GPU's
    address, so that an accepted one ends there)."""
    d = jmix.norm_dims(rows, cols, x_stride=x_stride)
    said = []
    for call in (lambda: jmix.jm_norm_fwd(d, x, F, F, stream=0),
                 lambda: jmix.jm_norm_bwd(d, F, x, F, F, F, W, 1 << 30, stream=0)):
        with pytest.raises(jmix.JmixError) as e:
            call()
        assert e.value.status == jmix.JM_ERR_INVALID_ARG
        said.append("ok" if "CUDA device" in str(e.value) else str(e.value))
    assert said[0] == said[1]
    return said[0]


def test_binding_checks_the_row_pitch():
    import torch
    x = torch.zeros(4, 6, 32, dtype=torch.bfloat16)
    wide = torch.zeros(24, 64, dtype=torch.bfloat16)
    # one pitch, and the dims say it
    assert rows_verdict(x, 24, 32) == "ok"
    assert rows_verdict(x, 4, 192) == "ok"                       # packed, grouped otherwise
    assert rows_verdict(x.view(-1), 24, 32) == "ok"
    assert rows_verdict(wide[:, :32], 24, 32, 64) == "ok"
    assert rows_verdict(wide, 24, 32, 64) == "ok"                # the rows' first 32 values
    assert rows_verdict(wide.view(4, 6, 64)[..., :32], 24, 32, 64) == "ok"
    assert rows_verdict(x[:, 0], 4, 32, 192) == "ok"
    assert rows_verdict(x[:, :1], 4, 32, 192) == "ok"
    assert rows_verdict(wide[:1, :32], 1, 32, 40) == "ok"        # one row has no pitch
    assert rows_verdict(wide[:, :1], 24, 1, 64) == "ok"
    # packed tensors and other strides in the dims
    assert "row stride 32, the dims say 64" in rows_verdict(x.view(24, 32), 24, 32, 64)
    assert "row stride 32, the dims say 40" in rows_verdict(x, 24, 32, 40)
    assert "row stride 64, the dims say 32" in rows_verdict(wide[:, :32], 24, 32)
    # more than two dimensions: a slice of the columns, every other one, transposed
    assert "row stride 64, the dims say 32" in rows_verdict(wide.view(4, 6, 64)[..., :32], 24, 32)
    assert "one stride" in rows_verdict(x[::2], 12, 32)
    assert "one stride" in rows_verdict(x.transpose(0, 1), 24, 32)
    assert "one stride" in rows_verdict(x[:, :3], 12, 32)
    # a gap between the values of a row, rows shorter than the dims say
    assert "not contiguous" in rows_verdict(wide[:, ::2], 24, 32, 64)
    assert "not contiguous" in rows_verdict(x.transpose(1, 2), 128, 6)
    assert "not contiguous" in rows_verdict(wide.view(-1)[::2], 24, 32)
    assert "rows of 16" in rows_verdict(wide[:, :16], 24, 32, 64)
    assert "row stride 0" in rows_verdict(x[0, :1].expand(24, 32), 24, 32)
    assert "row stride 0" in rows_verdict(x[0, 0].expand(4, 6, 32), 24, 32)


def test_binding_checks_the_number_of_values_of_x():
    import torch
    x = torch.zeros(24, 32, dtype=torch.bfloat16)
    assert "768 values, the call needs 800" in rows_verdict(x, 25, 32)
    assert rows_verdict(x, 23, 32) == "ok"                       # a buffer for more rows
    assert "768 values, the call needs 1504" in rows_verdict(x.view(-1), 24, 32, 64)
    assert rows_verdict(x.view(-1), 12, 32, 64) == "ok"
    assert "24 rows, the dims say 25" in rows_verdict(torch.zeros(24, 64, dtype=torch.bfloat16)[:, :32],
                                                      25, 32, 64)
    assert "24 rows, the dims say 25" in rows_verdict(x, 25, 16, 32)


NORM, LINEAR, MOE = (jmix.norm_dims(6, 40, kind=jmix.JM_NORM_LAYER), jmix.linear_dims(6, 40, 56, 1),
                     jmix.moe_dims(6, 40, 56, 5, 2))
SIZED = [  # call, dims, {argument: values the call reads or writes}
    ("jm_norm_fwd", NORM, dict(weight=40, y=240, bias=40, residual=240, sum_out=240, stats=12)),
    ("jm_norm_bwd", NORM, dict(g_y=240, weight=40, stats=12, g_x=240, g_sum=240, g_weight=40,
                               g_bias=40, workspace=1024)),
    ("jm_linear_fwd", LINEAR, dict(x=240, w=2240, out=336, bias=56, residual=336, pre=336,
                                   workspace=1024)),
    ("jm_linear_bwd", LINEAR, dict(g_out=336, x=240, w=2240, pre=336, g_x=240, g_w=2240, g_bias=56,
                                   workspace=1024)),
    ("jm_moe_fwd", MOE, dict(x=240, router_w=200, w_gate=11200, w_up=11200, w_down=11200, out=240,
                             residual=240, topk_idx=12, topk_w=12, workspace=1024)),
]


@pytest.mark.parametrize("call,d,needs", SIZED)
def test_binding_checks_the_number_of_values(call, d, needs):
    """A tensor with fewer values than the dims say is refused, one with more is not."""
    import torch
    types = dict(stats=torch.float32, topk_w=torch.float32, topk_idx=torch.int32,
                 workspace=torch.uint8)
    base = dict(x=F) if "x" not in needs else {}
    base.update({k: F for k in needs})
    if "workspace" in needs:
        base["ws_bytes"] = 1024
    for k, n in needs.items():
        for have, msg in ((n - 1, f"{k.replace('sum_out', 'sum')} has {n - 1} "), (n, "CUDA device"),
                          (n + 8, "CUDA device")):
            t = torch.zeros(have, dtype=types.get(k, torch.bfloat16))
            with pytest.raises(jmix.JmixError, match=msg) as e:
                getattr(jmix, call)(d, **{**base, k: t}, stream=0)
            assert e.value.status == jmix.JM_ERR_INVALID_ARG


def linear_fwd(d, nbytes=None, **over):
    a = dict(x=F, w=F + G, out=F + 2 * G, workspace=W,
             ws_bytes=jmix.jm_linear_fwd_workspace_size(d) if nbytes is None else nbytes)
    a.update(over)
    return jmix.jm_linear_fwd(d, **a, stream=0, check=False)


def linear_bwd(d, nbytes=None, **over):
    a = dict(g_out=F, x=F + G, w=F + 2 * G, g_x=F + 3 * G, g_w=F + 4 * G, g_bias=F + 5 * G,
             workspace=W,
             ws_bytes=jmix.jm_linear_bwd_workspace_size(d) if nbytes is None else nbytes)
    a.update(over)
    return jmix.jm_linear_bwd(d, **a, stream=0, check=False)


@pytest.mark.parametrize("over,code,msg", [
    (dict(rows=-1), jmix.JM_ERR_INVALID_ARG, "positive"),
    (dict(in_features=0), jmix.JM_ERR_INVALID_ARG, "positive"),
    (dict(in_features=60), jmix.JM_ERR_INVALID_ARG, "multiples of 8"),
    (dict(out_features=12), jmix.JM_ERR_INVALID_ARG, "multiples of 8"),
    (dict(io=jmix.JM_F32), jmix.JM_ERR_UNSUPPORTED, "bf16"),
    (dict(io=9), jmix.JM_ERR_INVALID_ARG, "io dtype"),
    (dict(act=4), jmix.JM_ERR_INVALID_ARG, "act"),
    (dict(rows=1 << 31), jmix.JM_ERR_INVALID_ARG, "large"),
])
def test_linear_rejects_bad_dims(over, code, msg):
    kw = dict(rows=4, in_features=64, out_features=128)
    kw.update(over)
    d = jmix.linear_dims(**kw)
    assert linear_fwd(d, 1 << 30) == code and msg in jmix.jm_last_error()
    assert linear_bwd(d, 1 << 30) == code and msg in jmix.jm_last_error()
    assert jmix.jm_linear_fwd_workspace_size(d) == 0
    assert jmix.jm_linear_bwd_workspace_size(d) == 0


def test_linear_rejects_bad_pointers():
    bad = jmix.JM_ERR_INVALID_ARG
    d = jmix.linear_dims(4, 64, 128, act=jmix.JM_ACT_SILU)
    for k in ("x", "w", "out"):
        assert linear_fwd(d, **{k: None}) == bad and "NULL" in jmix.jm_last_error(), k
        assert linear_fwd(d, **{k: F + 4}) == bad and "aligned" in jmix.jm_last_error(), k
    assert linear_fwd(d, out=F) == bad and "out overlaps x" in jmix.jm_last_error()
    assert linear_fwd(d, residual=F + 2 * G + 64) == bad
    assert "out overlaps residual" in jmix.jm_last_error()
    assert linear_fwd(d, pre=F + 2 * G) == bad and "pre overlaps out" in jmix.jm_last_error()
    r = F + 2 * G    # residual == out, but pre over it is not
    assert linear_fwd(d, residual=r, pre=r) == bad
    assert linear_fwd(d, workspace=F + G) == bad and "workspace overlaps w" in jmix.jm_last_error()
    n = jmix.jm_linear_fwd_workspace_size(d)
    assert linear_fwd(d, nbytes=n - 1) == jmix.JM_ERR_WORKSPACE
    assert linear_fwd(d, workspace=None) == jmix.JM_ERR_WORKSPACE
    assert linear_fwd(d, workspace=W + 64) == jmix.JM_ERR_WORKSPACE
    p = F + 6 * G
    assert linear_bwd(d) == bad and "pre is NULL" in jmix.jm_last_error()
    assert linear_bwd(jmix.linear_dims(4, 64, 128), pre=p) == bad
    for k in ("g_out", "x", "w"):
        assert linear_bwd(d, pre=p, **{k: None}) == bad and "NULL" in jmix.jm_last_error(), k
    assert linear_bwd(d, pre=p, g_x=F + G) == bad and "g_x overlaps x" in jmix.jm_last_error()
    assert linear_bwd(d, pre=p, g_w=F + 3 * G) == bad
    assert linear_bwd(d, pre=p, nbytes=255) == jmix.JM_ERR_WORKSPACE


def moe_fwd(d, nbytes=None, **over):
    a = dict(x=F, router_w=F + G, w_gate=F + 2 * G, w_up=F + 3 * G, w_down=F + 4 * G,
             out=F + 5 * G, workspace=W,
             ws_bytes=jmix.jm_moe_fwd_workspace_size(d) if nbytes is None else nbytes)
    a.update(over)
    return jmix.jm_moe_fwd(d, **a, stream=0, check=False)


@pytest.mark.parametrize("over,code,msg", [
    (dict(tokens=-1), jmix.JM_ERR_INVALID_ARG, "positive"),
    (dict(d_model=0), jmix.JM_ERR_INVALID_ARG, "positive"),
    (dict(top_k=0), jmix.JM_ERR_INVALID_ARG, "positive"),
    (dict(d_model=60), jmix.JM_ERR_INVALID_ARG, "multiples of 8"),
    (dict(d_ff=12), jmix.JM_ERR_INVALID_ARG, "multiples of 8"),
    (dict(top_k=5), jmix.JM_ERR_INVALID_ARG, "n_experts"),
    (dict(tokens=257), jmix.JM_ERR_UNSUPPORTED, "256 tokens"),
    (dict(n_experts=257), jmix.JM_ERR_UNSUPPORTED, "experts"),
    (dict(n_experts=16, top_k=9), jmix.JM_ERR_UNSUPPORTED, "top_k"),
    (dict(io=jmix.JM_F32), jmix.JM_ERR_UNSUPPORTED, "bf16"),
    (dict(io=9), jmix.JM_ERR_INVALID_ARG, "io dtype"),
    (dict(router=2), jmix.JM_ERR_INVALID_ARG, "router"),
    (dict(d_model=1 << 24, d_ff=1 << 24), jmix.JM_ERR_INVALID_ARG, "large"),
])
def test_moe_rejects_bad_dims(over, code, msg):
    kw = dict(tokens=4, d_model=64, d_ff=128, n_experts=4, top_k=2)
    kw.update(over)
    d = jmix.moe_dims(**kw)
    assert moe_fwd(d, 1 << 30) == code and msg in jmix.jm_last_error()
    assert jmix.jm_moe_fwd_workspace_size(d) == 0


def test_moe_rejects_bad_pointers():
    bad = jmix.JM_ERR_INVALID_ARG
    d = jmix.moe_dims(4, 64, 128, 4, 2)
    for k in ("x", "router_w", "w_gate", "w_up", "w_down", "out"):
        assert moe_fwd(d, **{k: None}) == bad and "NULL" in jmix.jm_last_error(), k
        assert moe_fwd(d, **{k: F + 8}) == bad and "aligned" in jmix.jm_last_error(), k
    assert moe_fwd(d, out=F) == bad and "out overlaps x" in jmix.jm_last_error()
    assert moe_fwd(d, residual=F + 5 * G + 64) == bad
    assert "out overlaps residual" in jmix.jm_last_error()
    assert moe_fwd(d, topk_idx=F + 5 * G) == bad and "topk_idx overlaps out" in jmix.jm_last_error()
    assert moe_fwd(d, topk_w=F + 2 * G) == bad and "topk_w overlaps w_gate" in jmix.jm_last_error()
    assert moe_fwd(d, workspace=F + 4 * G) == bad
    # the residual in out's place, but a list over it is not
    r = F + 5 * G
    assert moe_fwd(d, residual=r, topk_idx=r) == bad
    n = jmix.jm_moe_fwd_workspace_size(d)
    assert moe_fwd(d, nbytes=n - 1) == jmix.JM_ERR_WORKSPACE
    assert moe_fwd(d, workspace=None) == jmix.JM_ERR_WORKSPACE
    assert moe_fwd(d, workspace=W + 64) == jmix.JM_ERR_WORKSPACE


def test_moe_workspace_size_of_every_token_count():
    for t in range(257):
        for e, k in ((1, 1), (16, 2), (256, 8)):
            n = jmix.jm_moe_fwd_workspace_size(jmix.moe_dims(t, 64, 128, e, k))
            assert n >= 256 and n % 256 == 0
