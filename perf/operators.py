"""The operators of the decoder block around the mixer, as measured workloads.

Five operators: ``norm_fwd`` (residual add + LayerNorm / RMSNorm), ``norm_bwd``
(its backward with the weight and bias gradients), ``linear_fwd`` (matrix
product with bias, activation and residual), ``linear_bwd`` (its backward) and
``moe`` (a whole mixture-of-experts layer for few tokens).  ``run`` computes
them in a plain form of elementary torch operations, or, with ``own`` set,
through libjmix.
"""
import math

import torch

own = False

# Sizes: d_model 4096, d_inner 8192 (in_proj 4096 -> 16384, out_proj 8192 ->
# 4096), d_ff 14336, 16 experts of which 2 are used, decode batches of up to 256
# sequences, prefills of 8 x 4096 tokens.  The others are generic odd ones.


def listed():
    return [
        # the pre-norm of a decode step of 256 sequences, residual added on the way
        dict(name="norm_fwd_decode", op="norm_fwd", rows=256, cols=4096, io="bf16", kind="rms",
             residual=True, bias=False),
        # the pre-norm of a prefill of 8 x 4096 tokens
        dict(name="norm_fwd_prefill", op="norm_fwd", rows=32768, cols=4096, io="bf16", kind="rms",
             residual=True, bias=False),
        # one training micro-batch; the residual stream's own gradient joins g_x
        dict(name="norm_bwd_train", op="norm_bwd", rows=8192, cols=4096, io="bf16", kind="layer",
             residual=True, bias=True),
        # float32 training of a small model with an odd width (no vector loads)
        dict(name="norm_bwd_odd_f32", op="norm_bwd", rows=3001, cols=1021, io="f32", kind="layer",
             residual=False, bias=True),
        # single-token decode through in_proj: the weight's bytes decide
        dict(name="linear_fwd_token", op="linear_fwd", rows=1, k=4096, n=16384, act="none",
             bias=False, residual=False),
        # out_proj of a decode step of 256 sequences with the residual stream added
        dict(name="linear_fwd_decode", op="linear_fwd", rows=256, k=8192, n=4096, act="none",
             bias=False, residual=True),
        # first product of a feed-forward layer in a prefill of 2 x 4096 tokens
        dict(name="linear_fwd_prefill", op="linear_fwd", rows=8192, k=4096, n=14336, act="gelu",
             bias=True, residual=False),
        # the same product's backward in training
        dict(name="linear_bwd_train", op="linear_bwd", rows=8192, k=4096, n=14336, act="silu",
             bias=True),
        # a small model's ragged last micro-batch
        dict(name="linear_bwd_odd", op="linear_bwd", rows=1003, k=1032, n=2056, act="relu",
             bias=True),
        # one sequence decoding: two experts' weights stream through
        dict(name="moe_token", op="moe", tokens=1, d=4096, f=14336, experts=16, top_k=2,
             router="all", residual=True),
        # a decode batch of 256 sequences: every expert's weights are read
        dict(name="moe_decode", op="moe", tokens=256, d=4096, f=14336, experts=16, top_k=2,
             router="topk", residual=True),
        # a small model's decode batch: launch and hand-over latency decide
        dict(name="moe_small", op="moe", tokens=13, d=512, f=1416, experts=8, top_k=2,
             router="all", residual=False),
    ]


def _log_int(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // mult * mult))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "linear_fwd", "linear_bwd", "moe", "moe"])
    if op in ("norm_fwd", "norm_bwd"):
        cols = _log_int(rng, 16, 8192)
        if rng.random() < 0.5:
            cols = max(8, cols // 8 * 8)
        rows = _log_int(rng, 1, min(32768, 32768 * 4096 // cols))
        kind = rng.choice(["rms", "layer"])
        return dict(op=op, rows=rows if op == "norm_fwd" else min(rows, 16384), cols=cols,
                    io=rng.choice(["bf16", "bf16", "f32"]) if cols <= 2048 else "bf16", kind=kind,
                    residual=rng.random() < 0.5, bias=kind == "layer" and rng.random() < 0.7)
    if op in ("linear_fwd", "linear_bwd"):
        k, n = _log_int(rng, 64, 14336, 8), _log_int(rng, 64, 14336, 8)
        rows = _log_int(rng, 1, 8192)
        rows = max(1, min(rows, 8192 * 4096 * 14336 // (k * n)))
        c = dict(op=op, rows=rows, k=k, n=n, act=rng.choice(["none", "relu", "gelu", "silu"]),
                 bias=rng.random() < 0.5)
        if op == "linear_fwd":
            c["residual"] = rng.random() < 0.5
        return c
    experts = rng.choice([1, 2, 4, 7, 8, 16, 16, 24])
    d = _log_int(rng, 64, 4096, 8)
    f = _log_int(rng, 64, 14336, 8)
    if experts > 16:
        f = min(f, 8192)
    return dict(op=op, tokens=_log_int(rng, 1, 256), d=d, f=f, experts=experts,
                top_k=rng.randint(1, min(2, experts)), router=rng.choice(["all", "topk"]),
                residual=rng.random() < 0.5)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(mean, std, generator=g)


def _act(v, act):
    if act == "relu":
        return torch.clamp(v, min=0)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _act_grad(v, act):
    if act == "relu":
        return (v > 0).to(v.dtype)
    if act == "gelu":
        return (0.5 * (1 + torch.erf(v * math.sqrt(0.5)))
                + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi)))
    if act == "silu":
        s = 1 / (1 + torch.exp(-v))
        return s * (1 + v * (1 - s))
    return torch.ones_like(v)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] in ("norm_fwd", "norm_bwd"):
        dt = torch.bfloat16 if c["io"] == "bf16" else torch.float32
        r, n = c["rows"], c["cols"]
        # a residual stream: a scale of a few and an offset of its own per column
        s["x"] = (_randn(g, r, n, std=2.0, dtype=torch.float32)
                  + _randn(g, 1, n, std=0.5, dtype=torch.float32)).to(dt)
        s["w"] = _randn(g, n, std=0.1, mean=1.0, dtype=dt)
        s["b"] = _randn(g, n, std=0.1, dtype=dt) if c["bias"] else None
        if c["op"] == "norm_fwd":
            s["r"] = _randn(g, r, n, dtype=dt) if c["residual"] else None
        else:
            s["gy"] = _randn(g, r, n, dtype=dt)
            s["gs"] = _randn(g, r, n, dtype=dt) if c["residual"] else None
            x = s["x"].float()
            m = x.mean(1) if c["kind"] == "layer" else torch.zeros(r, device="cuda")
            v = ((x - m[:, None]) ** 2).mean(1)
            s["stats"] = torch.stack([m, (v + 1e-6) ** -0.5], 1).contiguous()
    elif c["op"] in ("linear_fwd", "linear_bwd"):
        m, k, n = c["rows"], c["k"], c["n"]
        s["x"] = _randn(g, m, k)
        s["w"] = _randn(g, n, k, std=k ** -0.5)
        s["b"] = _randn(g, n, std=0.5) if c["bias"] else None
        if c["op"] == "linear_fwd":
            s["r"] = _randn(g, m, n) if c["residual"] else None
        else:
            s["g"] = _randn(g, m, n)
            if c["act"] != "none":
                p = s["x"] @ s["w"].t()
                s["pre"] = p if s["b"] is None else p + s["b"]
            else:
                s["pre"] = None
    else:
        t, d, f, e = c["tokens"], c["d"], c["f"], c["experts"]
        s["x"] = _randn(g, t, d)
        s["wr"] = _randn(g, e, d, std=d ** -0.5)
        s["wg"] = _randn(g, e, f, d, std=d ** -0.5)
        s["wu"] = _randn(g, e, f, d, std=d ** -0.5)
        s["wd"] = _randn(g, e, d, f, std=f ** -0.5)
        s["r"] = _randn(g, t, d) if c["residual"] else None
    return s


# ------------------------------------------------------------ plain forms


def _plain_norm_fwd(s, c):
    dt = s["x"].dtype
    x = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(dt)
    v = x.float()
    m = v.mean(1, keepdim=True) if c["kind"] == "layer" else torch.zeros_like(v[:, :1])
    rstd = 1 / torch.sqrt(((v - m) ** 2).mean(1, keepdim=True) + 1e-6)
    y = (v - m) * rstd * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    out = {"y": y.to(dt), "stats": torch.cat([m, rstd], 1)}
    if s["r"] is not None:
        out["sum"] = x
    return out


def _plain_norm_bwd(s, c):
    dt = s["x"].dtype
    gy = s["gy"].float()
    rstd = s["stats"][:, 1:]
    xh = (s["x"].float() - s["stats"][:, :1]) * rstd
    g = gy * s["w"].float()
    t = g - xh * (g * xh).mean(1, keepdim=True)
    if c["kind"] == "layer":
        t = t - g.mean(1, keepdim=True)
    gx = t * rstd
    if s["gs"] is not None:
        gx = gx + s["gs"].float()
    out = {"gx": gx.to(dt), "gw": (gy * xh).sum(0).to(dt)}
    if s["b"] is not None:
        out["gb"] = gy.sum(0).to(dt)
    return out


def _plain_linear_fwd(s, c):
    v = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        v = v + s["b"].float()
    v = _act(v, c["act"])
    if s["r"] is not None:
        v = v + s["r"].float()
    return {"out": v.to(torch.bfloat16)}


def _plain_linear_bwd(s, c):
    gp = s["g"].float()
    if s["pre"] is not None:
        gp = gp * _act_grad(s["pre"].float(), c["act"])
    out = {"gx": (gp @ s["w"].float()).to(torch.bfloat16),
           "gw": (gp.t() @ s["x"].float()).to(torch.bfloat16)}
    if s["b"] is not None:
        out["gb"] = gp.sum(0).to(torch.bfloat16)
    return out


def _plain_moe(s, c):
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    # the choice of experts is a comparison of close values: logits in 64 bits
    logits = s["x"].double() @ s["wr"].double().t()
    val, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    w = torch.exp(val - val[:, :1])
    norm = w if c["router"] == "topk" else torch.exp(logits - val[:, :1])
    w = (w / norm.sum(1, keepdim=True)).float()
    x = s["x"].float()
    if t * k <= e:  # few rows: the chosen experts' weights are gathered
        ids = idx.reshape(-1)
        xr = x.repeat_interleave(k, 0)[:, :, None]
        h = _act((s["wg"][ids].float() @ xr)[..., 0], "silu") * (s["wu"][ids].float() @ xr)[..., 0]
        y = (s["wd"][ids].float() @ h[:, :, None])[..., 0]
        out = (y.view(t, k, -1) * w[:, :, None]).sum(1)
    else:  # every expert on every token, weighted by zero where it was not chosen
        cw = torch.zeros(t, e, device=x.device).scatter_(1, idx, w)
        xe = x[None].expand(e, t, c["d"])
        h = _act(xe @ s["wg"].float().transpose(1, 2), "silu")
        h = h * (xe @ s["wu"].float().transpose(1, 2))
        y = h @ s["wd"].float().transpose(1, 2)
        out = (y * cw.t()[:, :, None]).sum(0)
    if s["r"] is not None:
        out = out + s["r"].float()
    return {"out": out.to(torch.bfloat16), "idx": idx.to(torch.int32), "w": w}


# ------------------------------------------------------------ libjmix


def _own_state(s, c):
    """What a program keeps between calls: dims, output buffers and a workspace."""
    from mamba_selective_scan_jamba_b200 import devio, jmix
    o = {"jm": jmix}
    like = torch.empty_like
    if c["op"] in ("norm_fwd", "norm_bwd"):
        o["d"] = jmix.norm_dims(c["rows"], c["cols"],
                                jmix.JM_BF16 if c["io"] == "bf16" else jmix.JM_F32,
                                kind=jmix.JM_NORM_LAYER if c["kind"] == "layer"
                                else jmix.JM_NORM_RMS, eps=1e-6)
        if c["op"] == "norm_fwd":
            o["out"] = {"y": like(s["x"]),
                        "stats": torch.empty(c["rows"], 2, device="cuda", dtype=torch.float32)}
            if s["r"] is not None:
                o["out"]["sum"] = like(s["x"])
        else:
            o["out"] = {"gx": like(s["x"]), "gw": like(s["w"])}
            if s["b"] is not None:
                o["out"]["gb"] = like(s["w"])
            o["n"] = jmix.jm_norm_bwd_workspace_size(o["d"])
    elif c["op"] in ("linear_fwd", "linear_bwd"):
        act = {"none": jmix.JM_ACT_NONE, "relu": jmix.JM_ACT_RELU, "gelu": jmix.JM_ACT_GELU,
               "silu": jmix.JM_ACT_SILU}[c["act"]]
        o["d"] = jmix.linear_dims(c["rows"], c["k"], c["n"], act=act)
        if c["op"] == "linear_fwd":
            o["out"] = {"out": torch.empty(c["rows"], c["n"], device="cuda", dtype=torch.bfloat16)}
            o["n"] = jmix.jm_linear_fwd_workspace_size(o["d"])
        else:
            o["out"] = {"gx": like(s["x"]), "gw": like(s["w"])}
            if s["b"] is not None:
                o["out"]["gb"] = like(s["b"])
            o["n"] = jmix.jm_linear_bwd_workspace_size(o["d"])
    else:
        o["d"] = jmix.moe_dims(c["tokens"], c["d"], c["f"], c["experts"], c["top_k"],
                               router=jmix.JM_ROUTE_SOFTMAX_TOPK if c["router"] == "topk"
                               else jmix.JM_ROUTE_SOFTMAX_ALL)
        o["out"] = {"out": like(s["x"]),
                    "idx": torch.empty(c["tokens"], c["top_k"], device="cuda", dtype=torch.int32),
                    "w": torch.empty(c["tokens"], c["top_k"], device="cuda", dtype=torch.float32)}
        o["n"] = jmix.jm_moe_fwd_workspace_size(o["d"])
    if "n" in o:
        o["ws"] = devio.workspace(o["n"])
    return o


def _own_run(s, c):
    if "own" not in s:
        s["own"] = _own_state(s, c)
    o = s["own"]
    jm, out = o["jm"], o["out"]
    if c["op"] == "norm_fwd":
        jm.jm_norm_fwd(o["d"], s["x"], s["w"], out["y"], bias=s["b"], residual=s["r"],
                       sum_out=out.get("sum"), stats=out["stats"])
    elif c["op"] == "norm_bwd":
        jm.jm_norm_bwd(o["d"], s["gy"], s["x"], s["w"], s["stats"], out["gx"], o["ws"], o["n"],
                       g_sum=s["gs"], g_weight=out["gw"], g_bias=out.get("gb"))
    elif c["op"] == "linear_fwd":
        jm.jm_linear_fwd(o["d"], s["x"], s["w"], out["out"], o["ws"], o["n"], bias=s["b"],
                         residual=s["r"])
    elif c["op"] == "linear_bwd":
        jm.jm_linear_bwd(o["d"], s["g"], s["x"], s["w"], o["ws"], o["n"], pre=s["pre"],
                         g_x=out["gx"], g_w=out["gw"], g_bias=out.get("gb"))
    else:
        jm.jm_moe_fwd(o["d"], s["x"], s["wr"], s["wg"], s["wu"], s["wd"], out["out"], o["ws"],
                      o["n"], residual=s["r"], topk_idx=out["idx"], topk_w=out["w"])
    return out


def run(state):
    c = state["case"]
    if own:
        return _own_run(state, c)
    if c["op"] == "norm_fwd":
        return _plain_norm_fwd(state, c)
    if c["op"] == "norm_bwd":
        return _plain_norm_bwd(state, c)
    if c["op"] == "linear_fwd":
        return _plain_linear_fwd(state, c)
    if c["op"] == "linear_bwd":
        return _plain_linear_bwd(state, c)
    return _plain_moe(state, c)


def work(case):
    c = case
    if c["op"] in ("norm_fwd", "norm_bwd"):
        es = 2 if c["io"] == "bf16" else 4
        rc = c["rows"] * c["cols"]
        vec = c["cols"] * es * (2 if c["bias"] else 1)
        if c["op"] == "norm_fwd":
            return {"bytes": rc * es * (4 if c["residual"] else 2) + c["rows"] * 8 + vec,
                    "flops": 8 * rc}
        return {"bytes": rc * es * (4 if c["residual"] else 3) + c["rows"] * 8 + c["cols"] * es
                + vec, "flops": 14 * rc}
    if c["op"] in ("linear_fwd", "linear_bwd"):
        m, k, n = c["rows"], c["k"], c["n"]
        if c["op"] == "linear_fwd":
            return {"bytes": 2 * (m * k + n * k + m * n * (2 if c["residual"] else 1)
                                  + (n if c["bias"] else 0)), "flops": 2 * m * n * k}
        return {"bytes": 2 * (2 * m * k + 2 * n * k + m * n * (1 if c["act"] == "none" else 2)
                              + (n if c["bias"] else 0)), "flops": 4 * m * n * k}
    t, d, f, e, k = c["tokens"], c["d"], c["f"], c["experts"], c["top_k"]
    used = e * (1 - (1 - k / e) ** t)  # experts in use, expected for an even router
    return {"bytes": 2 * (used * 3 * d * f + e * d + t * d * (3 if c["residual"] else 2))
            + t * k * 8, "flops": 2 * t * (e * d + k * 3 * d * f)}


def exact(case, seed):
    """The operators from their definitions in 64 bits, on the same inputs."""
    c, s = case, prepare(case, seed)
    D = torch.float64
    if c["op"] == "norm_fwd":
        x = s["x"].to(D)
        if s["r"] is not None:  # the sum is stored in the io type, and that value is normalised
            x = (x + s["r"].to(D)).float().to(s["x"].dtype).to(D)
        mean = x.sum(1) / c["cols"] if c["kind"] == "layer" else x.new_zeros(c["rows"])
        ctr = x - mean[:, None]
        rstd = ((ctr * ctr).sum(1) / c["cols"] + 1e-6).rsqrt()
        y = torch.einsum("rc,r,c->rc", ctr, rstd, s["w"].to(D))
        out = {"y": y if s["b"] is None else y + s["b"].to(D),
               "stats": torch.stack((mean, rstd), dim=1)}
        if s["r"] is not None:
            out["sum"] = x
        return out
    if c["op"] == "norm_bwd":
        st = s["stats"].to(D)
        gy, w = s["gy"].to(D), s["w"].to(D)
        ctr = s["x"].to(D) - st[:, 0][:, None]
        n = c["cols"]
        dot = torch.einsum("rc,rc,c->r", gy, ctr, w) * st[:, 1]      # sum of g xhat
        tot = gy @ w if c["kind"] == "layer" else torch.zeros_like(dot)
        gx = (gy * w - (tot / n)[:, None]
              - ctr * (dot * st[:, 1] / n)[:, None]) * st[:, 1][:, None]
        if s["gs"] is not None:
            gx += s["gs"].to(D)
        out = {"gx": gx, "gw": torch.einsum("rc,rc,r->c", gy, ctr, st[:, 1])}
        if s["b"] is not None:
            out["gb"] = torch.ones(c["rows"], device="cuda", dtype=D) @ gy
        return out
    if c["op"] == "linear_fwd":
        v = torch.einsum("mk,nk->mn", s["x"].to(D), s["w"].to(D))
        if s["b"] is not None:
            v += s["b"].to(D)
        if c["act"] == "relu":
            v = torch.where(v > 0, v, torch.zeros_like(v))
        elif c["act"] == "gelu":
            v = v * torch.special.ndtr(v)
        elif c["act"] == "silu":
            v = v * torch.sigmoid(v)
        return {"out": v if s["r"] is None else v + s["r"].to(D)}
    if c["op"] == "linear_bwd":
        g = s["g"].to(D)
        if s["pre"] is not None:
            p = s["pre"].to(D)
            if c["act"] == "relu":
                g = torch.where(p > 0, g, torch.zeros_like(g))
            elif c["act"] == "gelu":
                g = g * (torch.special.ndtr(p)
                         + p * torch.exp(-p * p / 2) / math.sqrt(2 * math.pi))
            else:
                q = torch.sigmoid(p)
                g = g * (q + p * q * (1 - q))
        out = {"gx": torch.einsum("mn,nk->mk", g, s["w"].to(D)),
               "gw": torch.einsum("mn,mk->nk", g, s["x"].to(D))}
        if s["b"] is not None:
            out["gb"] = torch.einsum("mn->n", g)
        return out
    x = s["x"].to(D)
    logits = torch.einsum("td,ed->te", x, s["wr"].to(D))
    idx = torch.argsort(-logits, dim=1, stable=True)[:, :c["top_k"]]
    picked = torch.gather(logits, 1, idx)
    w = (torch.softmax(picked, 1) if c["router"] == "topk"
         else torch.gather(torch.softmax(logits, 1), 1, idx))
    out = torch.zeros_like(x) if s["r"] is None else s["r"].to(D)
    for e in range(c["experts"]):
        rows, col = torch.nonzero(idx == e, as_tuple=True)
        if rows.numel():
            a = x[rows] @ s["wg"][e].to(D).t()
            a = a * torch.sigmoid(a) * (x[rows] @ s["wu"][e].to(D).t())
            out.index_add_(0, rows, (a @ s["wd"][e].to(D).t()) * w[rows, col][:, None])
    return {"out": out, "idx": idx.to(torch.int32), "w": w}
