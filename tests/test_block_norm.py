"""The block norm (post norm, gate, residual scale, residual add, pre norm) against the
formulas in 64 bits, its backward against automatic differentiation and differences, and
its refusals.

Tolerances.  u = 2^-24 is half a step of fp32, `half(t)` half a step of the output's type.
A sum over a row takes at most 8 (a thread's values, or 16) + 6 (lanes) + 16 (waves)
additions, and a few more operations follow: 40 u times the magnitudes that enter covers
each of them (`lin` and `_norm_mag` carry those magnitudes through a norm).  A sum over rows
adds at most min(rows, 1024) + 64 values one after the other in fp32."""
import ctypes

import pytest
import torch

import conv2d_batchnorm_relu_amd as cbr

U = 2.0 ** -24
K = 40 * U
DT = {"bf16": (torch.bfloat16, cbr.CBR_BF16), "f16": (torch.float16, cbr.CBR_F16), "f32": (torch.float32, cbr.CBR_F32)}
KIND = {"none": cbr.CBR_NORM_NONE, "rms": cbr.CBR_NORM_RMS, "layer": cbr.CBR_NORM_LAYER}
ALPHA, EPS_POST, EPS_PRE = 0.75, 1e-5, 1e-6


def half(dtype, v):
    """Half a step of dtype at the values v (fp32: nothing is rounded a second time)."""
    if dtype == torch.float32:
        return U * v.abs()
    return torch.finfo(dtype).eps / 2 * v.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)


# ------------------------------------------------------------------- 64-bit formulas
def norm64(v, kind, eps, w, b):
    """(mean, 1/std, normed values, output) of each row."""
    if kind == "none":
        return None, None, v, v
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    inv = ((v - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    vh = (v - mean) * inv
    o = vh if w is None else vh * w
    return mean, inv, vh, o if b is None else o + b


def forward64(t):
    """t: dict of 64-bit tensors (None where not given)."""
    o = {}
    f = t["f"]
    if f is not None:
        o["pm"], o["pi"], o["nhat"], n = norm64(f, t["post"], EPS_POST, t["post_w"], t["post_b"])
        c = torch.full((1, 1), ALPHA, dtype=torch.float64, device=f.device)
        if t["res_scale"] is not None:
            c = c * t["res_scale"]
        if t["gate"] is not None:
            c = c * t["gate"].repeat_interleave(t["rpg"], 0)
        o["n"], o["c"] = n, c
        o["y"] = t["x"] + c * n
    else:
        o["y"] = t["x"]
    if t["pre"] != "none":
        o["qm"], o["qi"], o["yhat"], o["h"] = norm64(o["y"], t["pre"], EPS_PRE, t["pre_w"], t["pre_b"])
    return o


def _norm_mag(v, vh, mean, inv):
    """Error of the normed values from fp32 sums, over K: the values and the mean they come from."""
    absmean = v.abs().mean(1, keepdim=True)
    return vh.abs() * (1 + inv * absmean) + inv * (absmean + v.abs())


def lin(g, vha, inv):
    """Magnitude of inv (g - mean g - vhat mean(g vhat)) from magnitudes."""
    return inv * (g + g.mean(1, keepdim=True) + vha * (g * vha).mean(1, keepdim=True))


# ----------------------------------------------------------------------------- calls
def make(rows, c, stream, branch, post, pre, gate, seed, has_f=True, params=True, scale=1.0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    ts, tb = DT[stream][0], DT[branch][0]
    t = dict(rows=rows, c=c, stream=stream, branch=branch, post=post, pre=pre)
    t["rpg"] = gate if gate else 0
    t["x"] = (2 * scale * rn(rows, c) + 0.5).to(ts)
    t["f"] = (1.5 * scale * rn(rows, c) + 0.3).to(tb) if has_f else None
    t["gate"] = (0.7 + 0.5 * rn(rows // gate, c)).to(tb) if gate else None
    t["res_scale"] = 0.5 + 0.2 * rn(c) if has_f and params else None
    t["post_w"] = 1 + 0.2 * rn(c) if post != "none" and params else None
    t["post_b"] = 0.2 * rn(c) if post == "layer" and params else None
    t["pre_w"] = 1 + 0.2 * rn(c) if pre != "none" and params else None
    t["pre_b"] = 0.2 * rn(c) if pre == "layer" and params else None
    t["dy"] = (0.3 * rn(rows, c)).to(ts)
    t["dh"] = (0.3 * rn(rows, c)).to(tb) if pre != "none" else None
    return t


def shape_of(t):
    return cbr.make_block_shape(t["rows"], t["c"], t["rpg"], KIND[t["post"]], KIND[t["pre"]], DT[t["stream"]][1],
                                DT[t["branch"]][1], ALPHA, EPS_POST, EPS_PRE)


def wide(t):
    return {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in t.items()}


def run_forward(t, stats=True, y=None, h=None, stream=None):
    dev = t["x"].device
    new = lambda *s: torch.empty(*s, device=dev)  # noqa: E731
    o = dict(y=None, h=None, ps=None, qs=None)
    if t["f"] is not None:
        o["y"] = torch.empty_like(t["x"]) if y is None else y
        if stats and t["post"] != "none":
            o["ps"] = new(t["rows"], 2)
    if t["pre"] != "none":
        o["h"] = torch.empty(t["rows"], t["c"], dtype=DT[t["branch"]][0], device=dev) if h is None else h
        if stats:
            o["qs"] = new(t["rows"], 2)
    cbr.cbr_block_norm_forward(shape_of(t), t["x"], t["f"], t["post_w"], t["post_b"], t["gate"], t["res_scale"],
                               t["pre_w"], t["pre_b"], o["y"], o["h"], o["ps"], o["qs"], stream)
    return o


def check_forward(t, o):
    r, w = forward64(wide(t)), wide(t)
    tb, ts = DT[t["branch"]][0], DT[t["stream"]][0]

    def close(name, got, want, tol):
        bad = ~((got.double() - want).abs() <= tol)
        assert not bad.any(), (name, int(bad.sum()), got[bad][:4], want[bad][:4], tol.expand_as(want)[bad][:4])
    ey = torch.zeros_like(r["y"])
    if t["f"] is not None:
        en = K * w["f"].abs()
        if t["post"] != "none":
            en = K * _norm_mag(w["f"], r["nhat"], r["pm"], r["pi"])
            if w["post_w"] is not None:
                en = en * w["post_w"].abs()
            en = en + K * r["n"].abs()
            if w["post_b"] is not None:
                en = en + K * w["post_b"].abs()
            if o["ps"] is not None:
                am = w["f"].abs().mean(1, keepdim=True)
                close("post mean", o["ps"][:, :1], r["pm"], K * am)
                close("post 1/std", o["ps"][:, 1:], r["pi"], K * r["pi"] * (1 + r["pi"] * am))
        ey = r["c"].abs() * en + K * (r["y"].abs() + w["x"].abs())
        close("y", o["y"], r["y"], half(ts, r["y"]) + ey)
    if t["pre"] != "none":
        q = r["qi"]
        eh = q * (ey + ey.mean(1, keepdim=True)) + r["yhat"].abs() * q * ey.square().mean(1, keepdim=True).sqrt()
        eh = eh + K * _norm_mag(r["y"], r["yhat"], r["qm"], q)
        if w["pre_w"] is not None:
            eh = eh * w["pre_w"].abs()
        if w["pre_b"] is not None:
            eh = eh + K * w["pre_b"].abs()
        close("h", o["h"], r["h"], half(tb, r["h"]) + eh)


def run_backward(t, o, want=True, dy=True, ws=None, dx=None, df=None):
    dev, c = t["x"].device, t["c"]
    sp = shape_of(t)
    new = lambda on: torch.full((c,), 7.0, device=dev) if on else None  # noqa: E731
    has_f = t["f"] is not None
    g = dict(dx=torch.empty_like(t["x"]) if dx is None else dx,
             df=(torch.empty_like(t["f"]) if df is None else df) if has_f else None,
             post_w=new(want and t["post"] != "none"), post_b=new(want and t["post"] != "none"),
             gate=torch.empty_like(t["gate"]) if want and t["gate"] is not None else None,
             res_scale=new(want and has_f), pre_w=new(want and t["pre"] != "none"),
             pre_b=new(want and t["pre"] != "none"))
    if ws is None:
        ws = torch.empty(cbr.cbr_block_norm_workspace_bytes(sp), dtype=torch.uint8, device=dev)
    y = o["y"] if has_f else t["x"]
    cbr.cbr_block_norm_backward(sp, t["dy"] if dy else None, t["dh"], y if t["pre"] != "none" else None, t["f"],
                                t["post_w"], t["post_b"], t["gate"], t["res_scale"], t["pre_w"], o["ps"], o["qs"],
                                g["dx"], g["df"], g["post_w"], g["post_b"], g["gate"], g["res_scale"], g["pre_w"],
                                g["pre_b"], ws)
    return g


def check_backward(t, o, g, dy=True):
    """Against the formulas in 64 bits, from the y and the statistics that the call was given."""
    w, ts, tb = wide(t), DT[t["stream"]][0], DT[t["branch"]][0]
    rows, c = t["rows"], t["c"]
    has_f = t["f"] is not None
    ksum = (min(rows, 1024) + 64) * U
    one = torch.ones(1, c, dtype=torch.float64, device=w["x"].device)
    zero = torch.zeros(rows, c, dtype=torch.float64, device=w["x"].device)
    d = w["dy"] if dy else zero
    ed = K * d.abs()

    def close(name, got, want, tol):
        bad = ~((got.double() - want).abs() <= tol)
        assert not bad.any(), (name, int(bad.sum()), got[bad][:4], want[bad][:4], tol.expand_as(want)[bad][:4])

    def back(gv, vh, inv, kind):
        r = gv - vh * (gv * vh).mean(1, keepdim=True)
        return inv * (r - gv.mean(1, keepdim=True) if kind == "layer" else r)
    if t["pre"] != "none":
        y = (o["y"] if has_f else t["x"]).double()
        mean, inv = o["qs"].double()[:, :1], o["qs"].double()[:, 1:]
        yh, yha = (y - mean) * inv, (y.abs() + mean.abs()) * inv
        gw = w["dh"] * (one if w["pre_w"] is None else w["pre_w"])
        d = d + back(gw, yh, inv, t["pre"])
        ed = ed + K * lin(gw.abs(), yha, inv)
        if g["pre_w"] is not None:
            close("dpre_w", g["pre_w"], (w["dh"] * yh).sum(0), (ksum + K) * (w["dh"].abs() * yha).sum(0))
            close("dpre_b", g["pre_b"], w["dh"].sum(0), ksum * w["dh"].abs().sum(0))
    close("dx", g["dx"], d, half(ts, d) + ed)
    if not has_f:
        return
    co = ALPHA * (one if w["res_scale"] is None else w["res_scale"][None])
    pw = one if w["post_w"] is None else w["post_w"][None]
    pb = 0 * one if w["post_b"] is None else w["post_b"][None]
    gate = one if w["gate"] is None else w["gate"].repeat_interleave(t["rpg"], 0)
    if t["post"] != "none":
        mean, inv = o["ps"].double()[:, :1], o["ps"].double()[:, 1:]
        nh, nha = (w["f"] - mean) * inv, (w["f"].abs() + mean.abs()) * inv
    else:
        nh, nha, pw, pb = w["f"], w["f"].abs(), one, 0 * one
    u = co * gate * d
    if t["post"] != "none":
        uw, euw = u * pw, (co * gate * pw).abs() * ed
        df = back(uw, nh, inv, t["post"])
        close("df", g["df"], df, half(tb, df) + lin(euw, nha, inv) + K * lin(uw.abs(), nha, inv))
    else:
        close("df", g["df"], u, half(tb, u) + (co * gate).abs() * ed + K * u.abs())
    if g["res_scale"] is None and g["gate"] is None:
        return
    s1, s0 = d * nh, d
    e1, e0 = ed * nha + K * d.abs() * nha, ed
    rpg = t["rpg"] or rows
    seg = lambda v: v.view(-1, rpg, c).sum(1)  # noqa: E731
    gr = w["gate"] if w["gate"] is not None else one
    if g["gate"] is not None:
        want = co * (pw * seg(s1) + pb * seg(s0))
        mag = pw.abs() * seg(s1.abs()) + pb.abs() * seg(s0.abs())
        err = co.abs() * (pw.abs() * seg(e1) + pb.abs() * seg(e0) + (ksum + K) * mag)
        close("dgate", g["gate"], want, half(tb, want) + err)
    a1, a0 = (gr.abs() * seg(s1.abs())).sum(0), (gr.abs() * seg(s0.abs())).sum(0)
    b1, b0 = (gr.abs() * seg(e1)).sum(0), (gr.abs() * seg(e0)).sum(0)
    t1, t0 = (gr * seg(s1)).sum(0), (gr * seg(s0)).sum(0)
    ks = ksum + K
    if g["res_scale"] is not None:
        close("dres_scale", g["res_scale"], ALPHA * (pw * t1 + pb * t0)[0],
              ALPHA * (pw.abs() * (b1 + ks * a1) + pb.abs() * (b0 + ks * a0))[0])
    if g["post_w"] is not None:
        close("dpost_w", g["post_w"], (co * t1)[0], (co.abs() * (b1 + ks * a1))[0])
        close("dpost_b", g["post_b"], (co * t0)[0], (co.abs() * (b0 + ks * a0))[0])


def both(t, dy=True):
    o = run_forward(t)
    check_forward(t, o)
    g = run_backward(t, o, dy=dy)
    check_backward(t, o, g, dy=dy)
    return o, g


# ------------------------------------------------------------------------- CPU tests
def test_formula_gradients_match_differences():
    """The 64-bit formulas that the kernels are held to have the gradients of the forward."""
    t = wide(make(6, 5, "f32", "f32", "layer", "rms", 3, 1, device="cpu"))
    for k in ("post_w", "post_b", "pre_w", "gate", "res_scale", "x", "f"):
        t[k] = t[k].requires_grad_()
    names = ["x", "f", "gate", "res_scale", "post_w", "post_b", "pre_w"]

    def loss(*vals):
        o = forward64({**t, **dict(zip(names, vals))})
        return (o["y"] * t["dy"]).sum() + (o["h"] * t["dh"]).sum()
    assert torch.autograd.gradcheck(loss, [t[k] for k in names], eps=1e-6, atol=1e-6)


FAKE = 0x100000


def _fwd(sp, **over):
    a = dict(x=FAKE, f=FAKE, post_w=FAKE, post_b=FAKE, gate=FAKE, res=FAKE, pre_w=FAKE, pre_b=FAKE, y=FAKE, h=FAKE,
             ps=FAKE, qs=FAKE)
    a.update(over)
    return cbr._load().cbr_block_norm_forward(ctypes.byref(sp), *a.values(), 0)


def _bwd(sp, **over):
    a = dict(dy=FAKE, dh=FAKE, y=FAKE, f=FAKE, post_w=FAKE, post_b=FAKE, gate=FAKE, res=FAKE, pre_w=FAKE, ps=FAKE,
             qs=FAKE, dx=FAKE, df=FAKE, dpw=FAKE, dpb=FAKE, dg=FAKE, dr=FAKE, dqw=FAKE, dqb=FAKE, ws=FAKE, nb=1 << 40)
    a.update(over)
    return cbr._load().cbr_block_norm_backward(ctypes.byref(sp), *a.values(), 0)


def sh(rows=64, c=32, rpg=8, post=2, pre=2, ts=0, tb=0, **kw):
    return cbr.make_block_shape(rows, c, rpg, post, pre, ts, tb, **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), 2), (dict(rows=-3), 2), (dict(c=0), 2), (dict(rows=1 << 31, rpg=1), 3), (dict(c=8193), 3),
    (dict(post=3), 7), (dict(pre=-1), 7), (dict(ts=3), 7), (dict(tb=9), 7), (dict(ts=0, tb=1), 3), (dict(ts=1, tb=0), 3),
    (dict(ts=0, tb=2), 3), (dict(rpg=7), 2), (dict(rpg=0), 2), (dict(rpg=-8), 2), (dict(alpha=float("nan")), 7),
    (dict(eps_post=-1e-5), 7), (dict(eps_pre=float("inf")), 7),
])
def test_shape_refusals(kw, status):
    assert _fwd(sh(**kw)) == status
    assert _bwd(sh(**kw)) == status
    if "rpg" not in kw or "rows" in kw:
        assert cbr.cbr_block_norm_workspace_bytes(sh(**kw)) == 0


@pytest.mark.parametrize("shape,over,status", [
    ({}, dict(x=None), 1), ({}, dict(y=None), 1), ({}, dict(h=None), 1),
    ({}, dict(f=None), 7), (dict(post=0), dict(), 7), (dict(post=0), dict(post_w=None, post_b=None, ps=FAKE), 7),
    (dict(pre=0), dict(), 7), (dict(pre=0), dict(pre_w=None, pre_b=None, qs=None), 7),
    (dict(post=0, pre=0), dict(f=None, post_w=None, post_b=None, gate=None, res=None, pre_w=None, pre_b=None, y=None,
                               h=None, ps=None, qs=None), 7),
    ({}, dict(x=FAKE + 8), 4), ({}, dict(gate=FAKE + 2), 4), ({}, dict(post_w=FAKE + 4), 4), ({}, dict(h=FAKE + 2), 4),
    ({}, dict(qs=FAKE + 8), 4),
])
def test_forward_refusals(shape, over, status):
    assert _fwd(sh(**shape), **over) == status


@pytest.mark.parametrize("shape,over,status", [
    ({}, dict(dx=None), 1), ({}, dict(dh=None), 1), ({}, dict(y=None), 1), ({}, dict(qs=None), 1), ({}, dict(df=None), 1),
    ({}, dict(ps=None), 1), ({}, dict(f=None), 1), (dict(pre=0), dict(dy=None, dh=None, qs=None, pre_w=None, dqw=None, dqb=None), 1),
    (dict(pre=0), dict(), 7), (dict(post=0), dict(), 7), ({}, dict(gate=None), 7), (dict(post=0), dict(f=None), 7),
    ({}, dict(dy=FAKE + 4), 4), ({}, dict(dg=FAKE + 2), 4), ({}, dict(ws=FAKE + 4), 4),
    ({}, dict(ws=None), 5), ({}, dict(nb=16), 5),
])
def test_backward_refusals(shape, over, status):
    assert _bwd(sh(**shape), **over) == status


def test_null_shape_and_binding_refusals():
    L = cbr._load()
    assert L.cbr_block_norm_forward(None, *([FAKE] * 12), 0) == 1
    assert L.cbr_block_norm_backward(None, *([FAKE] * 20), 1 << 30, 0) == 1
    assert L.cbr_block_norm_workspace_bytes(None) == 0
    host = torch.zeros(64, 32, dtype=torch.bfloat16)
    with pytest.raises(cbr.CbrError, match="not a GPU tensor"):
        cbr.cbr_block_norm_forward(sh(), host, host, None, None, None, None, None, None, host, host)
    with pytest.raises(cbr.CbrError):
        cbr.cbr_block_norm_forward(sh(ts=7), *([None] * 10))


# ------------------------------------------------------------------------- GPU tests
gpu = pytest.mark.gpu

# rows, channels, rows of a gate row (0: no gate).  Channels: one value, parts of a chunk of
# eight, one lane to sixteen waves a row (8 values a thread), sixteen values a thread (bwd).
SIZES = [(1, 1, 0), (1, 8, 1), (3, 7, 3), (37, 9, 0), (64, 64, 16), (50, 100, 5), (33, 129, 1), (196, 256, 196),
         (21, 512, 7), (19, 520, 0), (16, 1000, 4), (10, 1001, 2), (9, 2048, 3), (5, 4096, 0), (5, 4099, 5),
         (4, 8192, 2), (3, 8191, 1)]


@gpu
@pytest.mark.parametrize("rows,c,gate", SIZES, ids=str)
@pytest.mark.parametrize("post,pre", [("layer", "rms"), ("rms", "layer")])
def test_sizes(rows, c, gate, post, pre):
    both(make(rows, c, "bf16", "bf16", post, pre, gate, rows * 7 + c))


@gpu
@pytest.mark.parametrize("stream,branch", [("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("c,gate", [(72, 6), (131, 0)])
def test_types_and_kinds(stream, branch, post, pre, c, gate):
    both(make(30, c, stream, branch, post, pre, gate, 3))


@gpu
@pytest.mark.parametrize("post,pre", [("layer", "layer"), ("none", "none"), ("rms", "rms")])
@pytest.mark.parametrize("rows,c,gate", [(24, 40, 0), (24, 40, 4), (700, 33, 350)])
def test_without_parameters(post, pre, rows, c, gate):
    """No weights, biases or residual scale: read as 1 and 0, and their gradients still exist."""
    both(make(rows, c, "bf16", "bf16", post, pre, gate, 5, params=False))


@gpu
@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("dy", [True, False])
def test_first_block_has_no_branch(pre, dy):
    both(make(45, 96, "f32", "bf16", "none", pre, 0, 6, has_f=False), dy=dy)


@gpu
@pytest.mark.parametrize("rows,c,gate", [
    (4096, 64, 1024),     # gate rows shared out among workgroups
    (4096, 8, 4096),      # 512 rows a workgroup
    (6000, 64, 3),        # many short gate rows: whole ones to each group of threads
    (3000, 512, 1),       # a gate row for every row
    (1500, 24, 500),
    (2048, 256, 0),
], ids=str)
def test_sums_over_many_rows(rows, c, gate):
    both(make(rows, c, "bf16", "bf16", "layer", "layer", gate, 11))


@gpu
def test_gradients_against_differences():
    """The kernels' gradients along a direction against central differences of the 64-bit loss.
    The loss is smooth on the scale of the step (1e-4 of values of order 1): the differences are
    good to about 1e-8 of the sum of magnitudes (third derivative, step^2 / 6), far below K."""
    t = make(60, 48, "f32", "f32", "layer", "rms", 20, 9)
    o = run_forward(t)
    g = run_backward(t, o)
    grads = dict(x=g["dx"], f=g["df"], gate=g["gate"], res_scale=g["res_scale"], post_w=g["post_w"], post_b=g["post_b"],
                 pre_w=g["pre_w"])
    w = wide(t)
    gen = torch.Generator(device="cuda").manual_seed(2)

    def loss(v):
        r = forward64(v)
        return float((r["y"] * w["dy"]).sum() + (r["h"] * w["dh"]).sum())
    for k, gv in grads.items():
        d = torch.randn(w[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        e = 1e-4
        num = (loss({**w, k: w[k] + e * d}) - loss({**w, k: w[k] - e * d})) / (2 * e)
        got = float((gv.double() * d).sum())
        mag = float((gv.double().abs() * d.abs()).sum())
        # the gradient's own error (sums of 60 rows and 48 channels, two norms deep) and the differences'
        assert abs(num - got) <= 16 * K * mag + 1e-6 * mag, (k, num, got, mag)


@gpu
def test_in_place():
    """y may be x and h may be f; dx may be dy and df may be f or dh."""
    for c in (64, 77):
        t = make(50, c, "bf16", "bf16", "layer", "rms", 10, 12)
        o = run_forward(t)
        g = run_backward(t, o)
        x, f = t["x"].clone(), t["f"].clone()
        o2 = run_forward({**t, "x": x, "f": f}, y=x, h=f)
        assert torch.equal(o2["y"], o["y"]) and torch.equal(o2["h"], o["h"])
        dy, dh = t["dy"].clone(), t["dh"].clone()
        g2 = run_backward({**t, "dy": dy, "dh": dh}, o, dx=dy, df=dh)
        f = t["f"].clone()
        g3 = run_backward({**t, "f": f}, o, df=f)
        for k in g:
            assert torch.equal(g2[k], g[k]) and torch.equal(g3[k], g[k]), k


@gpu
def test_special_rows():
    """Constant rows, zero rows, large means, infinities and NaN stay in their own rows."""
    t = make(12, 136, "f32", "bf16", "layer", "layer", 0, 13)
    t["f"][0] = 0
    t["f"][1] = 3.0
    t["x"][1] = -2.0
    t["f"][2] += 100.0
    o, _ = both(t)
    clean = run_forward(t)
    bad = {**t, "f": t["f"].clone(), "x": t["x"].clone()}
    bad["f"][4, 7] = float("inf")
    bad["f"][5, 0] = float("nan")
    bad["x"][6, 135] = float("-inf")
    o = run_forward(bad)
    keep = [i for i in range(12) if i not in (4, 5, 6)]
    assert torch.equal(o["y"][keep], clean["y"][keep]) and torch.equal(o["h"][keep], clean["h"][keep])
    assert o["y"][4].isnan().all() or not o["y"][4].isfinite().all()
    assert o["h"][5].isnan().all() and o["h"][6].isnan().all()


@gpu
def test_eps_zero_and_zero_row_is_nan_as_the_formula_says():
    t = make(2, 16, "f32", "f32", "none", "rms", 0, 1, has_f=False)
    t["x"][0] = 0
    sp = cbr.make_block_shape(2, 16, 0, 0, 1, cbr.CBR_F32, cbr.CBR_F32, 1.0, 0.0, 0.0)
    h = torch.empty(2, 16, device="cuda")
    cbr.cbr_block_norm_forward(sp, t["x"], None, None, None, None, None, t["pre_w"], None, None, h)
    assert h[0].isnan().all() and h[1].isfinite().all()


@gpu
def test_reproducible_and_partial_outputs():
    t = make(3000, 200, "bf16", "bf16", "layer", "layer", 300, 14)
    o, g = both(t)
    o2 = run_forward(t, stats=False)
    assert torch.equal(o2["y"], o["y"]) and torch.equal(o2["h"], o["h"])
    ws = torch.full((cbr.cbr_block_norm_workspace_bytes(shape_of(t)),), 255, dtype=torch.uint8, device="cuda")
    g2 = run_backward(t, o, ws=ws)          # the workspace's content does not matter
    assert all(torch.equal(g[k], g2[k]) for k in g)
    g3 = run_backward(t, o, want=False)     # no parameter's gradient
    assert torch.equal(g3["dx"], g["dx"]) and torch.equal(g3["df"], g["df"])


@gpu
def test_other_stream_and_graph():
    """On a side stream, and captured: replayed on new inputs with eager work in between."""
    t = make(512, 256, "bf16", "bf16", "layer", "rms", 128, 15)
    want_o, want_g = both(t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o = run_forward(t)
        g = run_backward(t, o)
    s.synchronize()
    assert torch.equal(o["h"], want_o["h"]) and all(torch.equal(g[k], want_g[k]) for k in g)
    ws = torch.empty(cbr.cbr_block_norm_workspace_bytes(shape_of(t)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = run_forward(t)
        g = run_backward(t, o, ws=ws)
    for seed in (16, 17, 18):
        new = make(512, 256, "bf16", "bf16", "layer", "rms", 128, seed)
        for k in ("x", "f", "dy", "dh", "gate"):
            t[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        eo = run_forward(t)
        eg = run_backward(t, eo)
        torch.cuda.synchronize()
        assert torch.equal(o["y"], eo["y"]) and torch.equal(o["h"], eo["h"])
        assert all(torch.equal(g[k], eg[k]) for k in g)


@gpu
def test_binding_refuses_wrong_tensors():
    sp = sh(64, 32, 8, 0, 0)
    x = torch.zeros(64, 32, dtype=torch.bfloat16, device="cuda")
    call = lambda x, f, y, gate=None: cbr.cbr_block_norm_forward(sp, x, f, None, None, gate, None, None, None, y, None)  # noqa: E731
    with pytest.raises(cbr.CbrError, match="x is torch.float16"):
        call(x.half(), x, x.clone())
    with pytest.raises(cbr.CbrError, match="contiguous"):
        call(x.t(), x, x.clone())
    with pytest.raises(cbr.CbrError, match="f holds"):
        call(x, x[:32], x.clone())
    with pytest.raises(cbr.CbrError, match="gate holds"):
        call(x, x, x.clone(), gate=x[:7])
    call(x, x, x.clone(), gate=x[:8])
