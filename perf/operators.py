"""The block norm, the 8-bit quantiser and the 8-bit matrix product: cases, inputs, plain forms and exact values.

A case names its operator ("op") and plain sizes.  ``run`` with ``own`` false computes the operator
with elementary torch operations in 32 bits; with ``own`` true it makes the library's call.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
MANT = {"e4m3": (3, -6), "e5m2": (2, -14)}   # mantissa bits, exponent of the smallest normal value
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1, "e5m2": 1}
BLK = 128
ALPHA = 0.75
EPS = 1e-5


# ------------------------------------------------------------------------------- cases
def _norm(name, op, images, pixels, c, stream, branch, post, pre, gate):
    """images x pixels rows of c channels; gate "image": one gate row an image, "pixel": one a
    row, "none".  Every case has a residual scale and the norms' weights (layer: biases too)."""
    return dict(name=name, op=op, images=images, pixels=pixels, c=c, stream=stream, branch=branch, post=post, pre=pre,
                gate=gate)


def _quant(name, rows, cols, src, fmt, transpose, block):
    return dict(name=name, op="quantize", rows=rows, cols=cols, src=src, fmt=fmt, transpose=transpose, block=block)


def _gemm(name, m, n, k, a, b, block, out, bias, relu):
    return dict(name=name, op="gemm", m=m, n=n, k=k, a=a, b=b, block=block, out=out, bias=bias, relu=relu)


def listed():
    return [
        # One image's 7x7 map in inference: a call that latency decides.
        _norm("norm_fwd_7x7x512", "norm_fwd", 1, 49, 512, "bf16", "bf16", "rms", "rms", "image"),
        # An odd channel count on a small batch, half precision branch on a single precision stream.
        _norm("norm_fwd_odd_1001", "norm_fwd", 16, 225, 1001, "f32", "f16", "layer", "layer", "pixel"),
        # The 28x28 stage of a 256-image training batch.
        _norm("norm_fwd_28x28x512", "norm_fwd", 256, 784, 512, "bf16", "bf16", "layer", "rms", "image"),
        # The backward of one image's 14x14 map: launches and the small reductions.
        _norm("norm_bwd_14x14x256", "norm_bwd", 1, 196, 256, "bf16", "bf16", "layer", "layer", "image"),
        # Wide rows on a single precision stream: the sums over rows of 4096 channels.
        _norm("norm_bwd_4096x4096", "norm_bwd", 4, 1024, 4096, "f32", "bf16", "rms", "rms", "none"),
        # The 56x56 stage of a 64-image training batch, a gate an image.
        _norm("norm_bwd_56x56x256", "norm_bwd", 64, 3136, 256, "bf16", "bf16", "layer", "layer", "image"),
        # A small batch's features on their way into a product.
        _quant("quant_rows_64x2048", 64, 2048, "bf16", "e4m3", False, 1),
        # The 14x14 stage's activations turned over for the weight gradient.
        _quant("quant_turned_50176x1024", 50176, 1024, "bf16", "e4m3", True, 1),
        # One image's features into 1000 classes.
        _gemm("gemm_classes_1x1000x2048", 1, 1000, 2048, "e4m3", "e4m3", 128, "f32", True, False),
        # A 1x1 layer of the 14x14 stage, 256 images less a few, bias and ReLU.
        _gemm("gemm_1x1_50001x256x1024", 50001, 256, 1024, "e4m3", "e4m3", 128, "bf16", True, True),
        # The same layer's weight gradient: a long sum over pixels, few outputs.
        _gemm("gemm_wgrad_1024x256x50176", 1024, 256, 50176, "e4m3", "e4m3", 1, "f32", False, False),
        # A large square product with the gradient's wider format: the card's rate.
        _gemm("gemm_square_8192", 8192, 8192, 8192, "e5m2", "e4m3", 128, "bf16", False, False),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("norm_fwd", "norm_bwd", "quantize", "gemm"))
    if kind.startswith("norm"):
        c = _logint(rng, 17, 8192)
        if rng.random() < 0.5:
            c = max(16, c // 16 * 16)
        images = _logint(rng, 1, 64)
        pixels = _logint(rng, 1, max(1, min(3136, 20_000_000 // (images * c))))
        stream, branch = rng.choice((("bf16", "bf16"), ("f32", "bf16"), ("f16", "f16"), ("f32", "f16"), ("f32", "f32")))
        return dict(op=kind, images=images, pixels=pixels, c=c, stream=stream, branch=branch,
                    post=rng.choice(("none", "rms", "layer")), pre=rng.choice(("none", "rms", "layer")),
                    gate=rng.choice(("none", "image", "pixel")))
    if kind == "quantize":
        cols = _logint(rng, 33, 8192)
        rows = _logint(rng, 1, min(65536, 50_000_000 // cols))
        transpose = rng.random() < 0.5
        return dict(op=kind, rows=rows, cols=cols, src=rng.choice(("bf16", "f16", "f32")), fmt=rng.choice(("e4m3", "e5m2")),
                    transpose=transpose, block=rng.choice((1, 128)))
    m, n, k = _logint(rng, 1, 65536), _logint(rng, 16, 8192), _logint(rng, 32, 8192)
    if rng.random() < 0.5:
        n, k = max(16, n // 16 * 16), max(64, k // 64 * 64)
    m = max(1, min(m, 67_000_000 // max(n, k), 2 ** 39 // (n * k)))
    if rng.random() < 0.2:   # a weight gradient's shape: the long axis is summed over
        m, k = max(16, k // 4), max(m, 64)
    return dict(op=kind, m=m, n=n, k=k, a=rng.choice(("e4m3", "e5m2")), b="e4m3", block=rng.choice((1, 128)),
                out=rng.choice(("bf16", "f16", "f32")), bias=rng.random() < 0.5, relu=rng.random() < 0.3)


def _cdiv(a, b):
    return -(-a // b)


def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        rows, c = case["images"] * case["pixels"], case["c"]
        s, b = SIZE[case["stream"]], SIZE[case["branch"]]
        h = case["pre"] != "none"
        gates = {"none": 0, "image": case["images"], "pixel": rows}[case["gate"]] * c * b
        if op == "norm_fwd":   # x, f in; y, h out; two statistics a row and norm
            return {"bytes": rows * c * (2 * s + b + h * b) + gates + 8 * rows * (h + (case["post"] != "none")) + 20 * c,
                    "flops": 14 * rows * c}
        # dy, f, (dh, y) in; dx, df out
        return {"bytes": rows * c * (2 * s + 2 * b + h * (b + s)) + 2 * gates + 8 * rows * (h + (case["post"] != "none")) + 36 * c,
                "flops": 30 * rows * c}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (SIZE[case["src"]] + 1) + 4 * (n // (BLK * case["block"])), "flops": 4 * n}
    m, n, k = case["m"], case["n"], case["k"]
    kb = _cdiv(k, BLK)
    return {"bytes": m * k + n * k + m * n * SIZE[case["out"]] + 4 * kb * (m + _cdiv(n, case["block"])) + 4 * n * case["bias"],
            "flops": 2 * m * n * k}


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _quantized(v, fmt, block):
    """v [rows, k] in fmt, in groups of 128 values of a row or blocks of 128 x 128, and the scales
    [k blocks, row blocks].  Divided by the largest value, not by the rounded scale: a value midway
    between two 8-bit ones (3/4 of a power of two times the largest, say) is then met exactly.
    (Tensors divide tensors here: torch multiplies by the reciprocal of a plain number.)"""
    rows, k = v.shape
    kb, rb = _cdiv(k, BLK), _cdiv(rows, block)
    p = torch.zeros(rb * block, kb * BLK, device=v.device)
    p[:rows, :k] = v
    p = p.view(rb, block, kb, BLK)
    amax = p.abs().amax((1, 3)).clamp_min(FMAX[fmt] * 2.0 ** -126)              # [rb, kb]
    q = (p * 0.875 / amax[:, None, :, None]) * (FMAX[fmt] / 0.875)
    q = q.view(rb * block, kb * BLK)[:rows, :k].to(TYPES[fmt])
    return q, (amax / torch.full_like(amax, FMAX[fmt])).t().contiguous()


def _encode(v, fmt, block):
    """Operand v in 8 bits with its scales, as a program holds it: rows padded to 16 bytes."""
    q, s = _quantized(v, fmt, block)
    out = torch.zeros(v.shape[0], _cdiv(v.shape[1], 16) * 16, dtype=torch.uint8, device=v.device)
    out[:, :v.shape[1]] = q.view(torch.uint8)
    return out, s


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        rows, c = case["images"] * case["pixels"], case["c"]
        ts, tb = TYPES[case["stream"]], TYPES[case["branch"]]
        vec = lambda mean, dev: mean + dev * _randn(g, c)  # noqa: E731
        st["f"] = (_randn(g, rows, c) * 1.5 + 0.3).to(tb)
        st["post_w"] = vec(1.0, 0.2) if case["post"] != "none" else None
        st["post_b"] = vec(0.0, 0.2) if case["post"] == "layer" else None
        st["pre_w"] = vec(1.0, 0.2) if case["pre"] != "none" else None
        st["pre_b"] = vec(0.0, 0.2) if case["pre"] == "layer" else None
        st["res_scale"] = vec(0.5, 0.2)
        gates = {"none": 0, "image": case["images"], "pixel": rows}[case["gate"]]
        st["gate"] = (0.7 + 0.5 * _randn(g, gates, c)).to(tb) if gates else None
        st["rows_per_gate"] = {"none": 0, "image": case["pixels"], "pixel": 1}[case["gate"]]
        if op == "norm_fwd":
            st["x"] = (2.0 * _randn(g, rows, c)).to(ts)
        else:
            st["y"] = (2.0 * _randn(g, rows, c)).to(ts)
            st["dy"] = (0.1 * _randn(g, rows, c)).to(ts)
            st["dh"] = (0.1 * _randn(g, rows, c)).to(tb) if case["pre"] != "none" else None
            st["post_stats"] = _stats(st["f"], case["post"])
            st["pre_stats"] = _stats(st["y"], case["pre"])
        return st
    if op == "quantize":
        v = _randn(g, case["rows"], case["cols"])
        st["src"] = (v * torch.exp(0.5 * _randn(g, 1, case["cols"]))).to(TYPES[case["src"]])
        return st
    m, n, k = case["m"], case["n"], case["k"]
    a, st["a_scale"] = _encode(_randn(g, m, k).clamp_min(-0.5), case["a"], 1)
    b, st["b_scale"] = _encode(_randn(g, n, k) * (2.0 / k) ** 0.5, case["b"], case["block"])
    st["a_q"], st["b_q"] = a, b
    st["bias_v"] = 0.1 * _randn(g, n) if case["bias"] else None
    return st


def _stats(v, kind):
    """(mean, 1/std) of each row as the forward saves them; the mean of an rms norm is 0."""
    if kind == "none":
        return None
    v = v.double()
    mean = v.mean(1) if kind == "layer" else torch.zeros(v.shape[0], dtype=v.dtype, device=v.device)
    var = (v - mean[:, None]).square().mean(1)
    return torch.stack((mean, (var + EPS).rsqrt()), 1).float()


# ------------------------------------------------------------------------- plain forms
def _normed(v, kind):
    """The row's normalised values and its (mean, 1/std), in 32 bits."""
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros(v.shape[0], 1, device=v.device)
    d = v - mean
    inv = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    return d * inv, torch.cat((mean, inv), 1)


def _affine(v, w, b):
    v = v * w
    return v if b is None else v + b


def _gate_rows(st, rows):
    """alpha * residual scale * gate, by rows [gates, pixels of a gate, C] or as one row."""
    coef = ALPHA * st["res_scale"]
    if st["gate"] is None:
        return coef[None, None]
    return (coef * st["gate"].float())[:, None]


def _plain_norm_fwd(st):
    x, f = st["x"].float(), st["f"].float()
    rows, c = f.shape
    out = {}
    if st["post"] != "none":
        f, out["post_stats"] = _normed(f, st["post"])
        f = _affine(f, st["post_w"], st["post_b"])
    rpg = st["rows_per_gate"] or rows
    y = x + (f.view(-1, rpg, c) * _gate_rows(st, rows)).view(rows, c)
    out["y"] = y.to(st["x"].dtype)
    if st["pre"] != "none":
        h, out["pre_stats"] = _normed(y, st["pre"])
        out["h"] = _affine(h, st["pre_w"], st["pre_b"]).to(st["f"].dtype)
    return out


def _norm_grad(gv, vhat, inv, kind):
    """Gradient of a row's norm to its input from gv, the gradient to the normalised values."""
    r = gv - vhat * (gv * vhat).mean(1, keepdim=True)
    if kind == "layer":
        r = r - gv.mean(1, keepdim=True)
    return r * inv


def _plain_norm_bwd(st):
    out = {}
    d, f = st["dy"].float(), st["f"].float()
    rows, c = f.shape
    if st["pre"] != "none":
        ps, dh = st["pre_stats"], st["dh"].float()
        yhat = (st["y"].float() - ps[:, :1]) * ps[:, 1:]
        d = d + _norm_grad(dh * st["pre_w"], yhat, ps[:, 1:], st["pre"])
        out["dpre_w"] = (dh * yhat).sum(0)
        if st["pre_b"] is not None:
            out["dpre_b"] = dh.sum(0)
    out["dx"] = d.to(st["dy"].dtype)
    rpg = st["rows_per_gate"] or rows
    if st["post"] != "none":
        qs = st["post_stats"]
        nhat = (f - qs[:, :1]) * qs[:, 1:]
        n = _affine(nhat, st["post_w"], st["post_b"])
    else:
        nhat = n = f
    coef = _gate_rows(st, rows)
    u = (d.view(-1, rpg, c) * coef).view(rows, c)      # gradient to the norm's output n
    s = (d * n).view(-1, rpg, c).sum(1)                # [gates, C]
    gate = st["gate"].float() if st["gate"] is not None else torch.ones(1, c, device=f.device)
    if st["gate"] is not None:
        out["dgate"] = (s * (ALPHA * st["res_scale"])).to(st["gate"].dtype)
    out["dres_scale"] = ALPHA * (s * gate).sum(0)
    if st["post"] != "none":
        out["dpost_w"] = (u * nhat).sum(0)
        if st["post_b"] is not None:
            out["dpost_b"] = u.sum(0)
        u = _norm_grad(u * st["post_w"], nhat, qs[:, 1:], st["post"])
    out["df"] = u.to(st["f"].dtype)
    return out


def _plain_quantize(st):
    v = st["src"].float()
    q, scale = _quantized(v.t() if st["transpose"] else v, st["fmt"], st["block"])
    return {"q": q, "scale": scale}


def _values(q, scale, fmt, rows, k, block):
    """What an 8-bit operand stands for, in 32 bits."""
    v = q[:, :k].contiguous().view(TYPES[fmt]).float()
    s = scale.t()                                     # [row blocks, k blocks]
    if block > 1:
        s = s.repeat_interleave(block, 0)[:rows]
    return v * s.repeat_interleave(BLK, 1)[:, :k]


def _plain_gemm(st):
    m, n, k = st["m"], st["n"], st["k"]
    a = _values(st["a_q"], st["a_scale"], st["a"], m, k, 1)
    b = _values(st["b_q"], st["b_scale"], st["b"], n, k, st["block"])
    d = a @ b.t()
    if st["bias_v"] is not None:
        d = d + st["bias_v"]
    if st["relu"]:
        d = d.clamp_min(0.0)
    return d.to(TYPES[st["out"]])


# --------------------------------------------------------------------- the library's calls
def _own_norm(cbr, st):
    rows, c = st["f"].shape
    dt = {"bf16": cbr.CBR_BF16, "f16": cbr.CBR_F16, "f32": cbr.CBR_F32}
    kind = {"none": cbr.CBR_NORM_NONE, "rms": cbr.CBR_NORM_RMS, "layer": cbr.CBR_NORM_LAYER}
    if "sp" not in st:
        st["sp"] = cbr.make_block_shape(rows, c, rows_per_gate=st["rows_per_gate"], post=kind[st["post"]],
                                        pre=kind[st["pre"]], stream_type=dt[st["stream"]],
                                        branch_type=dt[st["branch"]], alpha=ALPHA, eps_post=EPS, eps_pre=EPS)
    sp, f = st["sp"], st["f"]
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device=f.device)  # noqa: E731
    post, pre = st["post"] != "none", st["pre"] != "none"
    if st["op"] == "norm_fwd":
        y = torch.empty_like(st["x"])
        h = torch.empty_like(f) if pre else None
        ps = new(rows, 2) if post else None
        qs = new(rows, 2) if pre else None
        cbr.cbr_block_norm_forward(sp, st["x"], f, st["post_w"], st["post_b"], st["gate"], st["res_scale"],
                                   st["pre_w"], st["pre_b"], y, h, ps, qs)
        out = {"post_stats": ps, "y": y, "pre_stats": qs, "h": h}
        order = (["post_stats"] if post else []) + ["y"] + (["pre_stats", "h"] if pre else [])
        return {k: out[k] for k in order}
    if "ws" not in st:
        st["ws"] = new(max(256, cbr.cbr_block_norm_workspace_bytes(sp)), dtype=torch.uint8)
    vec = lambda like: None if like is None else torch.empty_like(like)  # noqa: E731
    out = {"dpre_w": vec(st["pre_w"]), "dpre_b": vec(st["pre_b"]), "dx": torch.empty_like(st["dy"]),
           "dgate": vec(st["gate"]), "dres_scale": vec(st["res_scale"]), "dpost_w": vec(st["post_w"]),
           "dpost_b": vec(st["post_b"]), "df": torch.empty_like(f)}
    cbr.cbr_block_norm_backward(sp, st["dy"], st["dh"], st["y"] if pre else None, f, st["post_w"], st["post_b"],
                                st["gate"], st["res_scale"], st["pre_w"], st["post_stats"], st["pre_stats"],
                                out["dx"], out["df"], out["dpost_w"], out["dpost_b"], out["dgate"],
                                out["dres_scale"], out["dpre_w"], out["dpre_b"], st["ws"])
    return {k: v for k, v in out.items() if v is not None}


def _own_quantize(cbr, st):
    rows, cols = (st["cols"], st["rows"]) if st["transpose"] else (st["rows"], st["cols"])
    dt = {"bf16": cbr.CBR_BF16, "f16": cbr.CBR_F16, "f32": cbr.CBR_F32, "e4m3": cbr.CBR_E4M3, "e5m2": cbr.CBR_E5M2}
    if "sp" not in st:
        src = {v: dt[k] for k, v in TYPES.items()}[st["src"].dtype]
        st["sp"] = cbr.make_quant_shape(st["rows"], st["cols"], src_type=src, q_type=dt[st["fmt"]],
                                        transpose=st["transpose"], block=st["block"])
    q = torch.empty(rows, _cdiv(cols, 16) * 16, dtype=TYPES[st["fmt"]], device=st["src"].device)
    s = torch.empty(_cdiv(cols, BLK), _cdiv(rows, st["block"]), device=st["src"].device)
    cbr.cbr_fp8_quantize(st["sp"], st["src"], q, s)
    return {"q": q[:, :cols], "scale": s}


def _own_gemm(cbr, st):
    dt = {"bf16": cbr.CBR_BF16, "f16": cbr.CBR_F16, "f32": cbr.CBR_F32, "e4m3": cbr.CBR_E4M3, "e5m2": cbr.CBR_E5M2}
    if "sp" not in st:
        st["sp"] = cbr.make_gemm_shape(st["m"], st["n"], st["k"], a_type=dt[st["a"]], b_type=dt[st["b"]],
                                       b_block=st["block"], d_type=dt[st["out"]], relu=st["relu"])
        st["ws"] = torch.empty(max(256, cbr.cbr_gemm_fp8_workspace_bytes(st["sp"])), dtype=torch.uint8, device="cuda")
    d = torch.empty(st["m"], st["n"], dtype=TYPES[st["out"]], device="cuda")
    cbr.cbr_gemm_fp8(st["sp"], st["a_q"], st["a_scale"], st["b_q"], st["b_scale"], st["bias_v"], d, st["ws"])
    return d


def run(state):
    op = state["op"]
    if own:
        import conv2d_batchnorm_relu_amd as cbr
        return (_own_gemm if op == "gemm" else _own_quantize if op == "quantize" else _own_norm)(cbr, state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "quantize": _plain_quantize,
            "gemm": _plain_gemm}[op](state)


# ------------------------------------------------------------------------------- exact
def _exact_norm(v, kind, w, b):
    """torch's own row statistics in 64 bits: (mean, 1/std) and the norm."""
    if kind == "layer":
        var, mean = torch.var_mean(v, 1, correction=0)
    else:
        mean = torch.zeros_like(v[:, 0])
        var = torch.linalg.vector_norm(v, dim=1) ** 2 / v.shape[1]
    inv = 1.0 / torch.sqrt(var + EPS)
    n = w.double() * ((v - mean[:, None]) * inv[:, None])
    return torch.stack((mean, inv), 1), n if b is None else n + b.double()


def _exact_gate(st, rows):
    """alpha * residual scale * gate of every row, [rows, C] (or [1, C])."""
    r = ALPHA * st["res_scale"].double()
    if st["gate"] is None:
        return r[None]
    return r * st["gate"].double().repeat_interleave(st["rows_per_gate"], 0)


def _exact_fwd(st):
    f, x = st["f"].double(), st["x"].double()
    out = {}
    if st["post"] != "none":
        out["post_stats"], f = _exact_norm(f, st["post"], st["post_w"], st["post_b"])
    y = torch.addcmul(x, f, _exact_gate(st, f.shape[0]))
    out["y"] = y
    if st["pre"] != "none":
        out["pre_stats"], out["h"] = _exact_norm(y, st["pre"], st["pre_w"], st["pre_b"])
    return out


def _exact_bwd(st):
    """Gradients by automatic differentiation of the forward's definition in 64 bits."""
    leaf = {k: st[k].double().requires_grad_() for k in ("f", "gate", "res_scale", "post_w", "post_b", "pre_w", "pre_b")
            if st[k] is not None}
    out = {}
    d = st["dy"].double()
    if st["pre"] != "none":
        y = st["y"].double().requires_grad_()
        h = _exact_norm(y, st["pre"], leaf["pre_w"], leaf.get("pre_b"))[1]
        want = [k for k in ("pre_w", "pre_b") if k in leaf]
        got = torch.autograd.grad((h * st["dh"].double()).sum(), [y] + [leaf[k] for k in want])
        d = d + got[0]
        out.update({"d" + k: v for k, v in zip(want, got[1:])})
    out["dx"] = d
    n = leaf["f"]
    if st["post"] != "none":
        n = _exact_norm(n, st["post"], leaf["post_w"], leaf.get("post_b"))[1]
    both = dict(st, gate=leaf.get("gate"), res_scale=leaf["res_scale"])
    want = [k for k in ("gate", "res_scale", "post_w", "post_b", "f") if k in leaf]
    got = torch.autograd.grad((n * _exact_gate(both, n.shape[0]) * d).sum(), [leaf[k] for k in want])
    out.update({"d" + k: v for k, v in zip(want, got)})
    return out


def _exact_quantize(st):
    v = st["src"].double()
    v = v.t().contiguous() if st["transpose"] else v
    rows, k = v.shape
    block, fmt = st["block"], st["fmt"]
    amax = torch.nn.functional.max_pool2d(
        torch.nn.functional.pad(v.abs(), (0, -k % BLK, 0, -rows % block))[None], (block, BLK))[0]
    amax = torch.maximum(amax, torch.full_like(amax, FMAX[fmt] * 2.0 ** -126))
    s = amax / FMAX[fmt]
    each = amax.repeat_interleave(block, 0)[:rows].repeat_interleave(BLK, 1)[:, :k]
    t = v * FMAX[fmt] / each
    bits, low = MANT[fmt]
    step = torch.exp2((torch.frexp(t).exponent - 1).clamp_min(low).double() - bits)   # the format's spacing at t
    return {"q": torch.round(t / step) * step, "scale": s.t().contiguous()}


def _exact_gemm(st):
    m, n, k, block = st["m"], st["n"], st["k"], st["block"]
    a = st["a_q"][:, :k].contiguous().view(TYPES[st["a"]]).double()
    b = st["b_q"][:, :k].contiguous().view(TYPES[st["b"]]).double()
    at, bt = torch.arange(k, device=a.device) // BLK, torch.arange(n, device=a.device) // block
    a = a * st["a_scale"].double()[at].t()
    b = b * st["b_scale"].double()[at][:, bt].t()
    d = torch.mm(a, b.t())
    if st["bias_v"] is not None:
        d = d + st["bias_v"].double()
    return torch.where(d < 0, torch.zeros_like(d), d) if st["relu"] else d


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm_fwd": _exact_fwd, "norm_bwd": _exact_bwd, "quantize": _exact_quantize, "gemm": _exact_gemm}[st["op"]](st)
