"""Group norm with an activation over channels-last maps, and 4-bit operands with shared exponents: cases, inputs, plain forms
and exact values.

A case names its operator ("op") and plain sizes.  ``run`` with ``own`` false computes the operator with elementary torch
operations in 32 bits; with ``own`` true it makes the library's calls.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
GROUP = 32                                                      # values that share an exponent
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)                # what a 4-bit value stands for; bit 3 is the sign
EPS = 1e-5


# ------------------------------------------------------------------------------- cases
def _norm(name, op, images, pixels, c, groups, dtype, act):
    return dict(name=name, op=op, images=images, pixels=pixels, c=c, groups=groups, type=dtype, act=act)


def _quant(name, rows, cols, src, transpose):
    return dict(name=name, op="quantize", rows=rows, cols=cols, src=src, transpose=transpose)


def _gemm(name, m, n, k, out, bias, relu):
    return dict(name=name, op="gemm", m=m, n=n, k=k, out=out, bias=bias, relu=relu)


# ReLU's gradient jumps where its argument passes 0, and rounding decides on which side a value near it lies: the measured
# backward cases are the smooth ones.
def listed():
    return [
        # One image's 7x7 map in inference: a call that latency decides.
        _norm("gn_fwd_7x7x512", "gn_fwd", 1, 49, 512, 32, "bf16", "relu"),
        # Odd channel and group counts on a small single precision batch.
        _norm("gn_fwd_odd_1001", "gn_fwd", 16, 225, 1001, 7, "f32", "silu"),
        # The 28x28 stage of a 256-image training batch.
        _norm("gn_fwd_28x28x512", "gn_fwd", 256, 784, 512, 32, "bf16", "relu"),
        # The backward of one image's 14x14 map: launches and the small reductions.
        _norm("gn_bwd_14x14x256", "gn_bwd", 1, 196, 256, 32, "bf16", "silu"),
        # The 56x56 stage of a 64-image training batch.
        _norm("gn_bwd_56x56x256", "gn_bwd", 64, 3136, 256, 32, "bf16", "silu"),
        # Few large images in single precision: the first stage at 224x224, where one group's map is 400 KB.
        _norm("gn_bwd_224x224x64", "gn_bwd", 8, 50176, 64, 32, "f32", "silu"),
        # A small batch's features on their way into a product.
        _quant("quant_rows_64x2048", 64, 2048, "bf16", False),
        # The 14x14 stage's activations turned over for the weight gradient.
        _quant("quant_turned_50176x1024", 50176, 1024, "bf16", True),
        # One image's features into 1000 classes.
        _gemm("gemm_classes_1x1000x2048", 1, 1000, 2048, "f32", True, False),
        # A 1x1 layer of the 14x14 stage, 256 images less a few, bias and ReLU.
        _gemm("gemm_1x1_50001x256x1024", 50001, 256, 1024, "bf16", True, True),
        # The same layer's weight gradient: a long sum over pixels, few outputs.
        _gemm("gemm_wgrad_1024x256x50176", 1024, 256, 50176, "f32", False, False),
        # A large square product: the card's rate.
        _gemm("gemm_square_8192", 8192, 8192, 8192, "bf16", False, False),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("gn_fwd", "gn_bwd", "quantize", "gemm"))
    if kind.startswith("gn"):
        groups = rng.choice((1, 2, 4, 7, 8, 16, 32, 32, 32))
        each = _logint(rng, 1, 2048 // groups)
        if rng.random() < 0.5:
            each = max(8, each // 8 * 8)
        c = groups * each
        pixels = _logint(rng, max(1, -(-64 // each)), 50176)   # 64 values a group: fewer leave no gradient but rounding
        images = _logint(rng, 1, max(1, min(256, 25_000_000 // (pixels * c))))
        pixels = min(pixels, max(-(-64 // each), 25_000_000 // c))
        return dict(op=kind, images=images, pixels=pixels, c=c, groups=groups, type=rng.choice(("bf16", "bf16", "f16", "f32")),
                    act=rng.choice(("none", "silu", "relu" if kind == "gn_fwd" else "silu")))
    if kind == "quantize":
        cols = _logint(rng, 33, 8192)
        rows = _logint(rng, 1, min(65536, 50_000_000 // cols))
        return dict(op=kind, rows=rows, cols=cols, src=rng.choice(("bf16", "f16", "f32")), transpose=rng.random() < 0.5)
    m, n, k = _logint(rng, 1, 65536), _logint(rng, 16, 8192), _logint(rng, 32, 8192)
    if rng.random() < 0.5:
        n, k = max(16, n // 16 * 16), max(64, k // 64 * 64)
    m = max(1, min(m, 67_000_000 // max(n, k), 2 ** 39 // (n * k)))
    if rng.random() < 0.2:   # a weight gradient's shape: the long axis is summed over
        m, k = max(16, k // 4), max(m, 64)
    return dict(op=kind, m=m, n=n, k=k, out=rng.choice(("bf16", "f16", "f32")), bias=rng.random() < 0.5, relu=rng.random() < 0.3)


def _cdiv(a, b):
    return -(-a // b)


def work(case):
    op = case["op"]
    if op.startswith("gn"):
        n, s = case["images"] * case["pixels"] * case["c"], SIZE[case["type"]]
        small = 8 * case["images"] * case["groups"] + 16 * case["c"]
        if op == "gn_fwd":   # x in, y out
            return {"bytes": 2 * n * s + small, "flops": 10 * n}
        return {"bytes": 3 * n * s + small, "flops": 25 * n}   # dy, x in, dx out
    if op == "quantize":     # there and back: src in, its 4-bit form out and in, the values out
        n, s = case["rows"] * case["cols"], SIZE[case["src"]]
        return {"bytes": 2 * n * s + n + n // 16, "flops": 4 * n}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": (m + n) * (k // 2 + k // 32) + m * n * SIZE[case["out"]] + 4 * n * case["bias"], "flops": 2 * m * n * k}


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _groups_of(v):
    """v [rows, k] as [rows, groups, 32], zeros behind k."""
    rows, k = v.shape
    p = torch.zeros(rows, _cdiv(k, GROUP) * GROUP, device=v.device)
    p[:, :k] = v
    return p.view(rows, -1, GROUP)


def _rounded(v):
    """v [rows, k] to 4-bit values and the exponents of its groups of 32: (values over the scale [rows, groups, 32], exponent
    [rows, groups]).  The scale is the power of two that brings a group's largest value to 4 .. 8; above 6 is 6."""
    p = _groups_of(v)
    amax = p.abs().amax(2)
    e = (torch.frexp(amax).exponent - 3).clamp_min(-127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    t = torch.ldexp(p, -e[:, :, None])
    a = t.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return ((a / step).round() * step).clamp_max(6.0) * torch.where(t < 0, -1.0, 1.0), e


def _scales(e):
    """Exponents [rows, groups] as scales [k / 128, rows, 4], 1 behind the last group."""
    rows, groups = e.shape
    s = torch.ones(rows, _cdiv(groups, 4) * 4, device=e.device)
    s[:, :groups] = torch.ldexp(torch.ones_like(s[:, :groups]), e)
    return s.view(rows, -1, 4).transpose(0, 1).contiguous().to(torch.float8_e8m0fnu)


def _encode(v):
    """Operand v as a program holds it: two values a byte, the lower four bits first, and its scales."""
    q, e = _rounded(v)
    a = q.abs()
    code = ((a > 0.25).int() + (a > 0.75) + (a > 1.25) + (a > 1.75) + (a > 2.5) + (a > 3.5) + (a > 5) + 8 * (q < 0)).to(torch.uint8)
    code = code.view(v.shape[0], -1)
    return code[:, ::2] | code[:, 1::2] << 4, _scales(e)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"].startswith("gn"):
        shape, t, c = (case["images"], case["pixels"], case["c"]), TYPES[case["type"]], case["c"]
        x = _randn(g, *shape) * torch.exp(0.3 * _randn(g, c)) + 0.5 * _randn(g, c)
        st["x"] = x.to(t)
        st["w"] = 1.0 + 0.2 * _randn(g, c)
        st["b"] = 0.2 * _randn(g, c)
        if case["op"] == "gn_bwd":
            st["dy"] = (0.1 * _randn(g, *shape)).to(t)
            st["stats"] = _stats64(st["x"].double(), case["groups"])[0].float()
        return st
    if case["op"] == "quantize":
        v = _randn(g, case["rows"], case["cols"])
        st["src"] = (v * torch.exp(0.5 * _randn(g, 1, case["cols"]))).to(TYPES[case["src"]])
        return st
    m, n, k = case["m"], case["n"], case["k"]
    st["a_q"], st["a_scale"] = _encode(_randn(g, m, k).clamp_min(-0.5))
    st["b_q"], st["b_scale"] = _encode(_randn(g, n, k) * (2.0 / k) ** 0.5)
    st["bias_v"] = 0.1 * _randn(g, n) if case["bias"] else None
    return st


# ------------------------------------------------------------------------- plain forms
def _normalised(x, groups):
    """[images, pixels, groups, channels of a group]: the normalised values, and (mean, 1/std) [images, groups, 2]."""
    v = x.float().view(x.shape[0], x.shape[1], groups, -1)
    mean = v.mean((1, 3), keepdim=True)
    d = v - mean
    inv = torch.rsqrt((d * d).mean((1, 3), keepdim=True) + EPS)
    return d * inv, torch.stack((mean[:, 0, :, 0], inv[:, 0, :, 0]), 2)


def _plain_gn_fwd(st):
    x = st["x"]
    v, stats = _normalised(x, st["groups"])
    u = v.view(x.shape) * st["w"] + st["b"]
    if st["act"] == "relu":
        u = u.clamp_min(0.0)
    elif st["act"] == "silu":
        u = u / (1.0 + torch.exp(-u))
    return {"y": u.to(x.dtype), "stats": stats}


def _plain_gn_bwd(st):
    x, groups = st["x"], st["groups"]
    split = (x.shape[0], x.shape[1], groups, -1)
    mean, inv = (st["stats"][:, :, i][:, None, :, None] for i in (0, 1))
    v = (x.float().view(split) - mean) * inv
    g = st["dy"].float()
    if st["act"] == "silu":
        u = v.view(x.shape) * st["w"] + st["b"]
        s = 1.0 / (1.0 + torch.exp(-u))
        g = g * (s * (1.0 + u * (1.0 - s)))
    out = {"dw": (g * v.view(x.shape)).sum((0, 1)), "db": g.sum((0, 1))}
    t = (g * st["w"]).view(split)
    dx = (t - t.mean((1, 3), keepdim=True) - v * (t * v).mean((1, 3), keepdim=True)) * inv
    out["dx"] = dx.view(x.shape).to(x.dtype)
    return out


def _plain_quantize(st):
    v = st["src"].float()
    v = v.t().contiguous() if st["transpose"] else v
    q, e = _rounded(v)
    values = torch.ldexp(q, e[:, :, None]).view(v.shape[0], -1)[:, :v.shape[1]]
    return {"values": values.to(st["src"].dtype).contiguous(), "scale": _scales(e)}


def _values(q, scale, k):
    """What a 4-bit operand stands for, in 32 bits."""
    lut = torch.tensor(CODES + tuple(-c for c in CODES), device=q.device)
    v = torch.stack((lut[(q & 15).int()], lut[(q >> 4).int()]), 2).view(q.shape[0], -1)
    s = scale.float().transpose(0, 1).reshape(q.shape[0], -1)[:, :v.shape[1] // GROUP]
    return (v.view(q.shape[0], -1, GROUP) * s[:, :, None]).view(q.shape[0], -1)[:, :k]


def _plain_gemm(st):
    d = _values(st["a_q"], st["a_scale"], st["k"]) @ _values(st["b_q"], st["b_scale"], st["k"]).t()
    if st["bias_v"] is not None:
        d = d + st["bias_v"]
    if st["relu"]:
        d = d.clamp_min(0.0)
    return d.to(TYPES[st["out"]])


# --------------------------------------------------------------------- the library's calls
def _dtypes(cbr):
    return {"bf16": cbr.CBR_BF16, "f16": cbr.CBR_F16, "f32": cbr.CBR_F32}


def _own_gn(cbr, st):
    x = st["x"]
    if "sp" not in st:
        act = {"none": cbr.CBR_ACT_NONE, "relu": cbr.CBR_ACT_RELU, "silu": cbr.CBR_ACT_SILU}[st["act"]]
        st["sp"] = cbr.make_group_norm_shape(st["images"], st["pixels"], st["c"], st["groups"], dtype=_dtypes(cbr)[st["type"]],
                                             act=act, eps=EPS)
        need = cbr.cbr_group_norm_workspace_bytes(st["sp"], backward=st["op"] == "gn_bwd")
        st["ws"] = torch.empty(max(256, need), dtype=torch.uint8, device=x.device)
    if st["op"] == "gn_fwd":
        y = torch.empty_like(x)
        stats = torch.empty(st["images"], st["groups"], 2, device=x.device)
        cbr.cbr_group_norm_forward(st["sp"], x, st["w"], st["b"], y, stats, st["ws"])
        return {"y": y, "stats": stats}
    dx, dw, db = torch.empty_like(x), torch.empty_like(st["w"]), torch.empty_like(st["b"])
    cbr.cbr_group_norm_backward(st["sp"], st["dy"], x, st["w"], st["b"], st["stats"], dx, dw, db, st["ws"])
    return {"dw": dw, "db": db, "dx": dx}


def _own_quantize(cbr, st):
    src = st["src"]
    if "sp" not in st:
        st["sp"] = cbr.make_fp4_shape(st["rows"], st["cols"], dtype=_dtypes(cbr)[{v: k for k, v in TYPES.items()}[src.dtype]], transpose=st["transpose"])
    sp = st["sp"]
    rows, cols = (st["cols"], st["rows"]) if st["transpose"] else (st["rows"], st["cols"])
    q = torch.empty(rows, sp.ldq, dtype=torch.uint8, device=src.device)
    scale = torch.empty(_cdiv(cols, 128), rows, 4, dtype=torch.float8_e8m0fnu, device=src.device)
    cbr.cbr_fp4_quantize(sp, src, q, scale)
    values = torch.empty(rows, cols, dtype=src.dtype, device=src.device)
    cbr.cbr_fp4_dequantize(sp, q, scale, values)
    return {"values": values, "scale": scale}


def _own_gemm(cbr, st):
    if "sp" not in st:
        st["sp"] = cbr.make_gemm_fp4_shape(st["m"], st["n"], st["k"], d_type=_dtypes(cbr)[st["out"]], relu=st["relu"])
        st["ws"] = torch.empty(max(256, cbr.cbr_gemm_fp4_workspace_bytes(st["sp"])), dtype=torch.uint8, device="cuda")
    d = torch.empty(st["m"], st["n"], dtype=TYPES[st["out"]], device="cuda")
    cbr.cbr_gemm_fp4(st["sp"], st["a_q"], st["a_scale"], st["b_q"], st["b_scale"], st["bias_v"], d, st["ws"])
    return d


def run(state):
    op = state["op"]
    if own:
        import conv2d_batchnorm_relu_amd as cbr
        return (_own_gemm if op == "gemm" else _own_quantize if op == "quantize" else _own_gn)(cbr, state)
    return {"gn_fwd": _plain_gn_fwd, "gn_bwd": _plain_gn_bwd, "quantize": _plain_quantize, "gemm": _plain_gemm}[op](state)


# ------------------------------------------------------------------------------- exact
def _stats64(x, groups):
    """(mean, 1/std) [images, groups, 2] in 64 bits, and the normalised values."""
    v = x.view(x.shape[0], x.shape[1], groups, -1).transpose(1, 2).reshape(x.shape[0], groups, -1)
    var, mean = torch.var_mean(v, 2, correction=0)
    stats = torch.stack((mean, (var + EPS) ** -0.5), 2)
    n = ((v - mean[:, :, None]) * stats[:, :, 1:]).view(x.shape[0], groups, x.shape[1], -1).transpose(1, 2)
    return stats, n.reshape(x.shape)


def _exact_gn(x, w, b, groups, act):
    stats, n = _stats64(x, groups)
    u = torch.addcmul(b, n, w)
    y = torch.maximum(u, torch.zeros_like(u)) if act == "relu" else u * torch.sigmoid(u) if act == "silu" else u
    return {"y": y, "stats": stats}


def _exact_quantize(st):
    v = st["src"].double()
    v = v.t().contiguous() if st["transpose"] else v
    rows, k = v.shape
    blocks = torch.nn.functional.pad(v, (0, -k % GROUP)).view(rows, -1, GROUP)
    top = blocks.abs().max(2).values
    scale = torch.exp2(torch.floor(torch.log2(top.clamp_min(2.0 ** -149))) - 2).clamp_min(2.0 ** -127)   # (a group of zeros: 2^-127)
    codes = torch.tensor(CODES, dtype=torch.float64, device=v.device)
    mid = (codes[1:] + codes[:-1]) / 2                  # ties go to the even code: 0, 1, 2, 4
    t = (blocks.abs() / scale[:, :, None]).contiguous()
    up, down = torch.bucketize(t, mid, right=True), torch.bucketize(t, mid)
    near = codes[torch.where(up % 2 == 0, up, down)]
    values = (near * torch.sign(blocks) * scale[:, :, None]).view(rows, -1)[:, :k]
    s = torch.ones(rows, _cdiv(k, 128) * 4, dtype=torch.float64, device=v.device)
    s[:, :scale.shape[1]] = scale
    return {"values": values, "scale": s.view(rows, -1, 4).permute(1, 0, 2)}


def _exact_operand(q, scale, k):
    """The values by their bits: sign, two of the exponent, one of the mantissa."""
    c = torch.stack((q & 15, q >> 4), 2).view(q.shape[0], -1)[:, :k]
    e, m = ((c >> 1) & 3).double(), (c & 1).double()
    v = torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2) * torch.where(c > 7, -1.0, 1.0)
    t = torch.arange(k, device=q.device) // GROUP
    return v * torch.exp2(scale.view(torch.uint8).double() - 127).permute(1, 0, 2).reshape(q.shape[0], -1)[:, t]


def _exact_gemm(st):
    d = torch.mm(_exact_operand(st["a_q"], st["a_scale"], st["k"]), _exact_operand(st["b_q"], st["b_scale"], st["k"]).t())
    if st["bias_v"] is not None:
        d = d + st["bias_v"].double()
    return torch.where(d < 0, torch.zeros_like(d), d) if st["relu"] else d


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "gemm":
        return _exact_gemm(st)
    if op == "quantize":
        return _exact_quantize(st)
    x, w, b = (st[k].double() for k in ("x", "w", "b"))
    if op == "gn_fwd":
        return _exact_gn(x, w, b, st["groups"], st["act"])
    x, w, b = (t.requires_grad_() for t in (x, w, b))   # gradients by automatic differentiation of the definition
    dx, dw, db = torch.autograd.grad(_exact_gn(x, w, b, st["groups"], st["act"])["y"], (x, w, b), st["dy"].double())
    return {"dw": dw, "db": db, "dx": dx}
