"""The block norm, the quantiser and the 8-bit product together, as a residual block of two 1x1
layers on NHWC activations uses them, forward and backward, beside the library's own bf16
convolution.  Each stage is held to the 64-bit formula of its inputs as the stage got them.

Tolerance of a product of quantised operands against the product of the values they came
from: a value moves by at most half an 8-bit step, 2^-4 of it (e4m3; e5m2: 2^-3) or, where the
group's scale makes it subnormal, half the smallest step (2^-10; 2^-17) times the scale; so a
product of sums moves by at most (|a| + da)(|b| + db) - |a||b|.  The arithmetic's own part
(tests/test_fp8.py) is 8 * 2^-13 + 2^-15 of the magnitudes, and half a step of the output."""
import pytest
import torch

import conv2d_batchnorm_relu_amd as cbr
import test_block_norm as B

pytestmark = pytest.mark.gpu

F8 = {cbr.CBR_E4M3: (torch.float8_e4m3fn, 2.0 ** -4, 2.0 ** -10), cbr.CBR_E5M2: (torch.float8_e5m2, 2.0 ** -3, 2.0 ** -17)}


def quant(v, fmt=cbr.CBR_E4M3, transpose=False, block=1):
    sp = cbr.make_quant_shape(*v.shape, cbr.CBR_BF16, fmt, transpose, block)
    rows, cols = v.shape[::-1] if transpose else v.shape
    q = torch.empty(rows, sp.ldq, dtype=torch.uint8, device=v.device)
    s = torch.empty(-(-cols // 128), -(-rows // block), device=v.device)
    cbr.cbr_fp8_quantize(sp, v, q, s)
    w = (v.t() if transpose else v).double()
    each = s.double().t().repeat_interleave(block, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return q, s, w, torch.maximum(F8[fmt][1] * w.abs(), F8[fmt][2] * each), fmt


def product(a, b, b_block, out=torch.bfloat16, bias=None, relu=False):
    qa, sa, va, da, fa = a
    qb, sb, vb, db, fb = b
    m, n, k = va.shape[0], vb.shape[0], va.shape[1]
    dt = {torch.bfloat16: cbr.CBR_BF16, torch.float32: cbr.CBR_F32}[out]
    sp = cbr.make_gemm_shape(m, n, k, fa, fb, dt, b_block, relu)
    ws = torch.empty(max(16, cbr.cbr_gemm_fp8_workspace_bytes(sp)), dtype=torch.uint8, device=qa.device)
    d = torch.empty(m, n, dtype=out, device=qa.device)
    cbr.cbr_gemm_fp8(sp, qa, sa, qb, sb, bias, d, ws)
    want = va @ vb.t()
    mag = (va.abs() + da) @ (vb.abs() + db).t()
    tol = mag - va.abs() @ vb.abs().t() + (8 * 2.0 ** -13 + 2.0 ** -15) * mag
    if bias is not None:
        want = want + bias.double()
    if relu:
        want = want.clamp_min(0)
    tol = tol + (torch.finfo(out).eps / 2) * (want.abs() + tol)
    assert ((d.double() - want).abs() <= tol).all()
    assert (d.double() - want).norm() <= 0.1 * want.norm()    # rounding is not one-sided: far inside the bound
    return d


def conv1x1(x, w, bias, images, h, wd):
    y = torch.empty(x.shape[0], w.shape[0], dtype=torch.bfloat16, device=x.device)
    cbr.cbr_conv2d_bias_relu(cbr.make_shape(images, h, wd, x.shape[1], w.shape[0], 1, 1), x, w, bias, y)
    return y


@pytest.mark.parametrize("images,h,w,c,hid,stream", [(2, 7, 7, 64, 256, "bf16"), (3, 14, 14, 96, 136, "f32"),
                                                     (1, 1, 1, 256, 512, "bf16")], ids=str)
def test_residual_block(images, h, w, c, hid, stream):
    rows = images * h * w
    t = B.make(rows, c, stream, "bf16", "layer", "rms", h * w, 21)
    first = {**t, "f": None, "post": "none", "gate": None, "rpg": 0, "res_scale": None, "post_w": None, "post_b": None}
    g = torch.Generator(device="cuda").manual_seed(3)
    w1 = (torch.randn(hid, c, generator=g, device="cuda") * (2 / c) ** 0.5).bfloat16()
    w2 = (torch.randn(c, hid, generator=g, device="cuda") * (2 / hid) ** 0.5).bfloat16()
    b1 = 0.1 * torch.randn(hid, generator=g, device="cuda")

    # forward: norm, two 1x1 layers in 8 bits, norm + gate + residual + norm of the next block
    o1 = B.run_forward(first)
    B.check_forward(first, o1)
    a = product(quant(o1["h"]), quant(w1, block=128), 128, bias=b1, relu=True)
    f = product(quant(a), quant(w2, block=128), 128)
    second = {**t, "f": f}
    o2 = B.run_forward(second)
    B.check_forward(second, o2)
    # the same layer as the library's convolution runs it in bf16: apart by the quantisation only
    ref = conv1x1(o1["h"], w1, b1, images, h, w)
    assert (a.double() - ref.double()).norm() <= 0.1 * ref.double().norm()

    # backward
    g2 = B.run_backward(second, o2)
    B.check_backward(second, o2, g2)
    df = g2["df"]
    E5 = cbr.CBR_E5M2
    da = product(quant(df, E5), quant(w2, transpose=True, block=128), 128)
    dw2 = product(quant(df, E5, transpose=True), quant(a, transpose=True), 1, out=torch.float32)
    da = torch.where(a > 0, da, torch.zeros_like(da))
    dh = product(quant(da, E5), quant(w1, transpose=True, block=128), 128)
    dw1 = product(quant(da, E5, transpose=True), quant(o1["h"], transpose=True), 1, out=torch.float32)
    back = {**first, "dy": g2["dx"], "dh": dh}
    g1 = B.run_backward(back, o1)
    B.check_backward(back, o1, g1)
    assert dw1.shape == w1.shape and dw2.shape == w2.shape and dw1.isfinite().all() and dw2.isfinite().all()


def test_block_in_a_graph_between_convolutions():
    """Captured with the library's convolution, replayed on new inputs with eager work between."""
    images, h, w, c = 2, 14, 14, 64
    rows = images * h * w
    t = B.make(rows, c, "bf16", "bf16", "rms", "layer", h * w, 31)
    wq = (torch.randn(c, c, device="cuda") * 0.2).bfloat16()
    qw = quant(wq, block=128)
    bias = torch.zeros(c, device="cuda")
    sp = cbr.make_quant_shape(rows, c)
    gp = cbr.make_gemm_shape(rows, c, c, relu=True)
    assert cbr.cbr_gemm_fp8_workspace_bytes(gp) == 0

    def step():
        o = B.run_forward(t)
        q = torch.empty(rows, sp.ldq, dtype=torch.uint8, device="cuda")
        s = torch.empty(1, rows, device="cuda")
        cbr.cbr_fp8_quantize(sp, o["h"], q, s)
        d = torch.empty(rows, c, dtype=torch.bfloat16, device="cuda")
        cbr.cbr_gemm_fp8(gp, q, s, qw[0], qw[1], bias, d)
        return o["y"], q, d, conv1x1(d, wq, bias, images, h, w)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (32, 33, 34):
        new = B.make(rows, c, "bf16", "bf16", "rms", "layer", h * w, seed)
        for k in ("x", "f", "gate"):
            t[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
