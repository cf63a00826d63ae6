"""The group norm, the 4-bit quantiser and the 4-bit product together, as a residual block of 1x1 layers and a
convolution with a 4-bit filter use them, forward and backward; captured and replayed; on two streams at once; and
far past 2^31 values and bytes.  Each link is held to the 64-bit formula of what it got, with the tolerances of
tests/test_group_norm.py and tests/test_fp4.py; runs of the same calls are equal bit for bit."""
import itertools

import pytest
import torch

import conv2d_batchnorm_relu_amd as cbr
import test_fp4 as F
import test_group_norm as G

cdiv = F.cdiv


def rnd(g, *s):
    return torch.randn(*s, generator=g, device="cuda")


def quant(v, transpose=False):
    _, q, s = F.quantize(v, transpose)
    return q, s


def product(a, b, m, n, k, out, bias=None):
    d = F.product(m, n, k, a, b, out, bias)
    va, vb = F.decode64(*a, k), F.decode64(*b, k)
    want, mag = va @ vb.t(), va.abs() @ vb.abs().t()
    if bias is not None:
        want, mag = want + bias.double(), mag + bias.double().abs()
    f = torch.finfo(d.dtype)
    tol = (cdiv(k, 128) + 512 + 10) * 2.0 ** -23 * mag
    assert ((d.double() - want).abs() <= tol + f.eps / 2 * (want.abs() + tol) + f.smallest_normal * f.eps).all()
    return d


@pytest.mark.gpu
@pytest.mark.parametrize("images,h,w,c,hid,groups", [(2, 7, 7, 64, 256, 32), (3, 14, 14, 96, 136, 8), (1, 5, 9, 40, 72, 9), (2, 28, 28, 256, 128, 32)], ids=str)
@pytest.mark.parametrize("act", ["relu", "silu"])
def test_block_forward_and_backward(images, h, w, c, hid, groups, act):
    """x -> 4-bit 1x1 layer -> group norm with activation -> 4-bit 1x1 layer, and the gradients of all of it."""
    g = F.gen(images + c)
    m = images * h * w
    x = rnd(g, m, c).bfloat16()
    w1, w2 = (rnd(g, hid, c) / c ** 0.5).bfloat16(), (rnd(g, c, hid) / hid ** 0.5).bfloat16()
    qx, q1, q2 = quant(x), quant(w1), quant(w2)
    t = dict(images=images, pixels=h * w, c=hid, groups=groups, dtype="bf16", act=act, w=1 + 0.3 * rnd(g, hid), b=0.3 * rnd(g, hid))
    t["x"] = product(qx, q1, m, hid, c, "bf16", 0.1 * rnd(g, hid)).view(images, h * w, hid)
    y, st = G.forward(t)
    G.check_forward(t, y, st)
    y = y.view(m, hid)
    out = product(quant(y), q2, m, c, hid, "bf16")
    # backward: the gradient is quantised along its rows for the data gradient, along its columns for the weights'
    dout = rnd(g, m, c).bfloat16()
    dw2 = product(quant(dout, True), quant(y, True), c, hid, m, "f32")
    t["dy"] = product(quant(dout), quant(w2, True), m, hid, c, "bf16").view(images, h * w, hid)
    dx, dw, db = G.backward(t, st)
    G.check_backward(t, st, dx, dw, db)
    dz = dx.view(m, hid)
    dw1 = product(quant(dz, True), quant(x, True), hid, c, m, "f32")
    dxx = product(quant(dz), quant(w1, True), m, c, hid, "bf16")
    assert all(v.isfinite().all() for v in (out, dw1, dw2, dxx, dw, db))


@pytest.mark.gpu
def test_convolution_with_a_four_bit_filter():
    """A filter kept in 4 bits, taken out to bf16 (exact), for the library's own convolution, and a group norm of its outputs."""
    g = F.gen(3)
    n, h, w, c, k = 2, 9, 9, 64, 64
    x = rnd(g, n, h, w, c).bfloat16()
    f = (rnd(g, k, 9 * c) / (9 * c) ** 0.5).bfloat16()
    sp, q, s = F.quantize(f)
    back = F.dequantize(sp, q, s)
    assert F.same(back.double(), F.quant64(f)[0])
    y = torch.empty(n, h, w, k, dtype=torch.bfloat16, device="cuda")
    cbr.cbr_conv2d_bias(cbr.make_shape(n, h, w, c, k, 3, 3, 1, 1), x, back.contiguous(), None, y)
    xd = x.double().permute(0, 3, 1, 2).cpu()
    fd = back.double().view(k, 3, 3, c).permute(0, 3, 1, 2).cpu()
    want = torch.nn.functional.conv2d(xd, fd, padding=1)
    mag = torch.nn.functional.conv2d(xd.abs(), fd.abs(), padding=1)
    # 576 additions in fp32, then half a step of bf16
    assert ((y.double().cpu().permute(0, 3, 1, 2) - want).abs() <= 580 * 2.0 ** -24 * mag + 2.0 ** -8 * (want.abs() + 1e-4)).all()
    t = dict(images=n, pixels=h * w, c=k, groups=8, dtype="bf16", act="silu", w=None, b=None, x=y.view(n, h * w, k))
    G.check_forward(t, *G.forward(t))


class Block:
    """The block's calls on buffers of its own, as a program that captures them keeps them."""

    def __init__(self, images, pixels, c, hid, groups, seed):
        g = F.gen(seed)
        self.g, m = g, images * pixels
        E = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        U8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.x, self.dout = E(m, c), E(m, c)
        self.w1, self.w2 = (rnd(g, hid, c) / c ** 0.5).bfloat16(), (rnd(g, c, hid) / hid ** 0.5).bfloat16()
        self.gw, self.gb = 1 + 0.3 * rnd(g, hid), 0.3 * rnd(g, hid)
        self.outs, self.steps = [], []
        gn = cbr.make_group_norm_shape(images, pixels, hid, groups, cbr.CBR_BF16, cbr.CBR_ACT_SILU)
        ws = [U8(max(16, cbr.cbr_group_norm_workspace_bytes(gn, b))) for b in (False, True)]

        def q(v, turned=False):
            rows, cols = (v.shape[1], v.shape[0]) if turned else v.shape
            sp = cbr.make_fp4_shape(*v.shape, cbr.CBR_BF16, turned)
            o = torch.zeros(rows, sp.ldq, dtype=torch.uint8, device="cuda"), U8(cdiv(cols, 128), rows, 4)
            self.steps.append(lambda st: cbr.cbr_fp4_quantize(sp, v, *o, stream=st))
            self.outs += o
            return o

        def mul(a, b, m, n, k, dt=torch.bfloat16):
            d = E(m, n, dtype=dt)
            sp = cbr.make_gemm_fp4_shape(m, n, k, cbr.CBR_BF16 if dt == torch.bfloat16 else cbr.CBR_F32)
            w = U8(max(16, cbr.cbr_gemm_fp4_workspace_bytes(sp)))
            self.steps.append(lambda st: cbr.cbr_gemm_fp4(sp, *a, *b, None, d, w, stream=st))
            self.outs.append(d)
            return d
        z = mul(q(self.x), q(self.w1), m, hid, c)
        y, stats = E(m, hid), E(images, groups, 2, dtype=torch.float32)
        self.steps.append(lambda st: cbr.cbr_group_norm_forward(gn, z, self.gw, self.gb, y, stats, ws[0], stream=st))
        mul(q(y), q(self.w2), m, c, hid)
        mul(q(self.dout, True), q(y, True), c, hid, m, torch.float32)
        dy = mul(q(self.dout), q(self.w2, True), m, hid, c)
        dz, dw, db = E(m, hid), E(hid, dtype=torch.float32), E(hid, dtype=torch.float32)
        self.steps.append(lambda st: cbr.cbr_group_norm_backward(gn, dy, z, self.gw, self.gb, stats, dz, dw, db, ws[1], stream=st))
        mul(q(dz, True), q(self.x, True), hid, c, m, torch.float32)
        mul(q(dz), q(self.w1, True), m, c, hid)
        self.outs += [y, stats, dz, dw, db]

    def feed(self):
        self.x.copy_(rnd(self.g, *self.x.shape))
        self.dout.copy_(rnd(self.g, *self.x.shape))

    def run(self, stream=None):
        for s in self.steps:
            s(stream)

    def wipe(self):
        for o in self.outs:
            o.view(torch.uint8).fill_(0xFF) if o.dtype != torch.uint8 else o.zero_()

    def results(self):
        return [o.clone() for o in self.outs]


def equal(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b, strict=True))


BLOCKS = [(2, 49, 64, 256, 32), (1, 5000, 64, 128, 8), (3, 35, 40, 72, 9)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", BLOCKS, ids=str)
def test_replayed_from_a_graph(size):
    """Two graphs of the block, each with its own workspaces, replayed in turn on new inputs with the eager calls between."""
    blocks = [Block(*size, seed) for seed in (1, 2)]
    graphs = []
    for b in blocks:
        b.feed()
        b.run()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            b.run()
        graphs.append(gr)
    for _ in range(4):
        for b, gr in zip(blocks, graphs):
            b.feed()
            b.run()
            torch.cuda.synchronize()
            want = b.results()
            b.wipe()
            gr.replay()
            torch.cuda.synchronize()
            assert equal(b.results(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("size", BLOCKS, ids=str)
def test_two_streams_at_once(size):
    blocks = [Block(*size, seed) for seed in (3, 4)]
    wants = []
    for b in blocks:
        b.feed()
        b.run()
        wants.append(b.results())
        b.wipe()
    streams = [torch.cuda.Stream() for _ in blocks]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for k in range(len(blocks[0].steps)):
            for b, s in zip(blocks, streams):
                b.steps[k](s)
    torch.cuda.synchronize()
    for b, want in zip(blocks, wants):
        assert equal(b.results(), want)


# ---------------------------------------------------------------- past 2^31 values
PERIOD = 7


def repeats(v, base):
    """Every slice i of v equals slice i % PERIOD of base, bit for bit."""
    full = v.shape[0] // PERIOD * PERIOD
    return bool((v[:full].view(-1, PERIOD, *v.shape[1:]) == base).all()) and torch.equal(v[full:], base[:v.shape[0] - full])


@pytest.mark.gpu
@pytest.mark.parametrize("images,pixels,c,groups", [(86005, 49, 512, 32), (22005, 49, 2001, 3), (170, 50176, 256, 32)], ids=str)
def test_group_norm_past_31_bits(images, pixels, c, groups):
    assert images * pixels * c > 2 ** 31
    small = G.make(PERIOD, pixels, c, groups, "bf16", "silu", 5)
    reps = cdiv(images, PERIOD)
    big = dict(small, images=images)
    for k in ("x", "dy"):
        big[k] = small[k].repeat(reps, 1, 1)[:images].contiguous()
    y, st = G.forward(big)
    G.check_forward(small, y[:PERIOD], st[:PERIOD])
    assert repeats(y, y[:PERIOD]) and repeats(st, st[:PERIOD])
    del y
    dx, dw, db = G.backward(big, st)
    G.check_backward(small, st[:PERIOD], dx[:PERIOD], None, None)
    assert repeats(dx, dx[:PERIOD])
    del dx
    # the sums over all images: each base image's as often as it repeats; an image's own are within its part of the
    # tolerance of tests/test_group_norm.py, and the sum over the images is in fp64
    count = torch.tensor([cdiv(images - i, PERIOD) for i in range(PERIOD)], dtype=torch.float64, device="cuda")
    wb, bb, tw, tb = 0, 0, 0, 0
    for i in range(PERIOD):
        one = dict(small, images=1, x=small["x"][i:i + 1], dy=small["dy"][i:i + 1])
        s1 = st[i:i + 1]
        _, w1, b1, (_, _, _, xh, _), mw, mb, u = G.gradients64(one, s1)
        dg = one["dy"].double().abs() * (3.3 * G.U * (xh * one["w"].abs() + one["b"].abs()) + (3 * u.abs() + 24) * G.U)
        wb, bb = wb + count[i] * w1, bb + count[i] * b1
        add = G.longest(pixels) + 8
        tw = tw + count[i] * ((dg * xh).sum((0, 1)) + add * G.U * mw)
        tb = tb + count[i] * (dg.sum((0, 1)) + add * G.U * mb)
    assert ((dw.double() - wb).abs() <= tw + G.U * wb.abs()).all()
    assert ((db.double() - bb).abs() <= tb + G.U * bb.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("turned", [False, True])
def test_quantiser_past_31_bits(turned):
    rows, cols = 70001, 32770
    base = rnd(F.gen(6), PERIOD, cols).bfloat16()
    want, _ = F.quant64(base)
    v = base.repeat(cdiv(rows, PERIOD), 1)[:rows]
    v = v.t().contiguous() if turned else v.contiguous()
    assert v.numel() > 2 ** 31
    sp = cbr.make_fp4_shape(*v.shape, cbr.CBR_BF16, turned)
    q = torch.zeros(rows, sp.ldq, dtype=torch.uint8, device="cuda")
    s = torch.zeros(cdiv(cols, 128), rows, 4, dtype=torch.uint8, device="cuda")
    cbr.cbr_fp4_quantize(sp, v, q, s)
    del v
    assert F.same(F.decode64(q[:PERIOD], s[:, :PERIOD], cols), want)
    assert repeats(q, q[:PERIOD]) and repeats(s.transpose(0, 1).contiguous(), s[:, :PERIOD].transpose(0, 1))
    back = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    cbr.cbr_fp4_dequantize(sp, q, s, back)
    assert F.same(back[:PERIOD].double(), want) and repeats(back, back[:PERIOD])


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(280009, 8200, 64), (600005, 24, 8192), (5, 600005, 8192), (80, 600005, 8192)], ids=str)
def test_product_past_31_bits(m, n, k):
    long_a = m > n
    rows = max(m, n)
    qb, sb = F.operand(PERIOD, k, 7, 1)
    big = qb.repeat(cdiv(rows, PERIOD), 1)[:rows].contiguous(), sb.repeat(1, cdiv(rows, PERIOD), 1)[:, :rows].contiguous()
    other = F.operand(min(m, n), k, 8, 1)
    a, b = (big, other) if long_a else (other, big)
    sp = cbr.make_gemm_fp4_shape(m, n, k, cbr.CBR_BF16, lda=a[0].shape[1], ldb=b[0].shape[1])
    need = cbr.cbr_gemm_fp4_workspace_bytes(sp)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    d = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert max(d.numel(), big[0].numel()) > 2 ** 31
    cbr.cbr_gemm_fp4(sp, *a, *b, None, d, ws)
    if not long_a:
        d = d.t().contiguous()
    assert repeats(d, d[:PERIOD])
    vb, vo = F.decode64(qb, sb, k), F.decode64(*other, k)
    want, mag = vb @ vo.t(), vb.abs() @ vo.abs().t()
    tol = (cdiv(k, 128) + 512 + 10) * 2.0 ** -23 * mag
    assert ((d[:PERIOD].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()


# ---------------------------------------------------------------- layouts of many sizes, on the CPU
def test_workspaces_of_many_sizes():
    """Every legal size has a layout: a workspace within a small multiple of the data, and asking does not end the process."""
    sizes = (1, 2, 3, 7, 8, 31, 33, 100, 256, 1000, 4097, 65537, 1000003)
    for p, c, n in itertools.product(sizes, sizes[:11], (1, 2, 17, 300, 70001)):
        for groups in {1, c, 2 if c % 2 == 0 else 1, c // 8 if c % 8 == 0 else 1}:
            if c // groups > 8192 or n * p * c > 2 ** 46:
                continue
            for dt, back in itertools.product((cbr.CBR_BF16, cbr.CBR_F32), (False, True)):
                need = cbr.cbr_group_norm_workspace_bytes(cbr.make_group_norm_shape(n, p, c, groups, dt, cbr.CBR_ACT_SILU), back)
                assert 0 <= need <= 16 * n * p * c + 64 * (1024 * c + n * groups) + (1 << 20)
    for m, n, k in itertools.product(sizes + (1 << 20,), sizes + (1 << 22,), sizes[:11] + (1 << 23,)):
        need = cbr.cbr_gemm_fp4_workspace_bytes(cbr.make_gemm_fp4_shape(m, min(n, 1 << 22), k))
        assert 0 <= need <= 512 * 4 * max(m * n, 256 * 256)
