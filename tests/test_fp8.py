"""The 8-bit quantiser and the 8-bit matrix product against their definitions in 64 bits, and
their refusals.

The quantiser is compared value for value: v fmax / a, rounded to nearest even, is computed
from exact products in 64 bits.  Tolerance of the product: fp32 sums of 128 products, then of
the blocks (and of splits), so at most 128 + blocks + 16 roundings of 2^-24 each, of the sum
of magnitudes; then half a step of the output's type.  For 16-bit outputs the
8-bit matrix instruction adds: of each eight consecutive products it keeps multiples
of 2^-13 times the power of two at or below the largest (a product of 2^-13 times the largest
is kept, one of 2^-14 is lost), so a product loses less than 2^-13 times the largest of its
eight, and the eight lose less than 8 * 2^-13 times it; the largest product is at most the
product of the eights' largest operands.  Small whole numbers with power-of-two
scales are exact in fp32 and have to come out equal."""
import ctypes

import pytest
import torch

import conv2d_batchnorm_relu_amd as cbr

U = 2.0 ** -24
F8 = {"e4m3": (torch.float8_e4m3fn, cbr.CBR_E4M3, 448.0, 3, -6), "e5m2": (torch.float8_e5m2, cbr.CBR_E5M2, 57344.0, 2, -14)}
DT = {"bf16": (torch.bfloat16, cbr.CBR_BF16), "f16": (torch.float16, cbr.CBR_F16), "f32": (torch.float32, cbr.CBR_F32)}


def cdiv(a, b):
    return -(-a // b)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# --------------------------------------------------------------------------- quantiser
def quant64(v, fmt, block):
    """(q values, scale [k blocks, row blocks]) of v [rows, k] in 64 bits.  A group with an
    infinity has scale infinity, its finite values 0 and its infinities NaN."""
    _, _, fmax, bits, low = F8[fmt]
    rows, k = v.shape
    p = torch.zeros(cdiv(rows, block) * block, cdiv(k, 128) * 128, dtype=torch.float64, device=v.device)
    p[:rows, :k] = v.double()
    p = p.view(p.shape[0] // block, block, -1, 128)
    a = p.abs().amax((1, 3)).clamp_min(fmax * 2.0 ** -126)
    t = p * fmax / a[:, None, :, None]      # v * fmax is exact, the quotient rounded once in 64 bits
    step = torch.exp2((torch.frexp(t).exponent - 1).clamp_min(low).double() - bits)
    q = (torch.round(t / step) * step).view(p.shape[0] * block, -1)[:rows, :k]
    return q, (a / fmax).t()


def same(x, y):
    return x.shape == y.shape and bool(((x == y) | (x.isnan() & y.isnan())).all())


def scale_close(s, ws):
    return bool(((s.double() == ws) | ((s.double() - ws).abs() <= U * ws)).all())


def quantize(src, fmt, transpose=False, block=1, ldq=None, fill=0xA5):
    rows, cols = (src.shape[1], src.shape[0]) if transpose else src.shape
    st = {torch.bfloat16: cbr.CBR_BF16, torch.float16: cbr.CBR_F16, torch.float32: cbr.CBR_F32}[src.dtype]
    sp = cbr.make_quant_shape(src.shape[0], src.shape[1], st, F8[fmt][1], transpose, block, ldq)
    q = torch.full((rows, sp.ldq), fill, dtype=torch.uint8, device=src.device)
    s = torch.full((cdiv(cols, 128), cdiv(rows, block)), -1.0, device=src.device)
    cbr.cbr_fp8_quantize(sp, src, q, s)
    assert (q[:, cols:] == fill).all()       # what lies past a row stays as it was
    return q, q[:, :cols].contiguous().view(F8[fmt][0]).double(), s


QSIZES = [(1, 1), (1, 128), (3, 130), (17, 8), (64, 256), (100, 1000), (129, 127), (257, 384), (130, 67), (5, 4099), (300, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", QSIZES, ids=str)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("block", [1, 128])
def test_quantise_sizes(rows, cols, transpose, block):
    for src, fmt in (("bf16", "e4m3"), ("f16", "e5m2")):
        v = (torch.randn(rows, cols, generator=gen(rows + cols), device="cuda") * 3).to(DT[src][0])
        _, q, s = quantize(v, fmt, transpose, block)
        wq, ws = quant64(v.t() if transpose else v, fmt, block)
        assert same(q, wq)
        assert scale_close(s, ws)


@pytest.mark.gpu
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("transpose,block", [(False, 1), (True, 1), (False, 128), (True, 128)])
def test_quantise_types(src, fmt, transpose, block):
    g = gen(5)
    v = torch.randn(200, 333, generator=g, device="cuda") * torch.exp(3 * torch.randn(200, 333, generator=g, device="cuda"))
    v = v.to(DT[src][0])
    _, q, s = quantize(v, fmt, transpose, block)
    vv = v.t() if transpose else v
    wq, ws = quant64(vv, fmt, block)
    assert scale_close(s, ws)
    if src != "f32":
        assert same(q, wq)
        return
    # fp32 values: v * 7/8 and the quotient are rounded to fp32 first, so a value within 2^-22 of
    # its size of the middle between two 8-bit ones may go to the other of the two
    _, _, fmax, bits, low = F8[fmt]
    t = vv.double() / ws.repeat_interleave(128, 0)[:vv.shape[1]].t().repeat_interleave(block, 0)[:vv.shape[0]]
    step = torch.exp2((torch.frexp(t).exponent - 1).clamp_min(low).double() - bits)
    mid = ((t / step).abs() % 1.0 - 0.5).abs() * step <= 2.0 ** -22 * t.abs()
    off = (q != wq) & ~mid
    assert not off.any() and ((q - wq).abs() <= step).all()


@pytest.mark.gpu
def test_quantise_midpoints():
    """Every ratio of two 8-bit mantissas, so every tie that bf16 values can make."""
    x = torch.arange(128, 256, device="cuda", dtype=torch.float64)
    for fmt in F8:
        for e in (0.0, -3.0, -9.0, 90.0, -100.0):
            big = (x * 2.0 ** e).bfloat16()[:, None]                        # a row's largest value
            row = torch.cat([big, (x[None, :127] * 2.0 ** (e - 1)).bfloat16().expand(128, 127)], 1).contiguous()
            row[:, 1:64] *= -0.125
            _, q, _ = quantize(row, fmt)
            assert same(q, quant64(row, fmt, 1)[0]), (fmt, e)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantise_special_values(fmt):
    fmax = F8[fmt][2]
    v = torch.randn(8, 384, generator=gen(3), device="cuda")
    v[0] = 0
    v[1] = 1e-45                       # below the smallest scale: 2^-126
    v[2, 5], v[2, 6] = 3.38e38, -3e38
    v[3, 7] = float("nan")
    v[4, 130] = float("inf")
    v[5, :128] = -0.0
    _, q, s = quantize(v, fmt)
    assert (q[0] == 0).all() and (s[:, 0] == 2.0 ** -126).all() and (q[5, :128] == 0).all()
    assert (q[1] * s[0, 1].double() <= 2e-45).all() and (s[:, 1] == 2.0 ** -126).all()
    assert q[2, 5] == fmax and q[2, 6] < 0
    assert q[3, 7].isnan() and q[3].isnan().sum() == 1                     # a NaN stays alone
    clean = v.clone()
    clean[3, 7] = 0
    assert torch.equal(quantize(clean, fmt)[1][3, :7], q[3, :7])
    assert s[1, 4].isinf() and q[4, 130].isnan() and not q[4, :128].isnan().any()
    assert (q[4, 128:256] * s[1, 4].double()).isnan().all()                # the group stands for NaN
    for transpose, block in ((True, 1), (False, 128), (True, 128)):
        _, q, s = quantize(v, fmt, transpose, block)
        assert s.isinf().sum() == (1 if block == 128 else 1)
        w = torch.zeros(130, 260, device="cuda")
        _, q, s = quantize(w, fmt, transpose, block)
        assert (q == 0).all() and (s == 2.0 ** -126).all()


# ----------------------------------------------------------------------------- product
def operand(v, fmt, block, pad=0):
    """v [rows, k] quantised by the library, with `pad` bytes of NaN after each row's 16 bytes."""
    ld = cdiv(v.shape[1], 16) * 16 + pad
    q, val, s = quantize(v, fmt, False, block, ldq=ld, fill=0x7F)
    rows, k = v.shape
    each = s.double().t().repeat_interleave(block, 0)[:rows].repeat_interleave(128, 1)[:, :k]
    return q, s, val * each, ld


def gemm(m, n, k, a, b, block, out, bias, relu, seed, pad=0):
    g = gen(seed)
    av = torch.randn(m, k, generator=g, device="cuda")
    bv = torch.randn(n, k, generator=g, device="cuda") * 0.1
    qa, sa, ra, lda = operand(av, a, 1, pad)
    qb, sb, rb, ldb = operand(bv, b, block, pad)
    bi = torch.randn(n, generator=g, device="cuda") if bias else None
    sp = cbr.make_gemm_shape(m, n, k, F8[a][1], F8[b][1], DT[out][1], block, relu, lda, ldb)
    ws = torch.full((cbr.cbr_gemm_fp8_workspace_bytes(sp),), 255, dtype=torch.uint8, device="cuda")
    d = torch.full((m + 1, n), 9.0, dtype=DT[out][0], device="cuda")
    cbr.cbr_gemm_fp8(sp, qa, sa, qb, sb, bi, d, ws if ws.numel() else None)
    assert (d[m] == 9).all()                # the row behind the last one stays as it was
    want = ra @ rb.t()
    mag = ra.abs() @ rb.abs().t()
    if bias:
        want, mag = want + bi.double(), mag + bi.double().abs()
    if relu:
        want = want.clamp_min(0)
    tol = (128 + cdiv(k, 128) + 16) * U * mag
    if out != "f32":
        eights = lambda v: torch.nn.functional.max_pool1d(  # noqa: E731
            torch.nn.functional.pad(v.abs(), (0, -k % 8))[None], 8)[0]
        tol = tol + 8 * 2.0 ** -13 * (eights(ra) @ eights(rb).t())
    if out != "f32":
        tol = tol + torch.finfo(DT[out][0]).eps / 2 * want.abs() + (2.0 ** -25 if out == "f16" else 0)
    bad = ~((d[:m].double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4], d[:m][bad][:4], want[bad][:4], tol[bad][:4])
    return d[:m]


# m: the forms for up to 16, 32 and 64 rows, the 128- and 256-wide tiles; n and k odd, short, long
GSIZES = [(1, 1, 1), (1, 1000, 2048), (3, 17, 130), (16, 128, 128), (17, 33, 100), (32, 256, 4100), (50, 130, 257),
          (64, 64, 640), (65, 65, 65), (100, 1, 1000), (128, 128, 128), (129, 255, 384), (200, 300, 1111), (513, 130, 96),
          (1000, 77, 16), (4100, 4200, 200), (4096, 4096, 256), (96, 64, 20011)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", GSIZES, ids=str)
@pytest.mark.parametrize("block", [128, 1])
def test_gemm_sizes(m, n, k, block):
    gemm(m, n, k, "e4m3", "e4m3", block, "bf16", True, False, m + n + k)


@pytest.mark.gpu
@pytest.mark.parametrize("a", ["e4m3", "e5m2"])
@pytest.mark.parametrize("b", ["e4m3", "e5m2"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bias,relu", [(False, False), (True, True)])
@pytest.mark.parametrize("m,n,k", [(40, 70, 300), (150, 140, 300)], ids=str)
def test_gemm_types(a, b, out, bias, relu, m, n, k):
    for block in (1, 128):
        gemm(m, n, k, a, b, block, out, bias, relu, 4, pad=32)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(5, 40, 777), (64, 200, 1500), (300, 200, 777), (4200, 4100, 130)], ids=str)
def test_gemm_whole_numbers_are_exact(m, n, k):
    """Every product, lane, block and tail byte, with no rounding to hide behind."""
    g = gen(k)
    for block in (1, 128):
        ld = cdiv(k, 16) * 16 + 16
        val = lambda r: torch.randint(-4, 5, (r, k), generator=g, device="cuda").float()  # noqa: E731
        av, bv = val(m), val(n)

        def raw(v):
            q = torch.full((v.shape[0], ld), 0x7F, dtype=torch.uint8, device="cuda")   # NaN past the rows
            q[:, :k] = v.to(torch.float8_e4m3fn).view(torch.uint8)
            return q
        kb = cdiv(k, 128)
        sa = torch.exp2(torch.randint(-2, 3, (kb, m), generator=g, device="cuda").float())
        sb = torch.exp2(torch.randint(-2, 3, (kb, cdiv(n, block)), generator=g, device="cuda").float())
        each = torch.arange(k, device="cuda") // 128
        ra = av.double() * sa.double()[each].t()
        rb = bv.double() * sb.double()[each].t().repeat_interleave(block, 0)[:n]
        sp = cbr.make_gemm_shape(m, n, k, d_type=cbr.CBR_F32, b_block=block, lda=ld, ldb=ld)
        ws = torch.empty(max(16, cbr.cbr_gemm_fp8_workspace_bytes(sp)), dtype=torch.uint8, device="cuda")
        d = torch.empty(m, n, device="cuda")
        cbr.cbr_gemm_fp8(sp, raw(av), sa, raw(bv), sb, None, d, ws)
        assert torch.equal(d.double(), ra @ rb.t())


@pytest.mark.gpu
def test_gemm_nan_and_infinity():
    """A NaN operand or an infinite scale reaches its row's results and no others; relu keeps a NaN."""
    for m in (20, 200):
        g = gen(m)
        qa, sa, _, lda = operand(torch.randn(m, 300, generator=g, device="cuda"), "e4m3", 1)
        qb, sb, _, ldb = operand(torch.randn(140, 300, generator=g, device="cuda"), "e4m3", 128)
        sp = cbr.make_gemm_shape(m, 140, 300, d_type=cbr.CBR_F32, relu=True, lda=lda, ldb=ldb)
        ws = torch.empty(max(16, cbr.cbr_gemm_fp8_workspace_bytes(sp)), dtype=torch.uint8, device="cuda")
        run = lambda: (cbr.cbr_gemm_fp8(sp, qa, sa, qb, sb, None, d := torch.empty(m, 140, device="cuda"), ws), d)[1]  # noqa: E731
        clean = run()
        qa[3, 299] = 0x7F
        sa[1, 7] = float("inf")
        d = run()
        keep = [i for i in range(m) if i not in (3, 7)]
        assert torch.equal(d[keep], clean[keep]) and d[3].isnan().all()
        assert not d[7][d[7] != 0].isfinite().any()


@pytest.mark.gpu
def test_gemm_reproducible_graph_and_stream():
    """A split sum, eagerly, on another stream and replayed from a graph on new operands."""
    m, n, k = 256, 256, 20000
    sp = cbr.make_gemm_shape(m, n, k, d_type=cbr.CBR_F32, b_block=1)
    ws = torch.empty(cbr.cbr_gemm_fp8_workspace_bytes(sp), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    mk = lambda s: [*operand(torch.randn(m, k, generator=gen(s), device="cuda"), "e4m3", 1)[:2],  # noqa: E731
                    *operand(torch.randn(n, k, generator=gen(s + 1), device="cuda"), "e4m3", 1)[:2]]
    x = mk(1)
    d, e = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    cbr.cbr_gemm_fp8(sp, *x, None, d, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cbr.cbr_gemm_fp8(sp, *x, None, e, ws.clone(), stream=s)
    s.synchronize()
    assert torch.equal(d, e)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        cbr.cbr_gemm_fp8(sp, *x, None, e, ws)
    for seed in (5, 6, 7):
        for t, v in zip(x, mk(seed)):
            t.copy_(v)
        gr.replay()
        torch.cuda.synchronize()
        cbr.cbr_gemm_fp8(sp, *x, None, d, torch.empty_like(ws))
        torch.cuda.synchronize()
        assert torch.equal(d, e)


# ---------------------------------------------------------------------------- refusals
FAKE = 0x100000


def _q(sp, src=FAKE, q=FAKE, s=FAKE):
    return cbr._load().cbr_fp8_quantize(ctypes.byref(sp), src, q, s, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), 2), (dict(cols=-1), 2), (dict(ldq=120), 2), (dict(ldq=136), 2), (dict(src_type=3), 7),
    (dict(q_type=0), 7), (dict(block=64), 7), (dict(rows=1 << 31), 3), (dict(cols=1 << 31, ldq=1 << 31), 3),
    (dict(rows=2000000000, cols=1 << 20, ldq=1 << 20), 3), (dict(transpose=True, ldq=16), 2),
    (dict(rows=1 << 30, cols=1, ldq=16), 3),
])
def test_quantise_refusals(kw, status):
    a = dict(rows=64, cols=128)
    a.update(kw)
    assert _q(cbr.make_quant_shape(**a)) == status


@pytest.mark.parametrize("over,status", [(dict(src=None), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(src=FAKE + 2), 4),
                                         (dict(q=FAKE + 8), 4), (dict(s=FAKE + 4), 4)])
def test_quantise_pointer_refusals(over, status):
    assert _q(cbr.make_quant_shape(64, 128), **over) == status


def _g(sp, **over):
    a = dict(a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, bias=FAKE, d=FAKE, ws=FAKE, nb=1 << 40)
    a.update(over)
    return cbr._load().cbr_gemm_fp8(ctypes.byref(sp), *a.values(), 0)


@pytest.mark.parametrize("kw,status", [
    (dict(m=0), 2), (dict(n=0), 2), (dict(k=-5), 2), (dict(lda=1000), 2), (dict(ldb=1032), 2), (dict(a_type=0), 7),
    (dict(b_type=9), 7), (dict(d_type=3), 7), (dict(b_block=32), 7), (dict(m=1 << 31), 3), (dict(n=(1 << 23) + 1), 3),
    (dict(k=(1 << 23) + 16), 3), (dict(lda=(1 << 23) + 16), 3), (dict(m=(1 << 31) - 1, n=1 << 23), 3),
])
def test_gemm_refusals(kw, status):
    a = dict(m=512, n=256, k=1024)
    a.update(kw)
    sp = cbr.make_gemm_shape(**a)
    assert _g(sp) == status and cbr.cbr_gemm_fp8_workspace_bytes(sp) == 0


@pytest.mark.parametrize("over,status", [
    (dict(a=None), 1), (dict(sa=None), 1), (dict(b=None), 1), (dict(sb=None), 1), (dict(d=None), 1), (dict(a=FAKE + 8), 4),
    (dict(sb=FAKE + 4), 4), (dict(bias=FAKE + 4), 4), (dict(d=FAKE + 2), 4), (dict(ws=None), 5), (dict(nb=64), 5),
    (dict(ws=FAKE + 4), 4),
])
def test_gemm_pointer_refusals(over, status):
    sp = cbr.make_gemm_shape(256, 256, 20000, b_block=1)
    assert cbr.cbr_gemm_fp8_workspace_bytes(sp) > 0
    assert _g(sp, **over) == status


def test_null_shapes():
    L = cbr._load()
    assert L.cbr_fp8_quantize(None, FAKE, FAKE, FAKE, 0) == 1
    assert L.cbr_gemm_fp8(None, FAKE, FAKE, FAKE, FAKE, None, FAKE, None, 0, 0) == 1
    assert L.cbr_gemm_fp8_workspace_bytes(None) == 0


def test_binding_refuses_host_tensors():
    t = torch.zeros(64, 128)
    with pytest.raises(cbr.CbrError, match="not a GPU tensor"):
        cbr.cbr_fp8_quantize(cbr.make_quant_shape(64, 128, cbr.CBR_F32), t, t, t)
    with pytest.raises(cbr.CbrError, match="not a GPU tensor"):
        cbr.cbr_gemm_fp8(cbr.make_gemm_shape(64, 64, 128), t, t, t, t, None, t)
    with pytest.raises(cbr.CbrError):
        cbr.cbr_fp8_quantize(cbr.make_quant_shape(64, 128, 99), t, t, t)


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    t = torch.zeros(64, 128, device="cuda")
    q, s = torch.zeros(64, 128, dtype=torch.uint8, device="cuda"), torch.zeros(64, device="cuda")
    sp = cbr.make_quant_shape(64, 128, cbr.CBR_F32)
    with pytest.raises(cbr.CbrError, match="q is torch.float8_e5m2"):
        cbr.cbr_fp8_quantize(sp, t, q.view(torch.float8_e5m2), s)
    with pytest.raises(cbr.CbrError, match="scale holds"):
        cbr.cbr_fp8_quantize(sp, t, q, s[:63])
    d = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(cbr.CbrError, match="b holds"):
        cbr.cbr_gemm_fp8(cbr.make_gemm_shape(64, 64, 128, b_block=1), q, s, q[:60], s, None, d)
    with pytest.raises(cbr.CbrError, match="d is torch.bfloat16"):
        cbr.cbr_gemm_fp8(cbr.make_gemm_shape(64, 64, 128, b_block=1, d_type=cbr.CBR_F16), q, s, q, s, None, d)
