"""The 4-bit quantiser, its inverse and the 4-bit matrix product against their definitions in 64 bits, and
their refusals.

The quantiser and its inverse are compared value for value: scales are powers of two, so everything but the one
rounding is exact.  Tolerance of the product: an instruction of 128 values is within 2^-23 of the sum of
magnitudes it adds to and adds (measured: 2^-23.4), so `instructions` of them, the eight waves' or the splits'
sums and the bias are within (instructions + splits + 10) 2^-23 of all magnitudes; then half a step of the
output's type.  Small whole numbers with equal scales are exact in fp32 and have to come out equal."""
import ctypes

import pytest
import torch

import conv2d_batchnorm_relu_amd as cbr

DT = {"bf16": (torch.bfloat16, cbr.CBR_BF16), "f16": (torch.float16, cbr.CBR_F16), "f32": (torch.float32, cbr.CBR_F32)}
CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def cdiv(a, b):
    return -(-a // b)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# --------------------------------------------------------------------------- quantiser
def quant64(v):
    """(values [rows, k], scale bytes [rows, groups]) of v [rows, k]; a group with a NaN or infinity: NaN, 255."""
    rows, k = v.shape
    p = torch.zeros(rows, cdiv(k, 32) * 32, dtype=torch.float64, device=v.device)
    p[:, :k] = v.double()
    p = p.view(rows, -1, 32)
    a = p.abs().amax(2)
    bad = ~(a < float("inf"))               # (a NaN is the largest)
    e = (torch.frexp(torch.where(bad, torch.ones_like(a), a)).exponent - 3).clamp_min(-127)
    e = torch.where(a == 0, torch.full_like(e, -127), e)
    t = torch.where(bad[:, :, None], torch.zeros_like(p), p) * torch.exp2(-e.double())[:, :, None]
    codes = torch.tensor(CODES, dtype=torch.float64, device=v.device)
    d = (t.abs()[..., None] - codes).abs()
    best = d.amin(-1, keepdim=True)
    near = (d == best)
    even = near & (torch.arange(8, device=v.device) % 2 == 0)
    pick = torch.where(even.any(-1), even.int().argmax(-1), near.int().argmax(-1))    # ties: the even code
    q = codes[pick] * torch.where(t < 0, -1.0, 1.0) * torch.exp2(e.double())[:, :, None]
    q = torch.where(bad[:, :, None], torch.full_like(q, float("nan")), q)
    return q.view(rows, -1)[:, :k], torch.where(bad, torch.full_like(e, 255), e + 127)


def decode64(q, scale, k):
    """What bytes q [rows, ldq] and scales [k / 128, rows, 4] stand for."""
    lut = torch.tensor(CODES + [-c for c in CODES], dtype=torch.float64, device=q.device)
    v = torch.stack((lut[(q & 15).long()], lut[(q >> 4).long()]), 2).view(q.shape[0], -1)[:, :cdiv(k, 32) * 32]
    b = scale.transpose(0, 1).reshape(q.shape[0], -1)[:, :cdiv(k, 32)].double()
    s = torch.where(b == 255, torch.full_like(b, float("nan")), torch.exp2(b - 127))
    return (v.view(q.shape[0], -1, 32) * s[:, :, None]).view(q.shape[0], -1)[:, :k]


def same(x, y):
    return x.shape == y.shape and bool(((x == y) | (x.isnan() & y.isnan())).all())


def quantize(src, transpose=False, ldq=None):
    """q, scale; also checks what lies behind the rows and the groups."""
    rows, cols = (src.shape[1], src.shape[0]) if transpose else src.shape
    dt = {v[0]: v[1] for v in DT.values()}[src.dtype]
    sp = cbr.make_fp4_shape(src.shape[0], src.shape[1], dt, transpose, ldq)
    q = torch.full((rows, sp.ldq), 0xA5, dtype=torch.uint8, device=src.device)
    s = torch.full((cdiv(cols, 128), rows, 4), 0x5A, dtype=torch.uint8, device=src.device)
    cbr.cbr_fp4_quantize(sp, src, q, s)
    used = cdiv(cols, 32) * 16
    assert (q[:, used:] == 0xA5).all()
    pad = decode64(q, torch.full_like(s, 127), cdiv(cols, 32) * 32)[:, cols:]
    assert (pad == 0).all()
    assert (s.transpose(0, 1).reshape(rows, -1)[:, cdiv(cols, 32):] == 127).all()
    return sp, q, s


def dequantize(sp, q, s):
    rows, cols = (sp.cols, sp.rows) if sp.transpose else (sp.rows, sp.cols)
    t = {v[1]: v[0] for v in DT.values()}[sp.type]
    v = torch.full((rows * cols + 64,), 7.0, dtype=t, device=q.device)
    cbr.cbr_fp4_dequantize(sp, q, s, v)
    assert (v[rows * cols:] == 7).all()
    return v[:rows * cols].view(rows, cols)


def check_quantize(v, transpose=False, ldq=None):
    sp, q, s = quantize(v, transpose, ldq)
    vv = v.t() if transpose else v
    want, byte = quant64(vv)
    assert torch.equal(s.transpose(0, 1).reshape(vv.shape[0], -1)[:, :byte.shape[1]].int(), byte.int())
    assert same(decode64(q, s, vv.shape[1]), want)
    back = dequantize(sp, q, s)
    assert same(back, want.to(v.dtype))
    if v.dtype != torch.float16:
        assert same(back.double(), want)      # every one of these is a number of the type


SIZES = [(1, 1), (1, 31), (1, 32), (3, 33), (2, 128), (17, 8), (64, 256), (100, 1000), (129, 127), (257, 384), (130, 67), (5, 4099),
         (300, 16), (1000, 96), (70, 2049), (4099, 5), (520, 200)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("src", list(DT))
def test_quantise_sizes(size, transpose, src):
    g = gen(sum(size))
    v = torch.randn(*size, generator=g, device="cuda") * torch.exp(2 * torch.randn(*size, generator=g, device="cuda"))
    ld = cdiv(size[0] if transpose else size[1], 32) * 16 + 16 * (sum(size) % 3)
    check_quantize(v.to(DT[src][0]), transpose, ld)


@pytest.mark.gpu
@pytest.mark.parametrize("src", list(DT))
@pytest.mark.parametrize("transpose", [False, True])
def test_quantise_every_ratio(src, transpose):
    """Every 16-bit value against a group's largest of a few sizes: all ties and neighbours, small and large scales."""
    t = DT[src][0]
    every = torch.arange(0, 1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.float16 if src == "f16" else torch.bfloat16)
    every = every[every.isfinite()].float()
    for top in (1.0, 1.5, 1.9921875, 6.0, 7.5, 2.0 ** -14, 3 * 2.0 ** -120, 5 * 2.0 ** 125, 2.0 ** -126, 1e-39):
        if src == "f16" and not 1e-5 < top < 6e4:
            continue
        v = every[every.abs() <= top]
        v = torch.cat((v, torch.zeros(-v.numel() % 31, device="cuda"))).view(-1, 31)
        v = torch.cat((torch.full_like(v[:, :1], top), v), 1).to(t)
        check_quantize(v.t().contiguous() if transpose else v, transpose)


@pytest.mark.gpu
def test_quantise_single_precision_ties():
    """fp32 values next to the middles of 4-bit ones, one step to either side."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.0], device="cuda")
    up, down = torch.nextafter(mid, mid + 1), torch.nextafter(mid, mid - 1)
    v = torch.cat((torch.tensor([4.0, -7.99, 0, -0.0, 1e-44], device="cuda"), mid, up, down[:-6], -mid[:6]))[:32]
    v = torch.cat((v, torch.zeros(32 - v.numel(), device="cuda")))
    rows = torch.stack([v * 2.0 ** e for e in (0, 1, -3, 60, -60, 120, -100)])
    check_quantize(rows)
    check_quantize(rows.t().contiguous(), True)


@pytest.mark.gpu
@pytest.mark.parametrize("src", list(DT))
@pytest.mark.parametrize("transpose", [False, True])
def test_quantise_special_values(src, transpose):
    t = DT[src][0]
    v = torch.randn(9, 160, generator=gen(3), device="cuda").to(t)
    v[0] = 0
    v[1, 5], v[2, 40], v[3, 70], v[4, 159] = float("nan"), float("inf"), float("-inf"), float("nan")
    v[5] = torch.finfo(t).max
    v[6] = -torch.finfo(t).smallest_normal
    v[7] = torch.finfo(t).smallest_normal * torch.finfo(t).eps * 3
    v[8, :32] = -0.0
    if src != "f16":
        bits = v[1:2, 96:97].contiguous().view(torch.int16 if t.itemsize == 2 else torch.int32)
        bits.fill_(0x7F81 if t.itemsize == 2 else 0x7F800001)       # a signalling NaN
        v[1, 96] = bits.view(t)[0, 0]
    check_quantize(v.t().contiguous() if transpose else v, transpose)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
def test_dequantise_every_code_and_scale(dtype):
    """Every code under every scale, the smallest, the largest and NaN among them."""
    q = torch.arange(256, dtype=torch.uint8, device="cuda").view(16, 16).repeat(256, 1)       # 16 rows of 32 codes a scale
    byte = torch.arange(256, dtype=torch.uint8, device="cuda").repeat_interleave(16)
    s = torch.full((1, 4096, 4), 9, dtype=torch.uint8, device="cuda")
    s[0, :, 0] = byte
    sp = cbr.make_fp4_shape(4096, 32, DT[dtype][1])
    back = dequantize(sp, q, s)
    want = decode64(q, s, 32)
    assert same(back, want.to(DT[dtype][0]))


# ----------------------------------------------------------------------------- product
def operand(rows, k, seed, spread=0, ld_extra=0, whole=False):
    """bytes [rows, ld] and scales of random codes; what is not used is filled with what would show."""
    g = gen(seed)
    groups = cdiv(k, 32)
    ld = groups * 16 + ld_extra
    q = torch.randint(0, 256, (rows, ld), generator=g, device="cuda").to(torch.uint8)
    if whole:                                     # codes of 0, 1, 2 only
        lut = torch.tensor([0, 2, 4, 10], dtype=torch.uint8, device="cuda")
        q = lut[(q & 3).long()] | lut[(q >> 2 & 3).long()] << 4
    code = torch.stack((q & 15, q >> 4), 2).view(rows, -1)
    code[:, k:groups * 32] = 0
    q = (code[:, ::2] | code[:, 1::2] << 4).contiguous()
    s = torch.full((cdiv(k, 128), rows, 4), 255, dtype=torch.uint8, device="cuda")     # NaN where there is no group
    e = 127 + torch.randint(-spread, spread + 1, (rows, groups), generator=g, device="cuda")
    flat = torch.full((rows, cdiv(k, 128) * 4), 255, dtype=torch.uint8, device="cuda")
    flat[:, :groups] = e.to(torch.uint8)
    s = flat.view(rows, -1, 4).transpose(0, 1).contiguous()
    return q, s


def product(m, n, k, a, b, out, bias=None, relu=False):
    (qa, sa), (qb, sb) = a, b
    sp = cbr.make_gemm_fp4_shape(m, n, k, DT[out][1], relu, qa.shape[1], qb.shape[1])
    need = cbr.cbr_gemm_fp4_workspace_bytes(sp)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None
    d = torch.full((m * n + 64,), 7.0, dtype=DT[out][0], device="cuda")
    cbr.cbr_gemm_fp4(sp, qa, sa, qb, sb, bias, d, ws)
    assert (d[m * n:] == 7).all()
    return d[:m * n].view(m, n)


def check_product(m, n, k, a, b, out, bias=None, relu=False):
    d = product(m, n, k, a, b, out, bias, relu)
    va, vb = decode64(*a, k), decode64(*b, k)
    want, mag = va @ vb.t(), va.abs() @ vb.abs().t()
    if bias is not None:
        want, mag = want + bias.double(), mag + bias.double().abs()
    if relu:
        want = want.clamp_min(0)
    tol = (cdiv(k, 128) + 512 + 10) * 2.0 ** -23 * mag
    f = torch.finfo(DT[out][0])
    big = want.abs() + tol > f.max
    tol = tol + f.eps / 2 * (want.abs() + tol) + f.smallest_normal * f.eps
    assert ((d.double() - want).abs() <= tol)[~big].all()
    assert (d.double() - want)[~big].norm() <= (4 * f.eps + 2.0 ** -18) * mag.norm()     # errors are not one-sided: far inside the bound
    assert torch.equal(d, product(m, n, k, a, b, out, bias, relu))


PSIZES = [(1, 1, 1), (1, 1000, 2048), (3, 17, 33), (16, 16, 32), (17, 48, 64), (33, 130, 257), (64, 64, 128), (65, 63, 96), (64, 100, 5000),
          (100, 257, 511), (128, 128, 256), (129, 384, 1000), (256, 256, 512), (300, 520, 4099), (1000, 77, 160), (513, 255, 8192), (2049, 1030, 288),
          (48, 4100, 1056), (5000, 33, 64), (256, 64, 40000)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", PSIZES, ids=str)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_product_sizes(size, out):
    m, n, k = size
    i = PSIZES.index(size)
    a, b = operand(m, k, i, 2, 16 * (i % 3)), operand(n, k, 50 + i, 2, 32 * (i % 2))
    bias = torch.randn(n, generator=gen(i), device="cuda") if i % 2 else None
    check_product(m, n, k, a, b, out, bias, relu=i % 4 == 1)


# every form on one round of workgroups and on more, whole and in splits
FSIZES = [(1, 4260, 77), (7, 400, 18650), (25, 70, 9000), (17000, 1, 33), (1800, 40, 6266), (9001, 800, 96), (300, 7000, 1100), (1049, 81, 67300),
          (12622, 3, 13860), (24000, 300, 64), (3004, 141, 93800)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", FSIZES, ids=str)
def test_product_forms(size):
    m, n, k = size
    a, b = operand(m, k, 20, 1), operand(n, k, 21, 1)
    for out in ("bf16", "f32"):
        check_product(m, n, k, a, b, out, torch.randn(n, generator=gen(2), device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("size", PSIZES, ids=str)
def test_product_of_whole_numbers_is_exact(size):
    m, n, k = size
    a, b = operand(m, k, 3, whole=True), operand(n, k, 4, whole=True)
    want = decode64(*a, k) @ decode64(*b, k).t()
    assert torch.equal(product(m, n, k, a, b, "f32").double(), want)
    # every operand row shows in its own result only: one group of one row scaled up
    t = cdiv(k, 32) - 1
    a[1][t // 4, m - 1, t % 4] = 127 + 4
    want = decode64(*a, k) @ decode64(*b, k).t()
    assert torch.equal(product(m, n, k, a, b, "f32").double(), want)
    b[1][t // 4, n // 2, t % 4] = 127 - 3
    want = decode64(*a, k) @ decode64(*b, k).t()
    assert torch.equal(product(m, n, k, a, b, "f32").double(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(20, 40, 300), (64, 70, 1030), (200, 300, 700), (2100, 1100, 400), (300, 300, 9000)], ids=str)
def test_product_wide_scales(size):
    """Exponents spread over 2^-20 .. 2^20 of each operand: held to the magnitudes all the same."""
    m, n, k = size
    for out in DT:
        a, b = operand(m, k, 8, 20), operand(n, k, 9, 20)
        if out == "f16":
            a, b = operand(m, k, 8, 3), operand(n, k, 9, 3)
        check_product(m, n, k, a, b, out, relu=True)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(20, 40, 300), (200, 300, 700), (2100, 1100, 400)], ids=str)
def test_product_extreme_scales(size):
    """Scales far from 1 whose product is not: 2^100 against 2^-100, and the whole way to fp32's ends."""
    m, n, k = size
    for x, y in ((100, -100), (-125, 120), (120, -60), (-60, -50), (-127, 127)):
        (qa, sa), (qb, sb) = operand(m, k, 8), operand(n, k, 9)
        sa, sb = (torch.where(s == 127, torch.full_like(s, 127 + e), s) for s, e in ((sa, x), (sb, y)))
        check_product(m, n, k, (qa, sa), (qb, sb), "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(20, 40, 300), (200, 300, 700), (2100, 1100, 400)], ids=str)
def test_product_nan_scales_stay_in_their_rows(size):
    m, n, k = size
    a, b = operand(m, k, 5, 1), operand(n, k, 6, 1)
    clean = product(m, n, k, a, b, "f32", relu=True)
    a[1][1, 7, 2] = 255
    b[1][0, 11, 0] = 255
    d = product(m, n, k, a, b, "f32", relu=True)
    hit = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    hit[7], hit[:, 11] = True, True
    assert d[hit].isnan().all() and torch.equal(d[~hit], clean[~hit])


@pytest.mark.gpu
def test_quantised_product_is_the_product_of_what_was_quantised():
    g = gen(1)
    for m, n, k in ((50, 96, 200), (300, 260, 1000)):
        x = (torch.randn(m, k, generator=g, device="cuda") * 3).bfloat16()
        w = torch.randn(k, n, generator=g, device="cuda").bfloat16()       # turned over by the quantiser
        _, qa, sa = quantize(x)
        _, qb, sb = quantize(w, True)
        check_product(m, n, k, (qa, sa), (qb, sb), "bf16")
        va, vb = quant64(x)[0], quant64(w.t())[0]
        d = product(m, n, k, (qa, sa), (qb, sb), "f32").double()
        assert (d - va @ vb.t()).abs().max() <= 2.0 ** -18 * (va.abs() @ vb.abs().t()).max()


# ---------------------------------------------------------------------------- refusals
FAKE = 0x10000


def _status(name, sp, *args):
    return getattr(cbr._load(), name)(ctypes.byref(sp) if sp is not None else None, *args)


def test_quantiser_refusals():
    for name in ("cbr_fp4_quantize", "cbr_fp4_dequantize"):
        ok = [FAKE, 2 * FAKE, 3 * FAKE]
        for bad, want in ((dict(rows=0), 2), (dict(cols=0), 2), (dict(cols=-3), 2), (dict(type=3), 7), (dict(type=-1), 7), (dict(ldq=16), 2),
                          (dict(ldq=56), 2), (dict(ldq=0), 2), (dict(rows=2 ** 31), 3), (dict(cols=2 ** 31, ldq=2 ** 31), 3),
                          (dict(rows=2 ** 31 - 1, cols=1 << 10, ldq=1 << 9), 3)):
            sp = cbr.make_fp4_shape(9, 100)
            for k, v in bad.items():
                setattr(sp, k, v)
            assert _status(name, sp, *ok, None) == want, bad
        sp = cbr.make_fp4_shape(9, 100)
        assert _status(name, None, *ok, None) == 1
        for i in range(3):
            assert _status(name, sp, *(None if j == i else p for j, p in enumerate(ok)), None) == 1
            assert _status(name, sp, *(p + 8 if j == i else p for j, p in enumerate(ok)), None) == 4
        sp = cbr.make_fp4_shape(100, 9, transpose=True)
        assert sp.ldq == 64
        sp.ldq = 48
        assert _status(name, sp, *ok, None) == 2


def test_product_refusals():
    ok = [FAKE, 2 * FAKE, 3 * FAKE, 4 * FAKE, None, 5 * FAKE]
    for bad, want in ((dict(m=0), 2), (dict(n=0), 2), (dict(k=0), 2), (dict(d_type=3), 7), (dict(lda=32), 2), (dict(ldb=32), 2), (dict(lda=56), 2),
                      (dict(ldb=72), 2), (dict(m=2 ** 31), 3), (dict(n=2 ** 22 + 1), 3), (dict(lda=2 ** 22 + 16), 3), (dict(ldb=2 ** 22 + 16), 3),
                      (dict(k=2 ** 23 + 1, lda=2 ** 22, ldb=2 ** 22), 3), (dict(m=2 ** 31 - 1, n=2 ** 22), 3)):
        sp = cbr.make_gemm_fp4_shape(10, 20, 100)
        for k, v in bad.items():
            setattr(sp, k, v)
        assert _status("cbr_gemm_fp4", sp, *ok, None, 0, None) == want, bad
        assert cbr.cbr_gemm_fp4_workspace_bytes(sp) == 0
    sp = cbr.make_gemm_fp4_shape(10, 20, 100)
    assert _status("cbr_gemm_fp4", None, *ok, None, 0, None) == 1
    for i in (0, 1, 2, 3, 5):
        assert _status("cbr_gemm_fp4", sp, *(None if j == i else p for j, p in enumerate(ok)), None, 0, None) == 1
        assert _status("cbr_gemm_fp4", sp, *(p + 4 if j == i else p for j, p in enumerate(ok)), None, 0, None) == 4
    assert _status("cbr_gemm_fp4", sp, *ok[:4], FAKE + 4, ok[5], None, 0, None) == 4
    sp = cbr.make_gemm_fp4_shape(256, 256, 1 << 17)
    need = cbr.cbr_gemm_fp4_workspace_bytes(sp)
    assert need > 0
    assert _status("cbr_gemm_fp4", sp, *ok, None, 0, None) == 5 and _status("cbr_gemm_fp4", sp, *ok, FAKE, need - 1, None) == 5
    assert _status("cbr_gemm_fp4", sp, *ok, FAKE + 8, need, None) == 4


@pytest.mark.gpu
def test_binding_refuses_tensors_that_do_not_fit():
    (qa, sa), (qb, sb) = operand(10, 100, 1), operand(20, 100, 2)
    sp = cbr.make_gemm_fp4_shape(10, 20, 100)
    d = torch.empty(10, 20, dtype=torch.bfloat16, device="cuda")
    cbr.cbr_gemm_fp4(sp, qa, sa.view(torch.float8_e8m0fnu), qb.view(torch.float4_e2m1fn_x2), sb, None, d)
    for a, e, o in ((qa[:9], sa, d), (qa, sa[:, :9].contiguous(), d), (qa.cpu(), sa, d), (qa, sa, d.float()), (qa.float(), sa, d), (qa, sa.float(), d),
                    (qa, sa, d[:5])):
        with pytest.raises(cbr.CbrError):
            cbr.cbr_gemm_fp4(sp, a, e, qb, sb, None, o)
    qp = cbr.make_fp4_shape(8, 64)
    v = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty(8, 32, dtype=torch.uint8, device="cuda"), torch.empty(1, 8, 4, dtype=torch.uint8, device="cuda")
    for x, y, z in ((v.float(), q, s), (v[:7], q, s), (v, q[:7], s), (v, q, s[:, :7].contiguous()), (v.cpu(), q, s)):
        with pytest.raises(cbr.CbrError):
            cbr.cbr_fp4_quantize(qp, x, y, z)
        with pytest.raises(cbr.CbrError):
            cbr.cbr_fp4_dequantize(qp, y, z, x)
