"""The sums of the 8-bit product are fp32 whatever the output's type and the number of rows, unless
the caller asks for short ones, which are held to what the header says of them.

Whole numbers times powers of two: every partial sum, in any order, is a whole number below 2^24
and so exact in fp32; the one rounding is the output's.  Pairs of large products cancel within
eight consecutive k, which leaves small ones that a sum of fewer bits has lost."""
import pytest
import torch

import conv2d_batchnorm_relu_amd as cbr

gpu = pytest.mark.gpu
DT = {"bf16": (torch.bfloat16, cbr.CBR_BF16), "f16": (torch.float16, cbr.CBR_F16), "f32": (torch.float32, cbr.CBR_F32)}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def raw(v, fmt, ld):
    q = torch.full((v.shape[0], ld), 0x7F, dtype=torch.uint8, device="cuda")   # NaN past the rows
    q[:, :v.shape[1]] = v.to(fmt).view(torch.uint8)
    return q


def cancelling(m, n, k, seed):
    """a [m][k], b [n][k]: of each eight k the first two (at a place drawn for the eight) have products
    of 2^16 that cancel, the others products of at most 9."""
    g = gen(seed)
    small = lambda r: torch.randint(-3, 4, (r, k), generator=g, device="cuda").float()  # noqa: E731
    a, b = small(m), small(n)
    at = torch.arange(0, k - 7, 8, device="cuda")
    one = at + torch.randint(0, 4, at.shape, generator=g, device="cuda")
    two = one + 1 + torch.randint(0, 3, at.shape, generator=g, device="cuda")
    sign = torch.randint(0, 2, (m, at.numel()), generator=g, device="cuda").float() * 2 - 1
    a[:, one] = a[:, two] = 256 * sign
    sign = torch.randint(0, 2, (n, at.numel()), generator=g, device="cuda").float() * 2 - 1
    b[:, one], b[:, two] = 256 * sign, -256 * sign
    return a, b


# m: up to 64 rows straight from memory; 64-, 128- and 256-wide tiles, splits of the long sums
@gpu
@pytest.mark.parametrize("m,n,k", [(3, 40, 300), (40, 70, 777), (64, 200, 1500), (200, 300, 1111), (701, 1001, 3001),
                                   (1501, 1203, 1500), (4000, 4001, 500), (300, 200, 3990)], ids=str)
@pytest.mark.parametrize("block", [128, 1])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_cancelling_products_keep_the_small_ones(m, n, k, block, out):
    av, bv = cancelling(m, n, k, m + n + k)
    ld = -(-k // 16) * 16 + 16
    kb = -(-k // 128)
    sa = torch.exp2(torch.randint(-2, 1, (kb, m), generator=gen(1), device="cuda").float())
    sb = torch.exp2(torch.randint(-2, 1, (kb, -(-n // block)), generator=gen(2), device="cuda").float())
    each = torch.arange(k, device="cuda") // 128
    want = (av.double() * sa.double()[each].t()) @ \
           (bv.double() * sb.double()[each].t().repeat_interleave(block, 0)[:n]).t()
    sp = cbr.make_gemm_shape(m, n, k, d_type=DT[out][1], b_block=block, lda=ld, ldb=ld)
    ws = torch.full((max(16, cbr.cbr_gemm_fp8_workspace_bytes(sp)),), 255, dtype=torch.uint8, device="cuda")
    d = torch.full((m + 1, n), 9.0, dtype=DT[out][0], device="cuda")
    cbr.cbr_gemm_fp8(sp, raw(av, torch.float8_e4m3fn, ld), sa, raw(bv, torch.float8_e4m3fn, ld), sb, None, d, ws)
    assert torch.equal(want.float().double(), want)
    assert torch.equal(d[:m], want.float().to(DT[out][0])) and (d[m] == 9).all()


@gpu
@pytest.mark.parametrize("signed", [True, False])
@pytest.mark.parametrize("k", [256, 40000])
@pytest.mark.parametrize("a,b", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_same_value_for_few_rows_and_many(a, b, k, signed):
    """Wide values, long and short sums: each result within fp32's rounding of its sum (128 products of
    a block, then the blocks and the splits' parts, 16 more for scaling) and half a step of the
    output, so whichever form the number of rows asks for gives the same up to that."""
    fmt = {"e4m3": (torch.float8_e4m3fn, cbr.CBR_E4M3), "e5m2": (torch.float8_e5m2, cbr.CBR_E5M2)}
    g = gen(k)
    n, kb = 96, -(-k // 128)
    wide = lambda r: (torch.randn(r, k, generator=g, device="cuda")  # noqa: E731
                      * torch.exp2(torch.randint(-6, 7, (r, k), generator=g, device="cuda").float())).clamp(-448, 448)
    av, bv = wide(400), wide(n)
    if not signed:
        av, bv = av.abs(), bv.abs()
    aq, bq = raw(av, fmt[a][0], k), raw(bv, fmt[b][0], k)
    ad, bd = aq.view(fmt[a][0]).double(), bq.view(fmt[b][0]).double()
    sa, sb = torch.full((kb, 400), 2.0 ** -12, device="cuda"), torch.full((kb, 1), 2.0 ** -10, device="cuda")
    want, mag = (ad @ bd.t()) * 2.0 ** -22, (ad.abs() @ bd.abs().t()) * 2.0 ** -22
    tol = (128 + kb + 16) * 2.0 ** -24 * mag
    for out in ("f16", "bf16"):
        half = torch.finfo(DT[out][0]).eps / 2 * (want.abs() + tol) + (2.0 ** -25 if out == "f16" else 0.0)
        for m in (16, 64, 400):
            sp = cbr.make_gemm_shape(m, n, k, fmt[a][1], fmt[b][1], DT[out][1])
            ws = torch.empty(max(16, cbr.cbr_gemm_fp8_workspace_bytes(sp)), dtype=torch.uint8, device="cuda")
            d = torch.empty(m, n, dtype=DT[out][0], device="cuda")
            cbr.cbr_gemm_fp8(sp, aq[:m], sa[:, :m].contiguous(), bq, sb, None, d, ws)
            bad = ~((d.double() - want[:m]).abs() <= (tol + half)[:m])
            assert not bad.any(), (out, m, int(bad.sum()), d[bad][:3], want[:m][bad][:3])


# ------------------------------------------------------------------------ short sums, where asked for
F8 = {"e4m3": (torch.float8_e4m3fn, cbr.CBR_E4M3), "e5m2": (torch.float8_e5m2, cbr.CBR_E5M2)}


def test_short_sums_are_for_16_bit_outputs():
    for d_type, status in ((cbr.CBR_BF16, 0), (cbr.CBR_F16, 0), (cbr.CBR_F32, 7)):
        sp = cbr.make_gemm_shape(256, 256, 20000, d_type=d_type, short_sums=True)
        assert (cbr.cbr_gemm_fp8_workspace_bytes(sp) == 0) == (status != 0)
        if status:
            fake = 0x100000
            got = cbr._load().cbr_gemm_fp8(cbr._sp(sp), fake, fake, fake, fake, None, fake, fake, 1 << 40, 0)
            assert got == status


# 256-, 128- (two and four blocks deep) and 64-wide tiles, splits of the last two, few rows
@gpu
@pytest.mark.parametrize("m,n,k,out", [
    (40, 70, 300, "bf16"), (4000, 4001, 1500, "bf16"), (3001, 2500, 700, "f16"), (2000, 1999, 1333, "bf16"),
    (1501, 1203, 1500, "f16"), (601, 500, 9001, "bf16"), (701, 1001, 30001, "bf16"),
], ids=str)
@pytest.mark.parametrize("block", [1, 128])
def test_short_sums_of_small_whole_numbers(m, n, k, out, block):
    """Products of at most 16 need 5 of the 13 bits: exact, so one rounding is all there is."""
    g = gen(k)
    av = torch.randint(-4, 5, (m, k), generator=g, device="cuda").float()
    bv = torch.randint(-4, 5, (n, k), generator=g, device="cuda").float()
    ld, kb = -(-k // 16) * 16 + 16, -(-k // 128)
    sa = torch.exp2(torch.randint(-2, 2, (kb, m), generator=g, device="cuda").float())
    sb = torch.exp2(torch.randint(-2, 2, (kb, -(-n // block)), generator=g, device="cuda").float())
    each = torch.arange(k, device="cuda") // 128
    want = (av.double() * sa.double()[each].t()) @ \
           (bv.double() * sb.double()[each].t().repeat_interleave(block, 0)[:n]).t()
    sp = cbr.make_gemm_shape(m, n, k, d_type=DT[out][1], b_block=block, lda=ld, ldb=ld, short_sums=True)
    ws = torch.full((max(16, cbr.cbr_gemm_fp8_workspace_bytes(sp)),), 255, dtype=torch.uint8, device="cuda")
    d = torch.full((m + 1, n), 9.0, dtype=DT[out][0], device="cuda")
    cbr.cbr_gemm_fp8(sp, raw(av, torch.float8_e4m3fn, ld), sa, raw(bv, torch.float8_e4m3fn, ld), sb, None, d, ws)
    assert torch.equal(d[:m], want.float().to(DT[out][0])) and (d[m] == 9).all()


@gpu
@pytest.mark.parametrize("a,b", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("bias,relu", [(False, False), (True, True)])
def test_short_sums_lose_less_than_the_header_says(a, b, bias, relu):
    """8 * 2^-13 of the largest product of each eight, taken product by product, beside fp32's own."""
    m, n, k = 96, 70, 1100
    g = gen(7)
    wide = lambda r: (torch.randn(r, k, generator=g, device="cuda")  # noqa: E731
                      * torch.exp2(torch.randint(-6, 7, (r, k), generator=g, device="cuda").float())).clamp(-448, 448)
    ld = -(-k // 16) * 16
    aq, bq = raw(wide(m), F8[a][0], ld), raw(wide(n), F8[b][0], ld)
    ad, bd = (torch.nn.functional.pad(q[:, :k].contiguous().view(F8[f][0]).double(), (0, -k % 8)) for q, f in ((aq, a), (bq, b)))
    each = ad[:, None] * bd[None]
    loss = 8 * 2.0 ** -13 * each.abs().view(m, n, -1, 8).amax(3).sum(2)
    want, mag = each.sum(2), each.abs().sum(2)
    sa, sb = torch.full((9, m), 2.0 ** -6, device="cuda"), torch.full((9, 1), 2.0 ** -6, device="cuda")
    bi = torch.randn(n, generator=g, device="cuda") if bias else None
    want, tol = want * 2.0 ** -12, (loss + (128 + 9 + 16) * 2.0 ** -24 * mag) * 2.0 ** -12
    if bias:
        want, tol = want + bi.double(), tol + 2.0 ** -24 * bi.double().abs()
    if relu:
        want = want.clamp_min(0)
    for out in ("f16", "bf16"):
        sp = cbr.make_gemm_shape(m, n, k, F8[a][1], F8[b][1], DT[out][1], relu=relu, short_sums=True)
        ws = torch.empty(max(16, cbr.cbr_gemm_fp8_workspace_bytes(sp)), dtype=torch.uint8, device="cuda")
        d = torch.empty(m, n, dtype=DT[out][0], device="cuda")
        cbr.cbr_gemm_fp8(sp, aq, sa, bq, sb, bi, d, ws)
        half = torch.finfo(DT[out][0]).eps / 2 * (want.abs() + tol) + (2.0 ** -25 if out == "f16" else 0.0)
        assert ((d.double() - want).abs() <= tol + half).all()


@gpu
@pytest.mark.parametrize("k", [8000, 200000])
@pytest.mark.parametrize("kind,stated", [("normal", 1.4e-5), ("absolute", 2.5e-6), ("spread", 2.2e-5)])
def test_short_sums_are_as_near_as_the_header_says(k, kind, stated):
    """Twice the stated share of the norm, seen in the float parts of a split sum (before the output's
    rounding, which would hide it)."""
    m, n = 256, 192
    g = gen(k)

    def operand(rows, block):
        v = torch.randn(rows, k, generator=g, device="cuda")
        if kind == "absolute":
            v = v.abs()
        if kind == "spread":
            v = v * torch.exp(2 * torch.randn(rows, k, generator=g, device="cuda"))
        sp = cbr.make_quant_shape(rows, k, cbr.CBR_F32, block=block)
        q = torch.zeros(rows, sp.ldq, dtype=torch.uint8, device="cuda")
        s = torch.empty(-(-k // 128), -(-rows // block), device="cuda")
        cbr.cbr_fp8_quantize(sp, v, q, s)
        scale = s.double().t().repeat_interleave(block, 0)[:rows].repeat_interleave(128, 1)[:, :k]
        return q, s, q[:, :k].contiguous().view(torch.float8_e4m3fn).double() * scale
    (aq, sa, av), (bq, sb, bv) = operand(m, 1), operand(n, 128)
    sp = cbr.make_gemm_shape(m, n, k, d_type=cbr.CBR_F16, short_sums=True)
    ws = torch.empty(cbr.cbr_gemm_fp8_workspace_bytes(sp), dtype=torch.uint8, device="cuda")
    splits = ws.numel() // (4 * m * n)
    assert splits > 1
    cbr.cbr_gemm_fp8(sp, aq, sa, bq, sb, None, torch.empty(m, n, dtype=torch.float16, device="cuda"), ws)
    got = ws[:splits * 4 * m * n].view(torch.float32).view(splits, m, n).double().sum(0)
    want = av @ bv.t()
    assert (got - want).norm() <= 2 * stated * want.norm()


@gpu
@pytest.mark.parametrize("m", [96, 300, 2048])
def test_short_sums_keep_thirteen_bits(m):
    """A product of 2^-13 of the largest of its eight survives the largest's cancelling in another eight,
    in every tile."""
    n, k = 2048 if m == 2048 else 200, 128
    av, bv = torch.zeros(m, k, device="cuda"), torch.zeros(n, k, device="cuda")
    for place in range(1, 8):
        av.zero_(), bv.zero_()
        av[:, 8] = bv[:, 8] = 1.0
        av[:, 8 + place], bv[:, 8 + place] = 2.0 ** -6, 2.0 ** -7
        av[:, 64], bv[:, 64] = 1.0, -1.0
        sp = cbr.make_gemm_shape(m, n, k, d_type=cbr.CBR_BF16, short_sums=True)
        ws = torch.empty(max(16, cbr.cbr_gemm_fp8_workspace_bytes(sp)), dtype=torch.uint8, device="cuda")
        d = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        one = lambda r: torch.ones(1, r, device="cuda")  # noqa: E731
        cbr.cbr_gemm_fp8(sp, raw(av, torch.float8_e4m3fn, k), one(m), raw(bv, torch.float8_e4m3fn, k), one(-(-n // 128)), None,
                         d, ws)
        assert (d == 2.0 ** -13).all()
