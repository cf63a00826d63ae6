"""The 8-bit product with scales of any size: a_scale * b_scale, or a sum times one of them, may lie
outside fp32 (or among its subnormal numbers) where the result does not.

Each row and column has an exponent of its own and the blocks of k vary around it, so one tile holds
every combination.  Tolerance: 128 products of a block, the blocks, the splits' parts and the scaling
(16), each a rounding of 2^-24 of the magnitudes that enter; a result below 2^-126 is rounded to a
multiple of 2^-149 once a block and once a part; then half a step of the output."""
import pytest
import torch

import conv2d_batchnorm_relu_amd as cbr

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, cbr.CBR_BF16), "f32": (torch.float32, cbr.CBR_F32)}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def product(av, sa, bv, sb, block, out, short=False):
    """av [m][k], bv [n][k]: values that e4m3 holds."""
    (m, k), n = av.shape, bv.shape[0]
    ld = -(-k // 16) * 16

    def raw(v):
        q = torch.full((v.shape[0], ld), 0x7F, dtype=torch.uint8, device="cuda")
        q[:, :k] = v.to(torch.float8_e4m3fn).view(torch.uint8)
        return q
    sp = cbr.make_gemm_shape(m, n, k, d_type=DT[out][1], b_block=block, lda=ld, ldb=ld, short_sums=short)
    ws = torch.full((max(16, cbr.cbr_gemm_fp8_workspace_bytes(sp)),), 255, dtype=torch.uint8, device="cuda")
    d = torch.empty(m, n, dtype=DT[out][0], device="cuda")
    cbr.cbr_gemm_fp8(sp, raw(av), sa, raw(bv), sb, None, d, ws)
    return d


# few rows (three forms), 64- and 128-wide tiles of both depths, split sums
SIZES = [(5, 40, 300), (20, 130, 2100), (60, 70, 300), (150, 200, 300), (300, 200, 3990), (2000, 1999, 400), (4000, 4001, 260),
         (701, 1001, 9001)]


@pytest.mark.parametrize("m,n,k", SIZES, ids=str)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("out,short", [("f32", False), ("bf16", False), ("bf16", True)])
def test_scales_of_any_size(m, n, k, block, out, short):
    g = gen(m + n + k)
    kb, nb = -(-k // 128), -(-n // block)
    if short:    # products that the shorter sums hold exactly
        val = lambda r: torch.randint(-4, 5, (r, k), generator=g, device="cuda").float()  # noqa: E731
    else:
        val = lambda r: (torch.randn(r, k, generator=g, device="cuda") * torch.exp2(torch.randint(  # noqa: E731
            -6, 7, (r, k), generator=g, device="cuda").float())).clamp(-448, 448).to(torch.float8_e4m3fn).float()

    def scales(r):
        e = torch.randint(-110, 111, (1, r), generator=g, device="cuda") + torch.randint(-3, 4, (kb, r), generator=g, device="cuda")
        return torch.ldexp(1 + torch.rand(kb, r, generator=g, device="cuda"), e)
    av, bv, sa, sb = val(m), val(n), scales(m), scales(nb)
    d = product(av, sa, bv, sb, block, out, short).double()
    each = torch.arange(k, device="cuda") // 128
    ra = av.double() * sa.double()[each].t()
    rb = bv.double() * sb.double()[each].t().repeat_interleave(block, 0)[:n]
    want, mag = ra @ rb.t(), ra.abs() @ rb.abs().t()
    tol = (128 + kb + 16) * 2.0 ** -24 * mag + (kb + 16) * 2.0 ** -149
    if out == "bf16":
        tol = tol + 2.0 ** -8 * (want.abs() + tol) + 2.0 ** -126
    held = mag < 2.0 ** 127                       # beyond that parts of the sum may overflow
    assert held.float().mean() > 0.5
    bad = held & ~((d - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4], d[bad][:4], want[bad][:4])


@pytest.mark.parametrize("m", [5, 40, 150, 2000])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("short", [False, True])
def test_zero_sums_stay_zero_and_infinite_scales_are_nan(m, block, short):
    g = gen(m)
    n, k = 1999 if m == 2000 else 136, 384
    bv = torch.randint(-4, 5, (n, k), generator=g, device="cuda").float()
    av = torch.zeros(m, k, device="cuda")
    av[::2, 128:] = 1.0                                           # odd rows: zeros throughout
    sa, sb = torch.full((3, m), 2.0 ** 100, device="cuda"), torch.full((3, -(-n // block)), 2.0 ** 100, device="cuda")
    sa[1:] = sb[1:] = 1.0
    sa[0, 4] = float("inf")
    d = product(av, sa, bv, sb, block, "bf16", short)
    want = (av[:, 128:] @ bv[:, 128:].t()).bfloat16()
    keep = [i for i in range(m) if i != 4]
    assert torch.equal(d[keep], want[keep])
    assert d[4].isnan().all()                                     # an infinite scale times a sum of zero


@pytest.mark.parametrize("m", [5, 20, 60, 150, 2000])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("short", [False, True])
@pytest.mark.parametrize("big,ea,eb", [(448.0, -118, 118), (448.0, 118, -118), (2.0 ** -9, 110, -126), (2.0 ** -9, -126, 110)])
def test_opposite_scales(m, block, short, big, ea, eb):
    """A sum times one scale alone is past fp32's range, or among its subnormal numbers.  One value a
    block, so that the result is that product, rounded for the output only."""
    n, k = 1999 if m == 2000 else 136, 384
    av, bv = torch.zeros(m, k, device="cuda"), torch.zeros(n, k, device="cuda")
    av[:, 5::128] = bv[:, 5::128] = big
    f = lambda r: 1 + torch.arange(3 * r, device="cuda").view(3, r) % 7 / 8  # noqa: E731
    sa, sb = torch.ldexp(f(m), torch.tensor(ea, device="cuda")), torch.ldexp(f(-(-n // block)), torch.tensor(eb, device="cuda"))
    want = ((sa.double() * big).t() @ (sb.double() * big).repeat_interleave(block, 1)[:, :n])
    assert torch.equal(want.float().double(), want)
    assert torch.equal(product(av, sa, bv, sb, block, "bf16", short), want.float().bfloat16())
