"""The 4-bit product's sums, tightly.  A group of 32 values is exact: its products are multiples of a quarter, its sum below
2^13 of them.  The matrix instruction adds groups one after another to an fp32 sum.  Measured over every order of a small and a
large group: the smaller of the two keeps the bits down to 2^-22 of the larger (a large sum a last place, 2^-23; a sum below a large
product, which is aligned by its largest possible value, twice that).  So every group but the first costs at most 2^-22 of the
magnitudes so far.  The eight waves of few rows and the splits are added in fp32 (2^-24 each).  A result in f32 without a bias is
within (2 (groups - 1) + (waves + splits) / 2) 2^-23 of the sum of magnitudes."""
import pytest
import torch

import conv2d_batchnorm_relu_amd as cbr
import test_fp4 as F

cdiv = F.cdiv


def additions(m, n, k):
    """fp32 additions behind the instructions: eight waves with a run of 512 values each or more, and the splits."""
    need = cbr.cbr_gemm_fp4_workspace_bytes(cbr.make_gemm_fp4_shape(m, n, k, cbr.CBR_F32))
    splits = need // (4 * m * n) if need else 1
    return (min(8, cdiv(k, 512)) - 1 if m <= 64 else 0) + (splits if splits > 1 else 0)


def check(m, n, k, a, b, groups=None):
    d = F.product(m, n, k, a, b, "f32").double()
    va, vb = F.decode64(*a, k), F.decode64(*b, k)
    want, mag = va @ vb.t(), va.abs() @ vb.abs().t()
    tol = (2 * ((groups or cdiv(k, 32)) - 1) + additions(m, n, k) / 2) * 2.0 ** -23 * mag
    assert ((d - want).abs() <= tol).all()


# few rows in each height, tiles of every size, in one round and in more
SIZES = [(1, 40), (16, 300), (30, 77), (64, 130), (65, 63), (200, 130), (600, 700), (2100, 1100), (9001, 800)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_a_group_is_exact(size):
    m, n = size
    for k in (1, 31, 32):
        a, b = F.operand(m, k, 1, 20), F.operand(n, k, 2, 20)
        d = F.product(m, n, k, a, b, "f32").double()
        assert torch.equal(d, F.decode64(*a, k) @ F.decode64(*b, k).t())


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("spread", [0, 6, 12, 20])
def test_few_groups_of_any_scales(size, spread):
    m, n = size
    for k in (64, 96, 128, 256, 500, 512):
        check(m, n, k, F.operand(m, k, k + spread, spread), F.operand(n, k, k + 1, spread))


def ladder(rows, k, first, seed):
    """Group `first` holds one value, 2^0 .. 2^47 by row; the others random ones, or (second half of the rows) a sum of 63
    products of 1: just short of a power of two, so that much of it may be cut off."""
    g = F.gen(seed)
    groups = cdiv(k, 32)
    code = torch.randint(1, 8, (rows, groups, 32), generator=g, device="cuda").to(torch.uint8)
    code[rows // 2:] = 0
    for i, v in enumerate((7, 7, 7, 7, 7, 7, 7, 7, 7, 7, 5)):        # 10 * 6 + 3 = 63
        code[rows // 2:, :, i] = v
    code[:, first] = 0
    code[:, first, 5] = 2
    code = code.view(rows, -1)
    q = (code[:, ::2] | code[:, 1::2] << 4).contiguous()
    e = torch.full((rows, cdiv(k, 128) * 4), 127, device="cuda")
    e[:, first] += torch.arange(rows, device="cuda") % 48
    return q, e.to(torch.uint8).view(rows, -1, 4).transpose(0, 1).contiguous()


@pytest.mark.gpu
@pytest.mark.parametrize("m,k", [(48, 512), (64, 2048), (192, 256), (192, 512), (1536, 1024)])
def test_what_groups_lose_below_a_large_one(m, k):
    n = 300
    ones = torch.full((n, cdiv(k, 32) * 16), 0x22, dtype=torch.uint8, device="cuda"), torch.full((cdiv(k, 128), n, 4), 127, dtype=torch.uint8, device="cuda")
    for first in (0, 1, 2, 4, cdiv(k, 32) - 1):
        a = ladder(m, k, first, first)
        check(m, n, k, a, ones)
        check(m, n, k, a, F.operand(n, k, 7))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [48, 960])
@pytest.mark.parametrize("sign", [0, 8])
def test_two_groups_in_every_order(m, sign):
    """A single value 2^0 .. 2^47 times as large as another group's, before and behind it, in one instruction and in two."""
    n, k = 128, 256
    g = F.gen(m)
    for large in range(8):
        for small in range(8):
            if small == large:
                continue
            code = torch.zeros(m, 8, 32, dtype=torch.uint8, device="cuda")
            part = torch.rand(m, 32, generator=g, device="cuda") < torch.rand(m, 1, generator=g, device="cuda")
            code[:, small] = torch.randint(1, 8, (m, 32), generator=g, device="cuda").to(torch.uint8) * part + sign
            code[:, large, 5] = torch.randint(1, 8, (m,), generator=g, device="cuda").to(torch.uint8)
            e = torch.full((m, 8), 127, device="cuda")
            e[:, large] += torch.arange(m, device="cuda") % 48
            code = code.view(m, k)
            a = code[:, ::2] | code[:, 1::2] << 4, e.to(torch.uint8).view(m, 2, 4).transpose(0, 1).contiguous()
            q, s = F.operand(n, k, 2)
            check(m, n, k, a, (q & 0x77, s), groups=2)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(5, 300, 20000), (64, 256, 50176), (300, 260, 20000), (1024, 256, 50176)], ids=str)
def test_long_sums_of_one_sign(m, n, k):
    (qa, sa), (qb, sb) = F.operand(m, k, 1, 2), F.operand(n, k, 2, 2)
    check(m, n, k, (qa & 0x77, sa), (qb & 0x77, sb))
