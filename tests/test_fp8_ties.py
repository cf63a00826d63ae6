"""Rounding of fp32 values to 8 bits at, and next to, the middle of two 8-bit ones.

a is a group's largest value, t = v fmax / a.  fmax is 7 times a power of two, so v = x a / (7 2^p) has
t = x 2^e with x of one bit more than the format holds (odd): exactly between two 8-bit values where
7 divides a, and 1 / (x a) of it (some 2^-28, four bits below fp32's own) off where
x a = +-1 (mod 7 2^p).  The definition is computed in 64 bits: v fmax is exact there, and the quotient's
rounding of 2^-53 is far below that distance."""
import pytest
import torch

import conv2d_batchnorm_relu_amd as cbr
from test_fp8 import F8, quant64, quantize, same

pytestmark = pytest.mark.gpu


def groups(fmt, off, count, seed):
    """count rows of 128 values whose first is the largest, a (whole, 24 bits); each row the values of one x
    at all exponents where t is normal or subnormal, with both signs."""
    _, _, fmax, bits, low = F8[fmt]
    g = torch.Generator().manual_seed(seed)
    xs = [x for x in range(2 ** (bits + 1) + 1, 2 ** (bits + 2), 2) if off == 0 or x % 7]
    rows = []
    for i in range(count):
        x = xs[i % len(xs)]
        lead = x.bit_length() - 1
        if off == 0:
            # a = 7 j with x j of at most 24 bits
            j = int(torch.randint(2 ** 17, 2 ** 24 // x, (1,), generator=g)) | 1
            a, v = 7 * j, x * j
            while a < 2 ** 23:
                a *= 2
            v = float(v)
        else:
            mod = 7 * 2 ** (lead - 1)
            r = off * pow(x, -1, mod) % mod
            a = 2 ** 23 + int(torch.randint(0, 2 ** 22 // mod, (1,), generator=g)) * mod * 2
            a += (r - a) % mod
            assert (x * a - off) % mod == 0 and a < 2 ** 24
            v = float((x * a - off) // mod)
            assert v < 2 ** 24
        row = torch.zeros(128, dtype=torch.float64)
        row[0] = a
        # largest power of two that keeps |v| <= a, then downwards (exact in fp32: only the exponent moves)
        while v > a:
            v /= 2
        while 2 * v <= a:
            v *= 2
        for k in range(1, 64):
            row[2 * k - 1], row[2 * k] = v * 2.0 ** -(k % 24), -v * 2.0 ** -(k % 24)
        rows.append(row)
    t = torch.stack(rows)
    assert torch.equal(t.float().double(), t)
    return t.float()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("off", [0, 1, -1])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -60, 2.0 ** 90])
def test_ties_of_fp32_values(fmt, off, scale):
    v = (groups(fmt, off, 256, 3) * scale).cuda()
    want = quant64(v, fmt, 1)[0]
    _, q, _ = quantize(v, fmt)
    assert same(q, want)
    _, q, _ = quantize(v.t().contiguous(), fmt, transpose=True)
    assert same(q, want)
    # a 128 x 128 block for each row
    blocks = torch.zeros(64 * 128, 128, device="cuda")
    blocks[::128] = v[:64]
    want = quant64(blocks, fmt, 128)[0]
    assert same(want[::128], quant64(v[:64], fmt, 1)[0])
    _, q, _ = quantize(blocks, fmt, block=128)
    assert same(q, want)
    _, q, _ = quantize(blocks.t().contiguous(), fmt, transpose=True, block=128)
    assert same(q, want)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_random_fp32_values_are_rounded_as_defined(fmt):
    """Four million values with all 24 bits: some lie within fp32's rounding of a middle."""
    g = torch.Generator(device="cuda").manual_seed(1)
    v = torch.randn(2048, 2048, generator=g, device="cuda") * torch.exp(2 * torch.randn(2048, 2048, generator=g, device="cuda"))
    _, q, _ = quantize(v, fmt)
    assert same(q, quant64(v, fmt, 1)[0])
