"""Infinities, NaN and the smallest scales in every form of the quantiser, value by value against the
definition in 64 bits; and a split product on a stream of its own."""
import pytest
import torch

import conv2d_batchnorm_relu_amd as cbr
from test_fp8 import F8, gen, operand, quant64, quantize, same, scale_close

pytestmark = pytest.mark.gpu

# signalling and quiet NaN of each source type, with both signs, as the integers that hold them
NANS = {"bf16": (torch.bfloat16, torch.int16, (0x7F81, 0x7FC0, 0xFF81 - 0x10000)),
        "f16": (torch.float16, torch.int16, (0x7C01, 0x7E00, 0xFC01 - 0x10000)),
        "f32": (torch.float32, torch.int32, (0x7F800001, 0x7FC00000, 0xFF800001 - 0x100000000))}


@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("transpose,block", [(False, 1), (True, 1), (False, 128), (True, 128)])
@pytest.mark.parametrize("rows,cols", [(300, 390), (256, 384)])
def test_special_values(src, fmt, transpose, block, rows, cols):
    dt, it, nans = NANS[src]
    v = torch.randn(rows, cols, generator=gen(rows), device="cuda").to(dt)
    v[5, :128] = 0                                                  # a group of zeros, in one form or the other
    v[128:256, 256] = -0.0
    tiny = {"bf16": 1e-40, "f16": 6e-8, "f32": 1e-45}[src]          # subnormal values
    v[128:256, 128:256] = tiny
    v[131, 3], v[2, 300] = float("inf"), float("-inf")
    big = {"bf16": 3.3e38, "f16": 65504.0, "f32": 3.4e38}[src]
    v[70, 140], v[71, 140] = big, -big
    bits = v.view(it)
    for i, n in enumerate(nans):
        bits[i, 20 + i] = n
        bits[200 + i, 130] = n
        bits[128 + i, 380] = n
    # NaN right behind the largest value of its row, its column and its block
    v[8, 40] = v[16, 64] = v[24, 95] = 9.0
    for i, n in enumerate(nans):
        r, c = ((8, 40), (16, 64), (24, 95))[i]
        bits[r, c + 1] = bits[r + 1, c] = n
    # a group of nothing but NaN: its scale is the smallest
    bits[129, 256:384] = nans[0]
    vv = v.t() if transpose else v
    bad = vv.isnan()
    want, scale = quant64(torch.where(bad, torch.zeros_like(vv), vv), fmt, block)
    _, q, s = quantize(v, fmt, transpose, block)
    assert torch.equal(s.isinf(), scale.isinf()) and int(s.isinf().sum()) == 2
    fin = scale.isfinite()
    assert scale_close(s[fin], scale[fin])
    assert q[bad].isnan().all()
    assert same(q[~bad], want[~bad])
    if block == 1 and not transpose:
        assert s[2, 129] == 2.0 ** -126 and s[0, 5] == 2.0 ** -126


@pytest.mark.parametrize("out", [cbr.CBR_F32, cbr.CBR_BF16])
def test_split_product_on_another_stream(out):
    """With a workspace of its own, filled before the stream starts and kept until it is done."""
    m, n, k = 256, 256, 20000
    dt = torch.float32 if out == cbr.CBR_F32 else torch.bfloat16
    sp = cbr.make_gemm_shape(m, n, k, d_type=out, b_block=1)
    need = cbr.cbr_gemm_fp8_workspace_bytes(sp)
    assert need > 0
    x = [*operand(torch.randn(m, k, generator=gen(1), device="cuda"), "e4m3", 1)[:2],
         *operand(torch.randn(n, k, generator=gen(2), device="cuda"), "e4m3", 1)[:2]]
    ws, other = (torch.full((need,), fill, dtype=torch.uint8, device="cuda") for fill in (0, 255))
    d, e = torch.empty(m, n, dtype=dt, device="cuda"), torch.full((m, n), 7.0, dtype=dt, device="cuda")
    cbr.cbr_gemm_fp8(sp, *x, None, d, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cbr.cbr_gemm_fp8(sp, *x, None, e, other, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(d, e) and torch.equal(ws, other)
    # both at once, on other operands, with everything allocated and filled before either starts
    y = [*operand(torch.randn(m, k, generator=gen(3), device="cuda"), "e4m3", 1)[:2],
         *operand(torch.randn(n, k, generator=gen(4), device="cuda"), "e4m3", 1)[:2]]
    want = torch.empty_like(d)
    cbr.cbr_gemm_fp8(sp, *y, None, want, ws)
    ws.fill_(255), other.fill_(255)
    pairs = [(torch.empty_like(d), torch.empty_like(d)) for _ in range(8)]
    torch.cuda.synchronize()
    for p, r in pairs:
        cbr.cbr_gemm_fp8(sp, *x, None, p, ws)
        cbr.cbr_gemm_fp8(sp, *y, None, r, other, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(p, d) and torch.equal(r, want) for p, r in pairs)


@pytest.mark.parametrize("m,n,k,short", [(40, 70, 300, False), (300, 200, 777, False), (2000, 1990, 300, False),
                                         (4000, 4001, 130, True)], ids=str)
def test_longest_strides(m, n, k, short):
    """Rows 2^23 bytes apart: a tile's 256 rows are 2^31 bytes, its offsets just below.  Small whole numbers:
    exact but for the output's rounding."""
    ld = 1 << 23
    g = gen(k)
    if m > 2000:
        torch.cuda.empty_cache()
    val = lambda r: torch.randint(-4, 5, (r, k), generator=g, device="cuda").float()  # noqa: E731
    av, bv = val(m), val(n)

    def raw(v):
        q = torch.empty(v.shape[0], ld, dtype=torch.uint8, device="cuda")
        q[:, :k] = v.to(torch.float8_e4m3fn).view(torch.uint8)
        q[:, k:k + 256] = 0x7F                                     # NaN behind the row's values
        return q
    kb = -(-k // 128)
    sa, sb = torch.ones(kb, m, device="cuda"), torch.ones(kb, -(-n // 128), device="cuda")
    sp = cbr.make_gemm_shape(m, n, k, lda=ld, ldb=ld, short_sums=short)
    ws = torch.empty(max(16, cbr.cbr_gemm_fp8_workspace_bytes(sp)), dtype=torch.uint8, device="cuda")
    d = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    cbr.cbr_gemm_fp8(sp, raw(av), sa, raw(bv), sb, None, d, ws)
    assert torch.equal(d, (av.double() @ bv.double().t()).float().bfloat16())
