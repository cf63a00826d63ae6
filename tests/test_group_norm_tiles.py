"""The group norm of images in tiles whose threads take several pixels, so that one is asked for while another is finished
and stored: in place, with values that are no numbers, with sums of whole numbers, and far from 0.  (tests/test_group_norm_layout.py
holds the layouts to that.)

Tolerance far from 0: a thread's running mean of at most 28 pixels is off by one half step of the largest value a pixel and two
at the end, at most 30 dx with dx = 2^-24 max |x|; over rows and columns of sums, no more than 128 dx for a group's mean.  The
squares are taken about these, which moves their mean by up to 4 * 30 dx times the standard deviation, and by the mean's square."""
import pytest
import torch

import test_group_norm as G

U = G.U
# eight channels in one group, in two, each for itself, in rows of whole eights and others, in fewer than eight
TILES = [(2, 200000, 64, 8), (2, 60000, 56, 4), (2, 33000, 128, 32), (3, 4000, 708, 4), (2, 40001, 45, 9), (3, 800000, 7, 7)]
MOST = 28


@pytest.mark.gpu
@pytest.mark.parametrize("size", TILES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(size, dtype):
    t = G.make(*size, dtype, "silu", 9)
    y, st = G.forward(t)
    dx, dw, db = G.backward(t, st)
    if size[1] < 100000:
        G.check_forward(t, y, st)
        G.check_backward(t, st, dx, dw, db)
    for name in ("dy", "x"):
        into = t[name].clone()
        got = G.backward({**t, name: into}, st, into=into)
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)
    x = t["x"].clone()
    _, st2 = G.forward({**t, "x": x}, y=x)
    assert torch.equal(x, y) and torch.equal(st2, st)


@pytest.mark.gpu
@pytest.mark.parametrize("size", TILES, ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_is_no_number_stays_in_its_group(size, bad):
    G.test_what_is_no_number_stays_in_its_group(size, bad)


@pytest.mark.gpu
@pytest.mark.parametrize("size", TILES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_value_is_summed_once(size, dtype):
    """db without an activation: sums of small whole numbers, exact in any order."""
    t = G.make(*size, dtype, "none", 5)
    _, st = G.forward(t)
    g = torch.Generator(device="cuda").manual_seed(3)
    t["dy"] = torch.randint(-8, 9, t["x"].shape, generator=g, device="cuda").to(t["x"].dtype)
    db = G.backward(t, st, dx=False, dw=False)[2]
    assert torch.equal(db.double(), t["dy"].double().sum((0, 1)))


@pytest.mark.gpu
@pytest.mark.parametrize("size", TILES, ids=str)
def test_far_from_zero(size):
    """4096 and a spread of 1.5: a difference of the squares' mean and the mean's square would leave nothing of it."""
    images, pixels, c, groups = size
    t = G.make(*size, "f32", "none", 4)
    t["x"] = t["x"] + 4096.0
    y, st = G.forward(t)
    x = t["x"].double()
    v = G.by_group(x, groups)
    mean = v.mean(2)
    var = (v - mean[:, :, None]).square().mean(2)
    dx = U * x.abs().max()
    dmean, dvar = 128 * dx, 4 * 30 * dx * var.sqrt() + (128 * dx) ** 2 + 256 * U * var
    inv = (var + G.EPS).rsqrt()
    dinv = inv * (0.5 * dvar / var + 4 * U)
    assert ((st[..., 0].double() - mean).abs() <= dmean).all()
    assert ((st[..., 1].double() - inv).abs() <= dinv).all()
    e = lambda q: G.spread(q, x, groups)  # noqa: E731
    xhat = (x - e(mean)) * e(inv)
    u = xhat * t["w"].double() + t["b"].double()
    tol = t["w"].double().abs() * (dmean * e(inv) + (x - e(mean)).abs() * e(dinv) + 5 * U * xhat.abs()) + 3 * U * (t["b"].double().abs() + u.abs())
    assert ((y.double() - u).abs() <= tol).all()


# one image of some 2^32 bytes in tiles of up to 2^31
@pytest.mark.gpu
@pytest.mark.parametrize("size", [(1, 5890, 359504, 359504), (1, 131008, 16384, 512)], ids=str)
def test_parts_of_almost_two_to_the_31_bytes(size):
    images, pixels, c, groups = size
    t = dict(images=images, pixels=pixels, c=c, groups=groups, dtype="bf16", act="silu")
    g = torch.Generator(device="cuda").manual_seed(1)
    t["x"], t["dy"] = (torch.empty(size[:3], dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    t["w"], t["b"] = 1 + 0.3 * torch.randn(c, generator=g, device="cuda"), 0.3 * torch.randn(c, generator=g, device="cuda")
    y, st = G.forward(t)
    dx, dw, db = G.backward(t, st)
    per, many = c // groups, 2 ** 23 // pixels // (c // groups)
    for first in (0, groups // 3, groups - many):   # some groups at a time
        ch, gr = slice(first * per, (first + many) * per), slice(first, first + many)
        s = {**t, "c": many * per, "groups": many, "w": t["w"][ch], "b": t["b"][ch], "x": t["x"][:, :, ch].contiguous(), "dy": t["dy"][:, :, ch].contiguous()}
        G.check_forward(s, y[:, :, ch], st[:, gr])
        G.check_backward(s, st[:, gr].contiguous(), dx[:, :, ch], dw[ch], db[ch])
