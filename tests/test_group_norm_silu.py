"""SiLU and its slope over the whole range of its argument u, forward and backward.

With w = 0 the argument is b itself, and with one gradient of 1 among zeros db is the slope, so both come out of the kernels
alone.  Tolerances in half steps U = 2^-24, s the sigmoid: v = -log2(e) u is off by one and the constant by less than a
quarter, which moves 2^v by 1.25 |u|; the hardware's 2^v and reciprocal are within two each, every other operation within one.
  s:        (1 - s) (1.25 |u| + 2) + 3           (2^v is its part 1 - s of 1 + 2^v; the sum; the reciprocal)
  y = u s:  that and two (v, the product)
  u (1 - s) = v 2^v s:  s (1.25 |u| + 2) + 5     (v, the sum, the reciprocal, the product)
  slope = s h, h = 1 + u (1 - s):  those of s, of h (its term's as a part of h, and one), and three products.
Values and slopes below 2^-119 may be 0: the reciprocal of more than 2^126 may."""
import pytest
import torch

import test_group_norm as G

U = G.U
TINY = 2.0 ** -118
ARGS = [0.0, 1e-30, 1e-3, 0.25, 0.5, 1.0, 1.278, 2.0, 3.0, 4.0, 5.0, 6.0, 7.0] + [8 + 0.125 * i for i in range(88)]
ARGS += [20.0, 25.0, 30.0, 40.0, 60.0, 80.0, 86.0, 87.0, 87.5, 88.0, 88.5, 89.0, 100.0, 128.0, 1e3, 1e4, 1e6, 1e10, 1e20, 1e30, 1.7e38]


def sigmoid_steps(u, s):
    return (1 - s) * (1.25 * u.abs() + 2) + 3


def check_value(y, u):
    s = torch.sigmoid(u)
    assert ((y.double() - u * s).abs() <= U * (u * s).abs() * (sigmoid_steps(u, s) + 2) + TINY).all()


def slope_and_bound(u):
    s = torch.sigmoid(u)
    t = u * torch.sigmoid(-u)
    h = 1 + t
    bound = U * (s * h.abs() * (sigmoid_steps(u, s) + 3) + s * (t.abs() * (s * (1.25 * u.abs() + 2) + 5) + h.abs()))
    return s * h, torch.where(s < 2.0 ** -118, torch.zeros_like(u), bound) + TINY


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(1, 3), (2, 60), (1, 40000)], ids=str)   # held whole, and in tiles
@pytest.mark.parametrize("cpg", [1, 8, 14])
def test_every_argument(size, cpg):
    u = torch.tensor(ARGS, device="cuda")
    u = torch.cat((u, -u))
    u = torch.cat((u, u[:-u.numel() % 56]))
    images, pixels, c = *size, u.numel()
    t = G.make(images, pixels, c, c // cpg, "f32", "silu", 1)
    t["w"], t["b"] = torch.zeros(c, device="cuda"), u
    y, st = G.forward(t)
    check_value(y, u.double().expand_as(y))
    t["dy"].zero_()
    t["dy"][images - 1, pixels // 2] = 1
    db = G.backward(t, st)[2]
    want, bound = slope_and_bound(u.double())
    assert ((db.double() - want).abs() <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(2, 60, 64, 8), (2, 60, 56, 4), (1, 40000, 48, 6), (1, 40000, 42, 3), (2, 50, 40, 20)], ids=str)
def test_gradients_at_large_arguments(size):
    """dx where b takes whole groups far to either side."""
    images, pixels, c, groups = size
    per = c // groups
    t = G.make(*size, "f32", "silu", 2)
    far = torch.tensor([14.0, 17.0, 1e3, 1e6, -14.0, -1e3, 1e30], device="cuda")
    t["b"] = far[torch.arange(groups, device="cuda") % 7].repeat_interleave(per)
    y, st = G.forward(t)
    dx = G.backward(t, st)[0]
    want, _, _, (inv, wg, awg, xh, awgx), _, _, u = G.gradients64(t, st)
    s = torch.sigmoid(u)
    # |slope'|, and an argument off by three steps of its terms
    turn = (s * (1 - s) * (2 + u.clamp(-1e3, 1e3) * (1 - 2 * s))).abs()
    w, b, dy = t["w"].double().abs(), t["b"].double().abs(), t["dy"].double().abs()
    dg = dy * (slope_and_bound(u)[1] + 1.1 * turn * 3 * U * (xh.abs() * w + b))
    avg = lambda v: G.spread(G.by_group(v, groups).mean(2), dg, groups)  # noqa: E731
    add = G.longest(pixels * per) + 14
    tol = inv * (w * dg + avg(w * dg) + xh * avg(w * dg * xh) + U * (8 * wg + add * (awg + xh * awgx)))
    assert ((dx.double() - want).abs() <= tol + U * (want.abs() + tol) + TINY).all()
