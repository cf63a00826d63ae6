"""The group norm with an activation against its definition in 64 bits, and its refusals.

Tolerances.  Sums are fp32: a sum's rounding is at most L half steps of 2^-24 of the sum of magnitudes, L the
additions on the longest way to the total: 8 channels of 24 pixels in a thread, 6 steps in a wave, at most 1024
threads' parts and 8192 channels' columns by 64 lanes (128 each) with 6 steps; no sum has more additions than
terms.  So L = min(terms, 192 + 6 + 1024 + 128 + 6), and for the tiles' means and squares twice that.  The
value itself, (x - mean) inv w + b, has five roundings of the terms, the sigmoid's argument moves its exponential by |u| half steps and
the sigmoid has six more (two of its hardware functions' whole steps); the derivative of the sigmoid's product
three times that.  An output adds half a step of its type.  Sums of small whole numbers are exact in fp32, so a
pixel left out or taken twice shows there."""
import ctypes
import random

import pytest
import torch

import conv2d_batchnorm_relu_amd as cbr

U = 2.0 ** -24
DT = {"bf16": (torch.bfloat16, cbr.CBR_BF16), "f16": (torch.float16, cbr.CBR_F16), "f32": (torch.float32, cbr.CBR_F32)}
ACT = {"none": cbr.CBR_ACT_NONE, "relu": cbr.CBR_ACT_RELU, "silu": cbr.CBR_ACT_SILU}
EPS = 1e-5


def longest(terms):
    return 2 * min(terms, 192 + 6 + 1024 + 128 + 6)


def by_group(v, groups):
    """[images, pixels, channels] as [images, groups, values of a group]."""
    n, p, c = v.shape
    return v.view(n, p, groups, c // groups).transpose(1, 2).reshape(n, groups, -1)


def spread(t, like, groups):
    """[images, groups] at every value of [images, pixels, channels]."""
    return t.repeat_interleave(like.shape[2] // groups, 1)[:, None, :].expand_as(like)


def act64(u, act):
    return u.clamp_min(0) if act == "relu" else u * torch.sigmoid(u) if act == "silu" else u


def slope64(u, act):
    if act == "none":
        return torch.ones_like(u)
    if act == "relu":
        return (u > 0).double()
    s = torch.sigmoid(u)
    return s * (1 + u * (1 - s))


def make(images, pixels, c, groups, dtype, act, seed, w=True, b=True, mean=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = DT[dtype][0]
    return dict(images=images, pixels=pixels, c=c, groups=groups, dtype=dtype, act=act,
                x=(rnd(images, pixels, c) * 1.5 + mean * rnd(c)).to(t), dy=rnd(images, pixels, c).to(t),
                w=1 + 0.3 * rnd(c) if w else None, b=0.3 * rnd(c) if b else None)


def shape_of(t):
    return cbr.make_group_norm_shape(t["images"], t["pixels"], t["c"], t["groups"], DT[t["dtype"]][1], ACT[t["act"]], EPS)


def workspace(sp, backward):
    n = cbr.cbr_group_norm_workspace_bytes(sp, backward)
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None


def forward(t, y=None, stats=True):
    sp = shape_of(t)
    y = torch.full_like(t["x"], float("nan")) if y is None else y
    st = torch.full((t["images"], t["groups"], 2), float("nan"), device="cuda") if stats else None
    cbr.cbr_group_norm_forward(sp, t["x"], t["w"], t["b"], y, st, workspace(sp, False))
    return y, st


def half_step(v, dtype):
    """Half a step of the type at v, and its smallest step."""
    f = torch.finfo(dtype)
    return f.eps / 2 * v.abs() + f.smallest_normal * f.eps


def check_forward(t, y, st):
    x, groups, act = t["x"].double(), t["groups"], t["act"]
    v = by_group(x, groups)
    n = v.shape[2]
    mean, mag = v.mean(2), v.abs().mean(2)
    var = (v - mean[:, :, None]).square().mean(2)
    inv = (var + EPS).rsqrt()
    dmean = (longest(n) + 2) * U * mag
    # the squares' mean moves by their sum's rounding and by the mean's own (dmean^2), inv by half of that and four steps
    dvar = (longest(n) + 4) * U * var + dmean.square() + 2 * dmean * longest(n) * U * var.sqrt()
    dinv = inv * (0.5 * dvar / (var + EPS) + 4 * U)
    if st is not None:
        assert ((st[..., 0].double() - mean).abs() <= dmean + U * mean.abs()).all()
        assert ((st[..., 1].double() - inv).abs() <= dinv).all()
    w = t["w"].double() if t["w"] is not None else torch.ones(t["c"], dtype=torch.float64, device="cuda")
    b = t["b"].double() if t["b"] is not None else torch.zeros_like(w)
    e = lambda q: spread(q, x, groups)  # noqa: E731
    xhat = (x - e(mean)) * e(inv)
    u = xhat * w + b
    du = w.abs() * (e(dmean) * e(inv) + (x - e(mean)).abs() * e(dinv) + 5 * U * xhat.abs()) + 2 * U * (b.abs() + u.abs())
    want = act64(u, act)
    tol = du if act != "silu" else 1.1 * du + (u.abs() * 1.5 + 6) * 2 * U * want.abs()
    assert ((y.double() - want).abs() <= tol + half_step(want.abs() + tol, y.dtype)).all()


def backward(t, st, dx=True, dw=True, db=True, into=None):
    sp = shape_of(t)
    new = lambda on: torch.full((t["c"],), float("nan"), device="cuda") if on else None  # noqa: E731
    dx = (torch.full_like(t["x"], float("nan")) if into is None else into) if dx else None
    dw, db = new(dw), new(db)
    cbr.cbr_group_norm_backward(sp, t["dy"], t["x"], t["w"], t["b"], st, dx, dw, db, workspace(sp, True))
    return dx, dw, db


def gradients64(t, st):
    """The formula with the statistics as they were saved; also the sums of magnitudes."""
    x, dy, groups = t["x"].double(), t["dy"].double(), t["groups"]
    mean, inv = (spread(st[..., i].double(), x, groups) for i in (0, 1))
    w = t["w"].double() if t["w"] is not None else torch.ones(t["c"], dtype=torch.float64, device="cuda")
    b = t["b"].double() if t["b"] is not None else torch.zeros_like(w)
    xhat = (x - mean) * inv
    u = xhat * w + b
    g = dy * slope64(u, t["act"])
    avg = lambda v: spread(by_group(v, groups).mean(2), x, groups)  # noqa: E731
    dx = inv * (w * g - avg(w * g) - xhat * avg(w * g * xhat))
    mags = inv, (w * g).abs(), avg((w * g).abs()), xhat.abs(), avg((w * g * xhat).abs())
    return dx, (g * xhat).sum((0, 1)), g.sum((0, 1)), mags, (g * xhat).abs().sum((0, 1)), g.abs().sum((0, 1)), u


def check_backward(t, st, dx, dw, db):
    want_x, want_w, want_b, (inv, wg, awg, xh, awgx), mag_w, mag_b, u = gradients64(t, st)
    n, per = t["pixels"] * t["c"] // t["groups"], t["pixels"]
    # g itself: xhat's two roundings (of x - mean, so in absolute terms of |x| + |mean| where they cancel: exact by
    # Sterbenz there) move u by three steps of |xhat w| + |b|; the slope by 1.1 times that and its own twelve steps.
    # near a value where the slope is small the dy part stays: bounded by |dy|
    dy = t["dy"].double().abs()
    w = t["w"].double().abs() if t["w"] is not None else 1.0
    b = t["b"].double().abs() if t["b"] is not None else 0.0
    dg = 0 * dy if t["act"] != "silu" else dy * (1.1 * 3 * U * (xh * w + b) + (3 * u.abs() + 24) * U)
    if t["act"] == "relu":
        # on which side of 0 a value within its rounding of it lies is not decided here
        edge = u.abs() <= 4 * U * (xh * w + b)
        dg = dg + torch.where(edge, dy, torch.zeros_like(dy))
    groups = t["groups"]
    avg = lambda v: spread(by_group(v, groups).mean(2), dg, groups)  # noqa: E731
    if dx is not None:
        tol = inv * (w * dg + avg(w * dg) + xh * avg(w * dg * xh) + U * (8 * wg + (longest(n) + 6) * (awg + xh * awgx)) + U * 8 * (awg + xh * awgx))
        assert ((dx.double() - want_x).abs() <= tol + half_step(want_x.abs() + tol, dx.dtype)).all()
    add = longest(per) + 4   # fp32 within an image; fp64 beyond
    if dw is not None:
        assert ((dw.double() - want_w).abs() <= (dg * xh).sum((0, 1)) + add * U * mag_w + 4 * U * mag_w).all()
    if db is not None:
        assert ((db.double() - want_b).abs() <= dg.sum((0, 1)) + add * U * mag_b).all()


SIZES = [(1, 1, 1, 1), (2, 1, 8, 8), (3, 7, 6, 3), (3, 5, 7, 1), (1, 49, 512, 32), (2, 196, 256, 32), (5, 225, 1001, 7), (2, 30, 40, 8),
         (3, 64, 24, 3), (2, 100, 320, 32), (4, 33, 48, 2), (1, 5000, 64, 32), (2, 4097, 64, 1), (1, 3, 8192, 1), (1, 1, 16384, 2),
         (70, 1, 16, 2), (300, 4, 64, 4), (1000, 1, 512, 32), (2, 12544, 72, 9), (1, 20011, 13, 13), (1, 9, 2048, 1), (1, 4, 8193, 8193),
         (2, 3, 8190, 4095), (9, 785, 640, 32), (1, 40, 5003, 5003), (2, 70000, 8, 2), (1, 33000, 128, 32), (4, 64, 2048, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(size):
    i = SIZES.index(size)
    dtype, act = ("bf16", "f32", "f16")[i % 3], ("silu", "relu", "none")[(i // 3) % 3]
    t = make(*size, dtype, act, 100 + i, w=i % 5 != 4, b=i % 4 != 3)
    y, st = forward(t)
    check_forward(t, y, st)
    y2, _ = forward(t, stats=False)
    assert torch.equal(y, y2)
    got = backward(t, st)
    check_backward(t, st, *got)
    again = backward(t, st)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("size", [(3, 50, 64, 8), (2, 77, 45, 9), (2, 9000, 32, 4)], ids=str)
def test_types_and_activations(dtype, act, size):
    t = make(*size, dtype, act, 7)
    y, st = forward(t)
    check_forward(t, y, st)
    check_backward(t, st, *backward(t, st))


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_whole_numbers_are_summed_exactly(size, dtype):
    """Means of whole numbers and, without an activation, db: every value once, every gradient once."""
    images, pixels, c, groups = size
    g = torch.Generator(device="cuda").manual_seed(3)
    t = make(*size, dtype, "none", 5)
    t["x"] = torch.randint(-8, 9, t["x"].shape, generator=g, device="cuda").to(t["x"].dtype)
    t["dy"] = torch.randint(-8, 9, t["x"].shape, generator=g, device="cuda").to(t["x"].dtype)
    _, st = forward(t)
    mean = by_group(t["x"].double(), groups).mean(2)
    # |sum| < 2^24; one division, and for images in tiles each tile's mean and the mean of those: three steps of a mean of at most 8.
    # (A value of 1 of the largest group's 280000 moves the mean by 60 of them.)
    assert ((st[..., 0].double() - mean).abs() <= U * mean.abs() + 3 * 8 * U).all()
    db = backward(t, st, dx=False, dw=False)[2]
    assert torch.equal(db.double(), t["dy"].double().sum((0, 1)))


def drawn(i):
    """Sizes over the whole range, of 4 million values at most."""
    r = random.Random(i)
    while True:
        cpg, groups = (int(2 ** r.uniform(0, t)) for t in (10, 11))
        images, pixels = (int(2 ** r.uniform(0, t)) for t in (9, 17))
        if images * pixels * cpg * groups <= 4e6:
            return images, pixels, cpg * groups, groups


# (the last two: sums of 128 and 150 KB)
@pytest.mark.gpu
@pytest.mark.parametrize("size", [drawn(i) for i in range(60)] + [(10, 13, 33155, 6631), (476, 2, 4470, 894)], ids=str)
def test_drawn_sizes(size):
    r = random.Random(str(size))
    for dtype in ("f32", r.choice(("bf16", "f16"))):
        t = make(*size, dtype, r.choice(list(ACT)), 17)
        y, st = forward(t)
        check_forward(t, y, st)
        check_backward(t, st, *backward(t, st))


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(3, 50, 64, 8), (2, 77, 45, 9), (2, 9000, 32, 4), (1, 10, 6, 2), (1, 20011, 13, 13)], ids=str)
def test_in_place_and_parts_of_the_gradients(size):
    t = make(*size, "bf16", "silu", 9)
    y, st = forward(t)
    dx, dw, db = backward(t, st)
    for which in ((True, False, False), (False, True, False), (False, False, True), (True, True, False)):
        got = backward(t, st, *which)
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, (dx, dw, db)))
    into = t["dy"].clone()
    got = backward({**t, "dy": into}, st, into=into)
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    into = t["x"].clone()
    got = backward({**t, "x": into}, st, into=into)
    assert torch.equal(got[0], dx) and torch.equal(got[2], db)
    x = t["x"].clone()
    forward({**t, "x": x}, y=x)
    assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(2, 60, 40, 8), (2, 60, 64, 8), (2, 9000, 32, 4), (3, 5, 14, 2)], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_is_no_number_stays_in_its_group(size, bad):
    images, pixels, c, groups = size
    t = make(*size, "bf16", "relu", 13)
    clean = t["x"].clone()
    hit = c // groups                       # the second group's first channel
    t["x"][1, pixels // 2, hit] = bad
    y, st = forward(t)
    per = c // groups
    assert y[1, :, per:2 * per].isnan().any() and st[1, 1, 1].isnan()
    y0, st0 = forward({**t, "x": clean})
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1, :, per:2 * per] = False
    assert torch.equal(y[keep], y0[keep])
    t["x"], t["dy"], t["act"] = clean, t["dy"].clone(), "silu"
    dx0 = backward(t, st0)[0]
    t["dy"][1, 3, hit] = float("nan")
    dx, dw, db = backward(t, st0)
    assert torch.equal(dx[keep], dx0[keep]) and dx[1, :, per:2 * per].isnan().any()
    wrong = dw.isnan() | db.isnan()
    assert not wrong[:hit].any() and not wrong[hit + 1:].any()


@pytest.mark.gpu
def test_equal_values_and_large_means():
    """A group of equal values normalises to b; values far from 0 keep their differences."""
    t = make(2, 300, 32, 4, "f32", "none", 1)
    t["x"].fill_(3.25)
    y, st = forward(t)
    assert torch.equal(y, t["b"].expand_as(y)) and (st[..., 0] == 3.25).all()
    t = make(2, 300, 32, 4, "f32", "none", 2)
    t["x"] = t["x"] + 1000.0
    y, st = forward(t)
    check_forward(t, y, st)
    x = t["x"].double().requires_grad_()
    v = by_group(x, 4)
    n = (v - v.mean(2, keepdim=True)) * (v.var(2, unbiased=False, keepdim=True) + EPS).rsqrt()
    want = n.view(2, 4, 300, 8).transpose(1, 2).reshape(2, 300, 32) * t["w"].double() + t["b"].double()
    # a mean of 1000 is held to 2^-15 of a standard deviation of 1.5; the values were rounded to 2^-14 before
    assert (y.double() - want).abs().max() <= 2.0 ** -12


def test_formula_against_differences():
    """The backward's formula against central differences of the definition, in 64 bits on the CPU."""
    g = torch.Generator().manual_seed(0)
    n, p, c, groups, h = 2, 5, 12, 3, 1e-6
    for act in ACT:
        x, dy = (torch.randn(n, p, c, generator=g, dtype=torch.float64) for _ in range(2))
        w, b = (torch.randn(c, generator=g, dtype=torch.float64) for _ in range(2))

        def y(x, w, b):
            v = by_group(x, groups)
            m, inv = v.mean(2), (v.var(2, unbiased=False) + EPS).rsqrt()
            return act64((x - spread(m, x, groups)) * spread(inv, x, groups) * w + b, act), torch.stack((m, inv), 2)
        st = y(x, w, b)[1]
        t = dict(x=x, dy=dy, w=w, b=b, c=c, groups=groups, act=act)
        dx, dw, db = gradients64(t, st)[:3]
        for v, d, at in ((x, dx, (1, 2, 5)), (x, dx, (0, 4, 11)), (w, dw, (3,)), (b, db, (7,))):
            v[at] += h
            up = (y(x, w, b)[0] * dy).sum()
            v[at] -= 2 * h
            down = (y(x, w, b)[0] * dy).sum()
            v[at] += h
            assert abs((up - down) / (2 * h) - d[at]) <= 1e-6 * (1 + d[at].abs())


# ---------------------------------------------------------------------------- refusals
FAKE = 0x10000


def fwd_status(sp, x=FAKE, y=2 * FAKE, ws=None, nbytes=0, w=None, b=None, st=None):
    return cbr._load().cbr_group_norm_forward(ctypes.byref(sp) if sp is not None else None, x, w, b, y, st, ws, nbytes, None)


def bwd_status(sp, dy=FAKE, x=2 * FAKE, st=3 * FAKE, dx=4 * FAKE, dw=None, db=None, ws=None, nbytes=0, w=None, b=None):
    return cbr._load().cbr_group_norm_backward(ctypes.byref(sp) if sp is not None else None, dy, x, w, b, st, dx, dw, db, ws, nbytes, None)


def test_refusals():
    S, OK = cbr.make_group_norm_shape, (2, 9, 64, 8)
    for bad, want in ((dict(images=0), 2), (dict(pixels=0), 2), (dict(pixels=-1), 2), (dict(channels=0), 2), (dict(groups=0), 2),
                      (dict(groups=7), 2), (dict(groups=128), 2), (dict(type=3), 7), (dict(type=9), 7), (dict(act=3), 7), (dict(act=-1), 7),
                      (dict(eps=-1.0), 7), (dict(eps=float("nan")), 7), (dict(eps=float("inf")), 7), (dict(images=2 ** 31), 3),
                      (dict(pixels=2 ** 31), 3), (dict(channels=16392, groups=1), 3), (dict(images=2 ** 31 - 1, pixels=2 ** 31 - 1), 3)):
        sp = S(*OK)
        for k, v in bad.items():
            setattr(sp, k, v)
        assert fwd_status(sp) == want and bwd_status(sp) == want, bad
        assert cbr.cbr_group_norm_workspace_bytes(sp) == 0 and cbr.cbr_group_norm_workspace_bytes(sp, True) == 0
    sp = S(*OK)
    assert fwd_status(None) == 1 and bwd_status(None) == 1
    assert fwd_status(sp, x=None) == 1 and fwd_status(sp, y=None) == 1
    assert bwd_status(sp, dy=None) == 1 and bwd_status(sp, x=None) == 1 and bwd_status(sp, st=None) == 1
    assert bwd_status(sp, dx=None) == 1                                   # no gradient wanted
    for k in ("x", "y", "w", "b", "st"):
        assert fwd_status(sp, **{k: FAKE + 8}) == 4, k
    for k in ("dy", "x", "st", "dx", "dw", "db", "w", "b"):
        assert bwd_status(sp, **{k: FAKE + 4}) == 4, k
    big = S(1, 100000, 64, 8)
    need = cbr.cbr_group_norm_workspace_bytes(big)
    assert need > 0 and fwd_status(big) == 5 and fwd_status(big, ws=FAKE, nbytes=need - 1) == 5 and fwd_status(big, ws=FAKE + 8, nbytes=need) == 4
    need = cbr.cbr_group_norm_workspace_bytes(sp, True)
    assert need > 0 and bwd_status(sp) == 5 and bwd_status(sp, ws=FAKE, nbytes=need - 1) == 5 and bwd_status(sp, ws=FAKE + 8, nbytes=need) == 4


@pytest.mark.gpu
def test_binding_refuses_tensors_that_do_not_fit():
    t = make(2, 9, 64, 8, "bf16", "none", 1)
    sp, y = shape_of(t), torch.empty_like(t["x"])
    for call in (lambda: cbr.cbr_group_norm_forward(sp, t["x"].float(), t["w"], t["b"], y),
                 lambda: cbr.cbr_group_norm_forward(sp, t["x"][:1], t["w"], t["b"], y),
                 lambda: cbr.cbr_group_norm_forward(sp, t["x"].cpu(), t["w"], t["b"], y),
                 lambda: cbr.cbr_group_norm_forward(sp, t["x"].transpose(1, 2), t["w"], t["b"], y),
                 lambda: cbr.cbr_group_norm_forward(sp, t["x"], t["w"][:32], t["b"], y),
                 lambda: cbr.cbr_group_norm_forward(sp, t["x"], t["w"].double(), t["b"], y),
                 lambda: cbr.cbr_group_norm_forward(sp, t["x"], t["w"], t["b"], y, torch.empty(8, device="cuda"))):
        with pytest.raises(cbr.CbrError):
            call()
