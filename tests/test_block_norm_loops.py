"""The block norm's backward where its threads go round: rows of more than 4096 channels (sixteen values
a thread), groups of threads that own several gate rows of several rows, partial chunks in both, and
dozens of turns.

Values are small whole numbers (statistics too: the backward takes what it is given), so every sum over
rows is exact in any order and has to come out equal: a row, a channel or a gate row missed or taken
twice shows.  With random values the tolerance is that of test_block_norm.py, whose chain of fp32
additions, min(rows, 1024) + 64, is longer than the kernel's here: a group of threads takes at most
rows / 256 + 1 turns, or with a gate as many more as a gate row has rows, and the lanes and waves that
share a channel are added in at most 16 more."""
import pytest
import torch

import conv2d_batchnorm_relu_amd as cbr
import test_block_norm as B

pytestmark = pytest.mark.gpu

# rows, channels, rows of a gate row (0: no gate)
SIZES = [
    (1500, 4099, 0), (1500, 4099, 1), (1500, 4099, 3), (1500, 8192, 0), (1500, 8192, 1), (999, 8191, 3), (1000, 5000, 500),
    (6000, 129, 2), (9000, 129, 3), (6002, 1001, 2), (9000, 1001, 3), (3000, 1001, 1), (60000, 7, 2), (60000, 7, 1),
    (5001, 1, 3), (20000, 2048, 0), (20000, 2048, 100), (6500, 520, 50), (12740, 256, 49), (98000, 256, 49), (262144, 64, 0),
    (100001, 20, 0), (40000, 1003, 0), (9000, 130, 9),
]


def whole(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").float()


@pytest.mark.parametrize("rows,c,rpg", SIZES, ids=str)
@pytest.mark.parametrize("stream,branch", [("bf16", "bf16"), ("f32", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("pre", ["none", "rms"])
def test_sums_of_whole_numbers(rows, c, rpg, stream, branch, pre):
    g = torch.Generator(device="cuda").manual_seed(rows + c)
    ts, tb = B.DT[stream][0], B.DT[branch][0]
    f, mean = whole(g, -3, 3, rows, c), whole(g, -1, 1, rows)
    gate = whole(g, -2, 2, rows // rpg, c) if rpg else None
    inv = torch.exp2(whole(g, -1, 1, rows))
    stats = torch.stack((mean, inv), 1).contiguous()
    # rms after the block; its weight and the residual scale are powers of two
    w, r = torch.exp2(whole(g, -1, 1, c)), torch.exp2(whole(g, -1, 1, c))
    b = whole(g, -2, 2, c)
    nhat = (f.double() - mean.double()[:, None]) * inv.double()[:, None]
    sp = cbr.make_block_shape(rows, c, rpg, cbr.CBR_NORM_RMS, B.KIND[pre], B.DT[stream][1], B.DT[branch][1], 0.5, 0.0, 0.0)
    new = lambda *s: torch.full(s, 77.0, device="cuda")  # noqa: E731
    dx, df = torch.empty(rows, c, dtype=ts, device="cuda"), torch.empty(rows, c, dtype=tb, device="cuda")
    dgate = torch.full_like(gate, 77.0, dtype=tb) if rpg else None
    dpw, dpb, dr = new(c), new(c), new(c)
    ws = torch.full((cbr.cbr_block_norm_workspace_bytes(sp),), 255, dtype=torch.uint8, device="cuda")
    gt = gate.to(tb) if rpg else None
    if pre == "none":
        dy = whole(g, -2, 2, rows, c)
        cbr.cbr_block_norm_backward(sp, dy.to(ts), None, None, f.to(tb), w, b, gt, r, None, stats, None, dx, df, dpw, dpb,
                                    dgate, dr, None, None, ws)
        d = dy.double()
        assert torch.equal(dx.double(), d)
        seg = lambda v: v.view(-1, rpg or rows, c).sum(1)  # noqa: E731
        s1, s0 = seg(d * nhat), seg(d)
        gd = gate.double() if rpg else torch.ones(1, c, dtype=torch.float64, device="cuda")
        each = w.double() * s1 + b.double() * s0
        if rpg:
            want = 0.5 * r.double() * each
            assert torch.equal(want.float().double(), want) and torch.equal(dgate, want.float().to(tb))
        t1, t0 = (gd * s1).sum(0), (gd * s0).sum(0)
        assert torch.equal(dpw.double(), 0.5 * r.double() * t1) and torch.equal(dpb.double(), 0.5 * r.double() * t0)
        assert torch.equal(dr.double(), 0.5 * (w.double() * t1 + b.double() * t0))
        return
    # dpre_w, dpre_b: sums of dh yhat and dh
    dh, y = whole(g, -2, 2, rows, c), whole(g, -3, 3, rows, c)
    dqw, dqb = new(c), new(c)
    cbr.cbr_block_norm_backward(sp, None, dh.to(tb), y.to(ts), f.to(tb), w, b, gt, r, None, stats, stats, dx, df, dpw, dpb,
                                dgate, dr, dqw, dqb, ws)
    yhat = (y.double() - mean.double()[:, None]) * inv.double()[:, None]
    assert torch.equal(dqw.double(), (dh.double() * yhat).sum(0)) and torch.equal(dqb.double(), dh.double().sum(0))


@pytest.mark.parametrize("rows,c,rpg", [(1500, 4099, 1), (1500, 4099, 3), (1500, 8192, 0), (1500, 8192, 3), (999, 8191, 3),
                                        (9000, 129, 3), (6002, 1001, 2), (60000, 7, 2), (6500, 520, 50), (20000, 1003, 0),
                                        (12740, 256, 49)], ids=str)
@pytest.mark.parametrize("post,pre", [("layer", "layer"), ("rms", "layer")])
@pytest.mark.parametrize("stream,branch", [("bf16", "bf16"), ("f32", "f16")])
def test_random_values(rows, c, rpg, post, pre, stream, branch):
    assert rows // 256 + 1 + rpg + 16 <= min(rows, 1024) + 64
    t = B.make(rows, c, stream, branch, post, pre, rpg, rows * 3 + c)
    if t["post_b"] is None:
        t["post_b"] = 0.2 * torch.randn(c, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    B.both(t)


def test_gradients_of_a_bf16_stream_against_the_forward_as_it_ran():
    """The backward gets the statistics of y before its rounding and y after it: its gradients stay within
    what that rounding (half a step, h = 2^-8 |y|) moves.  yhat is off by inv h, so the pre norm's part
    of D by at most inv (e_k m(g yhat) + yhat m(g e)) with e = inv h, on top of fp32's own and the
    outputs' half steps; dpre_w by sum |dh| e."""
    t = B.make(700, 256, "bf16", "bf16", "none", "layer", 0, 5, has_f=True)
    o = B.run_forward(t)
    g = B.run_backward(t, o)
    w = B.wide(t)
    r = B.forward64(w)                                    # y unrounded, its statistics, yhat
    inv, yh = r["qi"], r["yhat"]
    gw = w["dh"] * w["pre_w"]
    m1, m0 = (gw * yh).mean(1, keepdim=True), gw.mean(1, keepdim=True)
    d = w["dy"] + inv * (gw - m0 - yh * m1)
    e = inv * 2.0 ** -8 * r["y"].abs() + B.K * (yh.abs() + inv * r["y"].abs().mean(1, keepdim=True))
    ed = inv * (e * m1.abs() + (yh.abs() + e) * (gw.abs() * e).mean(1, keepdim=True))
    ed = ed + B.K * (d.abs() + B.lin(gw.abs(), yh.abs() + e, inv))
    assert ((g["dx"].double() - d).abs() <= 2.0 ** -8 * (d.abs() + ed) + ed).all()
    tol = (w["dh"].abs() * e).sum(0) + (700 + 64) * B.U * (w["dh"].abs() * (yh.abs() + e)).sum(0)
    assert ((g["pre_w"].double() - (w["dh"] * yh).sum(0)).abs() <= tol).all()


@pytest.mark.parametrize("c", [520, 1001, 2049, 4099, 8191])
@pytest.mark.parametrize("post,pre", [("none", "none"), ("none", "rms"), ("layer", "none"), ("layer", "layer")])
def test_in_place_rows_of_several_waves(c, post, pre):
    """y in x, h in f, dx in dy, df in f, where several waves share a row and (but for 520) its last chunk is a
    part of one, read as the row's last eight values: other waves may be storing those it drops."""
    t = B.make(700, c, "bf16", "bf16", post, pre, 7, c)
    o = B.run_forward(t)
    x, f = t["x"].clone(), t["f"].clone()
    o2 = B.run_forward({**t, "x": x, "f": f}, y=x, h=f if pre != "none" else None)
    assert torch.equal(o2["y"], o["y"]) and (pre == "none" or torch.equal(o2["h"], o["h"]))
    g = B.run_backward(t, o)
    dy, f = t["dy"].clone(), t["f"].clone()
    g2 = B.run_backward({**t, "dy": dy, "f": f}, o, dx=dy, df=f)
    assert all((g[k] is None and g2[k] is None) or torch.equal(g[k], g2[k]) for k in g)
