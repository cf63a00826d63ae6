"""How the group norm lays calls out, on the CPU: its planner is compiled for the host and asked for the layouts of sizes
over all that include/cbr.h allows.  Whatever the size, the byte offsets that the kernels form inside a part of a tensor
are 32-bit ones, so none may reach 2^31: not those of pixels past the part's end either, whose loads are switched off."""
import ctypes
import math
import os
import random
import subprocess

import pytest

import conv2d_batchnorm_relu_amd as cbr
from conv2d_batchnorm_relu_amd import build

FIELDS = "V P ipw ng chunks tiles k pre lds".split()
DRIVER = """
#include "%s/group_norm_plan.cpp"
extern "C" void layout(const cbr_group_norm_shape *s, int backward, long long *o)
{
    using namespace cbr::gnorm;
    const Geo g = plan_group_norm(*s, backward != 0);
    const int cpg = s->channels / s->groups;
    const long long v[] = {g.V, g.P, g.ipw, g.ng, g.chunks, g.tiles, g.k, g.pre,
                           backward ? bwd_floats(g, cpg) : sum_floats(g, split_of(cpg), 1)};
    for (int i = 0; i < 9; ++i) o[i] = v[i];
}
"""


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    d = tmp_path_factory.mktemp("layout")
    src, so = d / "driver.cpp", d / "driver.so"
    src.write_text(DRIVER % build.CSRC)
    subprocess.run([build.HIPCC, "-O2", "-std=c++17", "-fPIC", "-shared", "-x", "hip", "--offload-host-only",
                    "-Wno-unused-function", str(src), "-o", str(so)], check=True, capture_output=True, env=dict(os.environ))
    fn = ctypes.CDLL(str(so)).layout
    out = (ctypes.c_longlong * len(FIELDS))()

    def ask(images, pixels, channels, groups, dtype=cbr.CBR_BF16, backward=False, act=cbr.CBR_ACT_SILU):
        sp = cbr.make_group_norm_shape(images, pixels, channels, groups, dtype, act)
        fn(ctypes.byref(sp), int(backward), out)
        return dict(zip(FIELDS, out))
    return ask


def size_of(dtype):
    return 4 if dtype == cbr.CBR_F32 else 2


def offsets(g, pixels, channels, size):
    """One past the largest byte offset that a workgroup forms: a thread's first pixel and `step` times the turn; tiles ask for two turns
    past the last."""
    step = g["P"] * channels * size
    if g["tiles"] > 1:
        return (g["k"] + 2) * step
    return ((g["ipw"] - 1) * pixels + g["k"] * g["P"]) * channels * size


def check(layout, images, pixels, channels, groups, dtype, backward):
    g = layout(images, pixels, channels, groups, dtype, backward)
    size = size_of(dtype)
    what = (images, pixels, channels, groups, dtype, backward, g)
    assert g["V"] > 0 and g["k"] > 0 and 1 <= g["V"] * g["P"] * g["ipw"] <= 1024, what
    assert g["tiles"] * g["P"] * g["k"] >= pixels > (g["tiles"] - 1) * g["P"] * g["k"], what     # no tile without a pixel
    assert g["chunks"] * g["ng"] >= groups > (g["chunks"] - 1) * g["ng"], what
    assert 8 * g["V"] >= g["ng"] * (channels // groups), what
    assert 4 * g["lds"] <= 160 * 1024, what
    if backward and g["tiles"] > 1:   # the second kernel's sums
        parts = max(1, min(g["P"] // 16, 8))
        assert 4 * (16 * g["V"] * (parts + 1) + 2 * g["ng"]) <= 160 * 1024, what
    last = (groups - (g["chunks"] - 1) * g["ng"]) * (channels // groups)
    assert last >= min(8, channels), what   # a partial vector of eight is read as the chunk's last eight channels
    assert g["tiles"] == 1 or g["V"] * g["P"] >= 64, what   # the tiles' kernels add up within whole waves
    assert offsets(g, pixels, channels, size) < 2 ** 31, what


# images, pixels, channels, groups: parts of some 2^31 bytes
LARGE = [(1, 524142, 8192, 64), (1, 5890, 359504, 359504), (2, 4705, 568064, 2536), (1, 131070, 16384, 512), (1, 131008, 16384, 512),
         (1, 2 ** 31 - 1, 8, 1), (1, 10, 2 ** 24 - 8, 2 ** 21 - 1), (3, 100, 2 ** 24 - 8, 2 ** 21 - 1), (2 ** 31 - 1, 1, 8, 8)]


@pytest.mark.parametrize("size", LARGE, ids=str)
def test_large_parts_keep_their_offsets(layout, size):
    for dtype in (cbr.CBR_BF16, cbr.CBR_F32):
        for backward in (False, True):
            check(layout, *size, dtype, backward)


def drawn(r, near):
    """A legal size of up to 2^46 values; near: an image of some 1 to 4 times 2^31 bytes."""
    while True:
        groups = int(2 ** r.uniform(0, 22))
        cpg = int(2 ** r.uniform(0, 13))
        c = groups * cpg
        if c >= 2 ** 24:
            continue
        if near:
            pixels = int(2 ** r.uniform(28, 32) / c * r.choice((1, 2)))
            images = r.randint(1, 3)
        else:
            pixels, images = int(2 ** r.uniform(0, 31)), int(2 ** r.uniform(0, 20))
        if 0 < pixels < 2 ** 31 and math.log2(images * pixels * c) <= 46:
            return images, pixels, c, groups


@pytest.mark.parametrize("near", [False, True])
def test_drawn_sizes_keep_their_offsets(layout, near):
    r = random.Random(near)
    for _ in range(20000):
        check(layout, *drawn(r, near), r.choice((cbr.CBR_BF16, cbr.CBR_F16, cbr.CBR_F32)), r.random() < 0.5)


def test_tiles_of_several_pixels_a_thread(layout):
    """The sizes of tests/test_group_norm_tiles.py are laid out as it says."""
    import test_group_norm_tiles as T
    for size in T.TILES:
        for dtype in (cbr.CBR_BF16, cbr.CBR_F32):
            for backward in (False, True):
                for act in (cbr.CBR_ACT_NONE, cbr.CBR_ACT_RELU, cbr.CBR_ACT_SILU):
                    g = layout(*size, dtype, backward, act)
                    assert g["tiles"] > 1 and 3 <= g["k"] <= T.MOST, (size, dtype, backward, act, g)
