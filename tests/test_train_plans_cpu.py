"""The plans of the gated backward call: a size for every tile, split and pair of launches that it can
choose, which the GPU tests run."""
import os

import pytest

import linear_amd as la

pytestmark = pytest.mark.skipif(not os.path.exists(la.LIB_PATH), reason="liblinear_amd.so not built")

# size, then the tile, stages and sets of dx and of dwg, dwu, with a split contraction ("s") or a
# second launch of another tile; J: both in one launch
SIZES = [
    ((1, 1, 1), "64x64/4x2", "128x128/4", "J"),
    ((1, 1835, 1), "64x64/4x2 s", "64x64/5"),
    ((2, 6696, 264), "64x64/4x2 s", "128x128/2"),
    ((2, 7544, 2192), "64x64/5 s", "256x256/2 + 128x128"),
    ((4, 960, 8160), "64x64/4x2", "256x256/2"),
    ((4, 5549, 132), "64x64/4x2 s", "128x128/4"),
    ((4, 7295, 1030), "64x64/4x2 s", "256x256/2 + 64x64"),
    ((33, 1, 1), "64x64/4x2", "128x128/4", "J"),
    ((33, 1916, 1), "64x64/4x2 s", "64x64/5"),
    ((36, 1, 5397), "128x128/4", "128x128/4", "J"),
    ((36, 4702, 399), "64x64/4x2 s", "128x128/2"),
    ((36, 5112, 1546), "64x64/4x2 s", "256x256/2 + 64x64"),
    ((48, 6568, 536), "64x64/4x2 s", "256x256/2"),
    ((65, 6552, 1160), "64x64/5 s", "256x256/2 + 128x128"),
    ((934, 2696, 3816), "128x128/4", "256x256/2 + 256x128"),
    ((1039, 4074, 999), "128x128/4 s", "256x128/3"),
    ((1349, 1, 1), "64x64/5", "64x64/5 s"),
    ((1524, 65, 1), "64x64/4x2", "64x64/5 s"),
    ((2306, 8, 7253), "256x256/2 + 128x128", "64x64/4x2"),
    ((3082, 8, 5168), "256x256/2 + 64x64", "64x64/5 s"),
    ((4815, 515, 840), "256x128/3", "64x64/4x2"),
    ((5057, 824, 720), "128x128/4", "128x128/4 s"),
    ((6117, 488, 3296), "256x256/2 + 256x128", "128x128/4"),
    ((7307, 2, 1025), "256x256/2", "64x64/5 s"),
    ((7487, 8, 520), "128x128/2", "64x64/4x2 s"),
    ((8, 136, 136), "64x64/4x2", "128x128/4", "J"),
    ((40, 264, 136), "64x64/4x2", "128x128/4", "J"),
]
IDS = ["%dx%dx%d" % s[0] for s in SIZES]


def text(p):
    s = "%dx%d/%d" % (p["tile_m"], p["tile_n"], p["stages"]) + ("x2" if p["sets"] == 2 else "")
    s += " s" if p["splits"] > 1 else ""
    return s + (" + %dx%d" % (p["tile_m2"], p["tile_n2"]) if p["split_c"] else "")


@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_each_size_takes_its_plan(size):
    (M, N, K), dx, dw, *joint = size
    p = la.linear_gated_backward_plan(M, N, K)
    assert (text(p["dx"]), text(p["dw"]), p["joint"], p["two_words"]) == (dx, dw, bool(joint), M <= 32)


def test_the_sizes_cover_every_kind_of_plan():
    """Every plan that a sample of the sizes takes is in the list, for dx and for the weights."""
    import random
    rng = random.Random(0)
    plans = [la.linear_gated_backward_plan(*size[0]) for size in SIZES]
    listed = [{(text(p[n]), p["joint"], p["two_words"]) for p in plans} for n in ("dx", "dw")]
    for _ in range(20000):
        M, N, K = (int(2 ** rng.uniform(0, 13)) for _ in range(3))
        p = la.linear_gated_backward_plan(M, N, K)
        for kinds, n in zip(listed, ("dx", "dw")):
            assert (text(p[n]), p["joint"], p["two_words"]) in kinds, (M, N, K)


def test_plan_refusals():
    lib = la._lib()
    assert lib.linear_gated_backward_plan(-1, 8, 8, la._GatedPlan()) == la.LINEAR_E_SHAPE
    assert lib.linear_gated_backward_plan(8, 1 << 30, 8, la._GatedPlan()) == la.LINEAR_E_SHAPE
    assert lib.linear_gated_backward_plan(8, 8, 8, None) == la.LINEAR_E_NULL
    with pytest.raises(la.LinearArgumentError):
        la.linear_gated_backward_plan(8, 8, 1 << 31)
