"""The gated gradients by every tile, split and pair of launches that a size can choose, and by the
any-layout kernel's two tiles."""
import pytest
import torch

import linear_amd as la
import train_refs as ref
from test_train_gpu import ACTS, DEV, IDS, TYPES, fn, make, padded
from test_train_plans_cpu import IDS as SIZE_IDS
from test_train_plans_cpu import SIZES, text

pytestmark = pytest.mark.gpu


def integers(M, N, K, t):
    """Words for which every dg, du and sum is an integer that FP32 holds: gates of 32, where SiLU is 32
    and its derivative 1 in FP32 (both to 1e-12), so dg = dh u and du = 32 dh; the sums stay below 2^24."""
    gen = torch.Generator().manual_seed(M + 3 * N + 7 * K)
    word = lambda top, *s: torch.randint(-top, top + 1, s, generator=gen).to(t).to(DEV)   # noqa: E731
    dh, x, wg, wu, u = word(1, M, N), word(2, M, K), word(2, N, K), word(2, N, K), word(2, M, N)
    return [dh, x, wg, wu, torch.full((M, N), 32.0, dtype=t, device=DEV), u]


def exact(got, dh, x, wg, wu, g, u, t):
    D, X, G, U, P = (v.double() for v in (dh, x, wg, wu, u))
    dg, du = D * P, 32 * D
    for o, want, n in zip(got, (dg @ G + du @ U, dg.t() @ X, du.t() @ X), ("dx", "dwg", "dwu")):
        assert float(want.abs().max()) < 2 ** 24
        assert torch.equal(o, want.float().to(t)), n


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("size", SIZES, ids=SIZE_IDS)
def test_every_plan(size, t):
    (M, N, K), dx, dw, *joint = size
    p = la.linear_gated_backward_plan(M, N, K)
    assert (text(p["dx"]), text(p["dw"]), p["joint"]) == (dx, dw, bool(joint))
    ops = integers(M, N, K, t)
    got = fn("gated_backward", t)(*ops)
    exact(got, *ops, t)
    # either group alone (where both run in one launch: by itself), into outputs with surroundings
    outs = [padded(torch.full(v.shape, 5.0, dtype=t, device=DEV), 8) for v in got]
    fn("gated_backward", t)(*ops, need_dw=False, dx=outs[0][0])
    fn("gated_backward", t)(*ops, need_dx=False, dwg=outs[1][0], dwu=outs[2][0])
    for (v, flat), o in zip(outs, got):
        assert torch.equal(v, o)
        v.fill_(9.0)
        assert bool((flat == 9.0).all()), "written outside"
    act = ACTS[(M + N + K) % 3]
    x, wg, wu, dh = make(M, N, K, t)
    g, u = ((x.double() @ w.double().t()).to(t) for w in (wg, wu))
    want, bound, _ = ref.gated_backward64(dh, x, wg, wu, g, u, act, t)
    for o, w, b, n in zip(fn("gated_backward", t)(dh, x, wg, wu, g, u, act), want, bound, ("dx", "dwg", "dwu")):
        ref.inside(o, w, b, n)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(20, 72, 72), (20, 2056, 2056), (72, 2056, 2056), (2056, 72, 2056), (2050, 2056, 72)])
def test_any_layout(M, N, K, t):
    """Odd row strides and bases: the any-layout kernel, by its 128-wide tile where 256 of them fill the
    chip, in segments of the two weights and of the two words of up to 32 rows."""
    ops = integers(M, N, K, t)
    views = [padded(v, 3, 1, float("nan"))[0] for v in ops]
    exact(fn("gated_backward", t)(*views), *ops, t)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(20, 264, 136), (300, 264, 136)])
def test_weights_of_different_row_strides(M, N, K, t):
    ops = integers(M, N, K, t)
    want = fn("gated_backward", t)(*ops)
    ops[3] = padded(ops[3], 24, 0, float("nan"))[0]
    got = fn("gated_backward", t)(*ops)
    exact(got, *ops, t)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
