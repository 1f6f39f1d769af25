"""The gated block's gradients over the whole range of their types, against 64-bit gradients of the
unrounded dg and du.

Bounds.  A word of dg or du is off by its FP32 evaluation, by u relative (u^2 up to 32 rows, which
keep two words), and, where it is subnormal, by half the spacing of the subnormals.  In binary16 the
words are scaled so that the largest of the call is 2^14 at least, so that half spacing, 2^-25, is
2^-39 of the largest; in bfloat16 it is 2^-134.  Nothing else is added for small values: the outputs'
own subnormals apart, a relative error stays a relative error whatever the size of dh.
"""
import pytest
import torch

import linear_amd as la
import train_refs as ref
from test_train_gpu import ACTS, DEV, IDS, TYPES, data, fn, padded, same

pytestmark = pytest.mark.gpu


def words64(dh, g, u, act, t):
    """dg and du in 64 bits, and what their words may be off by."""
    dh, g, u = (v.double() for v in (dh, g, u))
    a, d, r, ed = ref.act64(act, g)
    dg, du = dh * u * d, dh * a
    eg = (dh * u).abs() * ed + 2 * ref.S * dg.abs()
    eu = (r + ref.S) * du.abs() + dh.abs() * ref.FLOOR
    step = ref.half_step(t) ** (2 if dh.shape[0] <= 32 else 1)
    finite = torch.cat([dg, du]).abs()
    finite = finite[finite.isfinite()]
    small = float(finite.max()) * 2.0 ** -39 if t == torch.float16 and finite.numel() else ref.tiny(t)
    return (dg, du), [e + step * (v.abs() + e) + small for v, e in ((dg, eg), (du, eu))]


def check(got, dh, x, wg, wu, g, u, act, t, rows=None):
    """got against 64 bits; rows: only these rows of dx, and no weight gradients."""
    (dg, du), (eg, eu) = words64(dh, g, u, act, t)
    M, N = dh.shape
    x, wg, wu = x.double(), wg.double(), wu.double()
    parts = {"dx": ((dg, wg, eg), (du, wu, eu)), "dwg": ((dg.t(), x, eg.t()),), "dwu": ((du.t(), x, eu.t()),)}
    for o, (name, terms) in zip(got, parts.items()):
        if rows is not None and name != "dx":
            continue
        keep = slice(None) if rows is None else rows
        want = sum(a[keep] @ b for a, b, _ in terms)
        bound = sum(e[keep] @ b.abs() for _, b, e in terms)
        size = sum((a.abs() + e)[keep] @ b.abs() for a, b, e in terms)
        bound = bound + ref.acc(2 * (2 * N if name == "dx" else M), size)
        ref.inside(o[keep], want, ref.rounded(want, bound, t), name)


def case(seed, M, N, K, t, dh, x=8.0, w=8.0, u=1.0, g=2.0):
    """Words of these sizes: dh, x, wg, wu, gate, up."""
    shapes = ((M, N), (M, K), (N, K), (N, K), (M, N), (M, N))
    return [(s * v).to(t).to(DEV) for s, v in zip((dh, x, w, w, g, u), data(seed, *shapes, scale=1.0))]


SIZES = [(1, 72, 136), (5, 344, 136), (32, 136, 264), (40, 264, 520), (300, 77, 93), (517, 264, 1000), (1000, 520, 264),
         (4100, 72, 136)]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-5, 1e-6, 1e-7])
@pytest.mark.parametrize("i", range(len(SIZES)), ids=["%dx%dx%d" % s for s in SIZES])
def test_gated_gradients_of_small_outputs(i, size, t):
    """dh of a mean loss over many tokens."""
    M, N, K = SIZES[i]
    act = ACTS[i % 3]
    ops = case(i, M, N, K, t, size)
    check(fn("gated_backward", t)(*ops, act), *ops, act, t)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(9, 72, 136), (300, 264, 520), (2050, 2056, 72)])
def test_gated_gradients_of_small_outputs_in_any_layout(M, N, K, t):
    """Operands that the streaming kernels refuse: odd row strides and bases."""
    ops = case(M, M, N, K, t, 1e-6)
    views = [padded(v, 3, 1, float("nan"))[0] for v in ops]
    check(fn("gated_backward", t)(*views), *ops, la.EPI_SILU, t)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(16, 264, 136), (300, 264, 520), (1030, 520, 264)])
def test_gated_gradients_of_rows_of_very_different_size(M, N, K, t):
    """One row a million times the others'."""
    ops = case(M, M, N, K, t, 1e-6)
    ops[0][M // 2] = 1.0
    check(fn("gated_backward", t)(*ops), *ops, la.EPI_SILU, t)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(16, 264, 136), (300, 264, 520), (1030, 520, 264)])
def test_gated_gradients_past_the_largest_word(M, N, K, t):
    """dg and du past 65504 whose sums come back into binary16's range."""
    ops = case(M, M, N, K, t, 2000.0, x=2e-4, w=2e-4, u=300.0, g=300.0)
    got = fn("gated_backward", t)(*ops)
    check(got, *ops, la.EPI_SILU, t)
    assert all(bool(v.isfinite().all()) for v in got)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(9, 72, 136), (300, 264, 520)])
def test_infinite_gradients_leave_the_other_rows_their_precision(M, N, K, t):
    ops = case(M, M, N, K, t, 1e-6)
    ops[0][0, 0], ops[0][1, N - 1] = float("inf"), float("nan")
    got = fn("gated_backward", t)(*ops)
    check(got, *ops, la.EPI_SILU, t, rows=slice(2, None))
    assert bool(got[0][1].isnan().all()) and not bool(got[0][0].isfinite().any())


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (300, 264, 136)])
def test_zero_and_least_gradients(M, N, K):
    t = torch.float16
    ops = case(M, M, N, K, t, 0.0)
    assert all(not bool(v.any()) for v in fn("gated_backward", t)(*ops))
    for v in ops[0], ops[5]:
        v.fill_(2.0 ** -24)                     # the least word: products of 2^-48
    check(fn("gated_backward", t)(*ops), *ops, la.EPI_SILU, t)


@pytest.mark.parametrize("M,N,K", [(9, 264, 136), (300, 264, 520)])
def test_replays_take_the_size_of_their_own_gradients(M, N, K):
    """A captured call replayed with gradients of other sizes: the eager call's words each time."""
    t = torch.float16
    ops = case(M, M, N, K, t, 1.0)
    outs = {n: torch.empty(s, dtype=t, device=DEV) for n, s in (("dx", (M, K)), ("dwg", (N, K)), ("dwu", (N, K)))}
    ws = torch.full((la.gated_workspace_bytes(M, N, K),), 255, dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        fn("gated_backward", t)(*ops, workspace=ws, **outs)
    for i, size in enumerate((1e-6, 2000.0, 1e-3, 1e-7)):
        ops[0].copy_(case(i, M, N, K, t, size)[0])
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        eager = fn("gated_backward", t)(*ops)
        torch.cuda.synchronize()
        for a, b in zip(outs.values(), eager):
            assert same(a, b.double())
        check(eager, *ops, la.EPI_SILU, t)
