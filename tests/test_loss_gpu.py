"""A linear head's cross entropy and its gradients on the GPU against 64-bit forms."""
import pytest
import torch

import linear_amd as la
import loss_refs as ref
from train_refs import half_step, inside, tiny

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float16, torch.bfloat16]
IDS = ["f16", "bf16"]

# one row and few, one column, odd sizes, tile edges, rows past each tile, rows copied for their odd length
SHAPES = [(1, 1, 1), (1, 7, 64), (1, 8200, 4096), (2, 33, 65), (5, 129, 192), (16, 256, 128), (20, 4099, 520), (33, 1000, 72),
          (64, 64, 64), (65, 127, 130), (130, 515, 93), (257, 264, 1032), (300, 1000, 768), (517, 2049, 264),
          (1024, 1024, 768), (2100, 1032, 520), (4100, 264, 72), (3, 70000, 8), (4100, 8200, 40)]


def fn(name, t):
    return getattr(la, "linear_%s_cross_entropy%s" % ("bf16" if t == torch.bfloat16 else "f16", name))


def make(M, N, K, t, seed=0, bias=True, scale=2.0):
    gen = torch.Generator().manual_seed(seed + M + 3 * N + 7 * K)
    x = torch.randn(M, K, generator=gen)
    w = torch.randn(N, K, generator=gen) * scale * K ** -0.5
    b = torch.randn(N, generator=gen)
    target = torch.randint(0, max(N, 1), (M,), generator=gen)
    if M > 2:
        target[torch.rand(M, generator=gen) < 0.2] = -100
        target[1] = N                                 # just outside
    dloss, dlse = torch.randn(M, generator=gen) * 0.1, torch.randn(M, generator=gen) * 0.01
    return (x.to(t).to(DEV), w.to(t).to(DEV), target.to(DEV), b.to(t).to(DEV) if bias else None, dloss.to(DEV), dlse.to(DEV))


def check_forward(x, w, target, b, t, **kw):
    want, bound = ref.forward64(x, w, target, b)
    loss, lse = fn("", t)(x, w, target, b, **kw)
    inside(loss, want[0], bound[0], "loss")
    inside(lse, want[1], bound[1], "lse")
    return loss, lse


def check_backward(dloss, dlse, x, w, target, lse, b, t, f32=False, **kw):
    want, bound = ref.backward64(dloss, dlse, x, w, target, b, t, f32)
    got = fn("_backward_f32out" if f32 else "_backward", t)(dloss, x, w, target, lse, b, dlse=dlse, bias=True, **kw)
    for g, v, e, n in zip(got, want, bound, ("dx", "dw", "db")):
        inside(g, v, e, n)
    return got


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=["%dx%dx%d" % s for s in SHAPES])
def test_loss_and_gradients(i, t):
    M, N, K = SHAPES[i]
    x, w, target, b, dloss, dlse = make(M, N, K, t, bias=i % 2 == 0)
    loss, lse = check_forward(x, w, target, b, t)
    got = check_backward(dloss, dlse if i % 3 else None, x, w, target, lse, b, t)
    again = fn("_backward", t)(dloss, x, w, target, lse, b, dlse=dlse if i % 3 else None, bias=True)
    assert all(torch.equal(u, v) for u, v in zip(got, again)), "reruns give the same bits"
    assert all(torch.equal(u, v) for u, v in zip((loss, lse), fn("", t)(x, w, target, b)))


# the vocabulary in pieces: many rows, and rows that are copied
PIECES = [(20000, 8300, 64), (40, 17000, 2049), (16400, 8210, 33)]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", PIECES)
def test_vocabulary_in_pieces(M, N, K, t):
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    _, lse = check_forward(x, w, target, b, t)
    check_backward(dloss, dlse, x, w, target, lse, b, t)
    check_backward(dloss, None, x, w, target, lse, b, t, f32=True)


# few rows against weights of a million values and more: column tiles and row blocks of every remainder,
# outputs of aligned rows (and, with K odd or rows off alignment, the other kernels)
FEW = [(65, 4099, 520), (100, 3000, 776), (127, 16500, 72), (128, 9001, 1032), (128, 1100, 2008), (1, 4096, 264), (2, 16500, 64), (20, 4103, 520), (33, 5000, 776), (63, 2049, 1032), (64, 70001, 256), (64, 1100, 2008),
       (17, 3000, 513), (40, 524300, 8)]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", FEW)
def test_few_rows_and_a_large_vocabulary(M, N, K, t):
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    _, lse = check_forward(x, w, target, b, t)
    got = check_backward(dloss, dlse, x, w, target, lse, b, t)
    wide = check_backward(dloss, dlse, x, w, target, lse, b, t, f32=True)
    # the same sums times the factor's inverse, rounded to the type, or to FP32: half a step of each
    size = wide[1].double().abs()
    inside(got[1], wide[1].double(), (half_step(t) + 2.0 ** -24) * 1.001 * size + tiny(t), "dw of one rounding")
    for pad in (8, 3):
        dw, flat = padded(torch.zeros_like(w), pad, 8, 9.0)
        again = fn("_backward", t)(dloss, x, w, target, lse, b, dlse=dlse, dw=dw)
        inside(again[1], got[1].double(), 2 * ref.backward64(dloss, dlse, x, w, target, b, t)[1][1], "dw in wide rows")
        if pad == 8:
            assert torch.equal(again[1], got[1])
        dw.fill_(9.0)
        assert bool((flat == 9.0).all()), "written outside"


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(1, 70, 40), (30, 260, 264), (300, 777, 136)])
def test_f32_gradients_and_accumulation(M, N, K, t):
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    _, lse = fn("", t)(x, w, target, b)
    first = check_backward(dloss, dlse, x, w, target, lse, b, t, f32=True)
    dw, db = torch.full((N, K), 3.0, device=DEV), torch.full((N,), -2.0, device=DEV)
    fn("_backward_f32out", t)(dloss, x, w, target, lse, b, dlse=dlse, accumulate=True, dw=dw, db=db, need_dx=False)
    # one FP32 addition: half a step of the sum (and of a partial sum's, where the contraction is split)
    for got, one, base in ((dw, first[1], 3.0), (db, first[2], -2.0)):
        want = one.double() + base
        assert bool(((got.double() - want).abs() <= 2.0 ** -23 * (want.abs() + 1)).all())


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("wanted", ["dx", "dw", "db", "dx,db"])
def test_gradients_that_are_not_wanted(wanted, t):
    M, N, K = 70, 300, 72
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    _, lse = fn("", t)(x, w, target, b)
    every = fn("_backward", t)(dloss, x, w, target, lse, b, dlse=dlse)
    some = fn("_backward", t)(dloss, x, w, target, lse, b, dlse=dlse, need_dx="dx" in wanted, need_dw="dw" in wanted,
                              bias="db" in wanted)
    for n, a, c in zip(("dx", "dw", "db"), every, some):
        assert (c is None) == (n not in wanted)
        if c is not None:
            assert torch.equal(a, c)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K,share", [(1, 70, 40, 1.0), (20, 300, 72, 0.7), (300, 1030, 136, 0.9), (2500, 520, 72, 0.5),
                                         (2100, 1032, 520, 0.02), (5000, 300, 93, 0.995)])
def test_rows_without_a_gradient_take_no_part(M, N, K, share, t):
    """Rows that do not count, or of weight zero: their x and lse may hold anything, their dx is zero, and
    the other rows' gradients are those of a call without them (up to the order of sums: the same bounds)."""
    x, w, target, b, dloss, _ = make(M, N, K, t)
    gen = torch.Generator().manual_seed(9)
    off = (torch.rand(M, generator=gen) < share).to(DEV)
    target[off] = -1
    zero = ~off & (torch.rand(M, generator=gen) < 0.1).to(DEV)
    dloss[zero] = 0.0
    _, lse = fn("", t)(x, w, target, b)
    want, bound = ref.backward64(dloss, None, x, w, target, b, t)
    x[off | zero] = float("nan")
    lse[off | zero] = float("nan")
    dx = torch.full_like(x, 7.0)
    got = fn("_backward", t)(dloss, x, w, target, lse, b, dx=dx)
    for g, v, e, n in zip(got, want, bound, ("dx", "dw", "db")):
        inside(g, v, e, n)
    assert bool((dx[off | zero] == 0).all())
    wide = fn("_backward_f32out", t)(dloss, x, w, target, lse, b, need_dx=False)
    keep = ~(off | zero)
    alone = fn("_backward_f32out", t)(dloss[keep], x[keep], w, target[keep], lse[keep], b, need_dx=False)
    for g, v, e in zip(wide[1:], alone[1:], ref.backward64(dloss, None, x.nan_to_num(0), w, target, b, t, True)[1][1:]):
        inside(g, v.double(), 2 * e, "with and without the rows")


def padded(v, pad, shift, fill):
    """The matrix v with `pad` extra columns and a base `shift` words further on, in a sea of `fill`."""
    flat = torch.full((v.shape[0] * (v.shape[1] + pad) + shift + 64,), fill, dtype=v.dtype, device=v.device)
    out = flat[shift:].as_strided(v.shape, (v.shape[1] + pad, 1))
    out.copy_(v)
    return out, flat


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("pad,out_pad,shift", [(0, 8, 0), (8, 16, 8), (8, 3, 1), (3, 5, 0), (1, 0, 3)])
@pytest.mark.parametrize("M,N,K", [(1, 72, 64), (40, 264, 136), (300, 513, 93)])
def test_strides_bases_and_untouched_surroundings(M, N, K, pad, out_pad, shift, t):
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    xs, ws = (padded(v, pad, shift, float("nan"))[0] for v in (x, w))
    bs = torch.cat([torch.full((3,), float("nan"), dtype=t, device=DEV), b])[3:]
    vectors = [torch.full((M + 2,), 7.0, device=DEV) for _ in range(2)]
    loss, lse = check_forward(xs, ws, target, bs, t, loss=vectors[0][1:-1], lse=vectors[1][1:-1])
    assert all(float(v[0]) == 7.0 and float(v[-1]) == 7.0 for v in vectors)
    dx, dw = padded(torch.zeros_like(x), out_pad, shift, 9.0), padded(torch.zeros_like(w), out_pad, shift, 9.0)
    check_backward(dloss, dlse, xs, ws, target, lse, bs, t, dx=dx[0], dw=dw[0])
    for v, flat in (dx, dw):
        v.fill_(9.0)
        assert bool((flat == 9.0).all()), "written outside"


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M", [1, 20, 300])
def test_rows_that_do_not_count(M, t):
    """All rows outside the vocabulary: losses and gradients of zero (with dlse, lse's alone); a NaN
    row that does not count has loss 0 and leaves the other rows' losses and dx alone."""
    N, K = 270, 136
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    for outside in (-1, N, -100, 2 ** 40, -2 ** 62):
        off = torch.full_like(target, outside)
        loss, lse = check_forward(x, w, off, b, t)
        assert bool((loss == 0).all())
        for g in fn("_backward", t)(dloss, x, w, off, lse, b):
            assert bool((g == 0).all())
        check_backward(dloss, dlse, x, w, off, lse, b, t)
    if M == 1:
        return
    target[M // 2] = -100
    clean = fn("", t)(x, w, target, b)
    x[M // 2, 3] = float("nan")
    dirty = fn("", t)(x, w, target, b)
    assert torch.equal(clean[0], dirty[0]) and bool(dirty[1][M // 2].isnan())
    keep = torch.arange(M, device=DEV) != M // 2
    assert torch.equal(clean[1][keep], dirty[1][keep])
    dx = fn("_backward", t)(dloss, x, w, target, dirty[1], b, need_dw=False)[0]
    assert bool((dx[M // 2] == 0).all()) and bool(dx.isfinite().all())


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M", [1, 20, 300])
def test_masked_columns_and_empty_rows(M, t):
    """A bias of -inf takes its columns out; with all taken out lse is -inf and the loss NaN; an
    infinite logit gives an infinite lse."""
    N, K = 517, 64
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    b[::3] = float("-inf")
    target = target // 3 * 3 + 1
    want, bound = ref.forward64(x, w, target, b)
    loss, lse = fn("", t)(x, w, target, b)
    inside(loss, want[0], bound[0], "loss")
    inside(lse, want[1], bound[1], "lse")
    dx, dw, db = fn("_backward", t)(dloss, x, w, target, lse, b)
    assert bool((dw[::3] == 0).all()) and bool((db[::3] == 0).all()) and bool(dx.isfinite().all())
    b.fill_(float("-inf"))
    loss, lse = fn("", t)(x, w, target, b)
    ok = ref.counted(target, N)
    assert bool((lse == float("-inf")).all()) and bool(loss[ok].isnan().all()) and bool((loss[~ok] == 0).all())
    b.zero_()
    b[N - 1] = float("inf")
    loss, lse = fn("", t)(x, w, target, b)
    assert bool((lse == float("inf")).all())
    ok &= target != N - 1
    assert bool((loss[ok] == float("inf")).all())
    # the type's lowest value masks like -inf once another column stays
    b.zero_()
    b[::3] = torch.finfo(t).min
    loss, lse = check_forward(x, w, target, b, t)
    assert bool(lse.isfinite().all())


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("scale", [1e-3, 30.0])
def test_flat_and_peaked_rows(scale, t):
    """Logits all alike, and rows decided by one logit (|z| in the hundreds)."""
    M, N, K = 100, 1500, 256
    x, w, target, b, dloss, dlse = make(M, N, K, t, scale=scale, bias=False)
    _, lse = check_forward(x, w, target, None, t)
    check_backward(dloss, dlse, x, w, target, lse, None, t)


@pytest.mark.parametrize("size", [1e-12, 1e-7, 1.0, 1e3])
def test_binary16_gradients_of_any_size(size):
    """dz is scaled before its rounding: FP32 outputs keep their precision for weights of any size."""
    M, N, K = 48, 700, 128
    x, w, target, b, dloss, dlse = make(M, N, K, torch.float16)
    _, lse = fn("", torch.float16)(x, w, target, b)
    want, bound = ref.backward64(dloss * size, None, x, w, target, b, torch.float16, True)
    got = fn("_backward_f32out", torch.float16)(dloss * size, x, w, target, lse, b)
    for g, v, e in zip(got[1:], want[1:], bound[1:]):
        inside(g, v, e, "size %g" % size)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_empty_sizes(t):
    x, w, target, b, dloss, dlse = make(6, 9, 16, t)
    # no rows
    loss, lse = fn("", t)(x[:0], w, target[:0], b)
    assert loss.shape == lse.shape == (0,)
    dw, db = torch.full_like(w, 5.0), torch.full_like(b, 5.0)
    fn("_backward", t)(dloss[:0], x[:0], w, target[:0], lse, b, dw=dw, db=db)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    dw, db = torch.full((9, 16), 5.0, device=DEV), torch.full((9,), 5.0, device=DEV)
    fn("_backward_f32out", t)(dloss[:0], x[:0], w, target[:0], lse, b, dw=dw, db=db, accumulate=True)
    assert bool((dw == 5).all()) and bool((db == 5).all())
    # no vocabulary
    loss, lse = fn("", t)(x, w[:0], target, b[:0])
    assert bool((loss == 0).all()) and bool((lse == float("-inf")).all())
    dx, dw, db = fn("_backward", t)(dloss, x, w[:0], target, lse, b[:0])
    assert bool((dx == 0).all()) and dw.shape == (0, 16) and db.shape == (0,)
    # no width: the logits are the bias
    check_forward(x[:, :0], w[:, :0], target, b, t)
    _, lse = fn("", t)(x[:, :0], w[:, :0], target, b)
    db = fn("_backward", t)(dloss, x[:, :0], w[:, :0], target, lse, b)[2]
    want, bound = ref.backward64(dloss, None, x[:, :0], w[:, :0], target, b, t)
    inside(db, want[2], bound[2], "db")


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(3, 500, 72), (300, 1030, 93)])
def test_captured_calls_replayed(M, N, K, t):
    """A loss and its gradients captured into one graph, replayed on other data with eager calls between."""
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    warm = fn("", t)(x, w, target, b)
    fn("_backward", t)(dloss, x, w, target, warm[1], b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse = fn("", t)(x, w, target, b)
        grads = fn("_backward", t)(dloss, x, w, target, lse, b, dlse=dlse)
    for seed in range(3):
        for old, new in zip((x, w, target, b, dloss, dlse), make(M, N, K, t, seed=seed * 100)):
            old.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        eager = fn("", t)(x, w, target, b)
        want = fn("_backward", t)(dloss, x, w, target, eager[1], b, dlse=dlse)
        assert torch.equal(loss, eager[0]) and torch.equal(lse, eager[1])
        assert all(torch.equal(u, v) for u, v in zip(grads, want))


def test_another_stream_and_a_given_workspace():
    t = torch.bfloat16
    x, w, target, b, dloss, dlse = make(130, 515, 93, t)
    want = fn("", t)(x, w, target, b)
    grads = fn("_backward", t)(dloss, x, w, target, want[1], b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(max(la.cross_entropy_workspace_bytes(130, 515, 93), la.cross_entropy_backward_workspace_bytes(130, 515, 93)),
                     dtype=torch.uint8, device=DEV)
    got = fn("", t)(x, w, target, b, workspace=ws, stream=side)
    mine = fn("_backward", t)(dloss, x, w, target, got[1], b, workspace=ws, stream=side)
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want)) and all(torch.equal(u, v) for u, v in zip(mine, grads))


def test_a_weight_past_2_31_words():
    """Rows of the weight more than 2^31 words on: the first and last columns decide their rows."""
    t, M, N, K = torch.bfloat16, 40, 70000, 32768
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = (torch.randn(M, K, generator=gen, device=DEV) * K ** -0.5).to(t)
    w = torch.randn(N, K, generator=gen, device=DEV, dtype=t)
    target = torch.randint(0, N, (M,), generator=gen, device=DEV)
    target[0], target[1] = N - 1, 0
    loss, lse = fn("", t)(x, w, target)
    z = torch.cat([x.double() @ part.double().t() for part in w.split(5000)], 1)
    want = torch.logsumexp(z, 1)
    # |z| <= 1 by |x| |w| sums of some 200 in all: acc(K, 210) of train_refs
    bound = (K / 16 + 48) * 2.0 ** -23 * 210
    assert float((lse.double() - want).abs().max()) <= bound
    assert float((loss.double() - (want - z.gather(1, target[:, None])[:, 0])).abs().max()) <= 2 * bound
    dloss = torch.ones(M, device=DEV)
    dx, dw, _ = fn("_backward", t)(dloss, x, w, target, lse)
    dz = torch.exp(z - want[:, None])
    dz[torch.arange(M, device=DEV), target] -= 1
    for rows in (slice(0, 50), slice(N - 50, N)):
        exact = dz[:, rows].t() @ x.double()
        # the rounding of dz, of dw, and the sums': (1 + 2^-8)^2 - 1 of the products' magnitude and their FP32 sum
        room = (2.0 ** -8 * 2.1 + 4 * bound) * (dz[:, rows].abs().t() @ x.double().abs()) + 1e-30
        assert bool(((dw[rows].double() - exact).abs() <= room).all())
    part = torch.zeros(M, K, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(part)
    for n in range(0, N, 5000):
        piece = w[n:n + 5000].double()
        part += dz[:, n:n + 5000] @ piece
        size += dz[:, n:n + 5000].abs() @ piece.abs()
    assert bool(((dx.double() - part).abs() <= (2.0 ** -8 * 1.1 + 4 * bound) * size + 2.0 ** -8 * part.abs()).all())


def test_weights_of_extreme_ratios():
    """dloss far below dlse, and the reverse: the factor that dz is rounded under stays finite."""
    M, N, K = 33, 300, 72
    for t in TYPES:
        x, w, target, b, dloss, dlse = make(M, N, K, t)
        _, lse = fn("", t)(x, w, target, b)
        for one, more in ((1e-30, 1.0), (1.0, 1e-30), (1e-36, 1e30), (0.0, 1e-3), (1e-3, 0.0), (1e20, 1e20)):
            d, e = dloss * one, dlse * more
            want, bound = ref.backward64(d, e, x, w, target, b, t, True)
            got = fn("_backward_f32out", t)(d, x, w, target, lse, b, dlse=e, need_dx=False)
            inside(got[1], want[1], bound[1], "dw %g %g" % (one, more))
            inside(got[2], want[2], bound[2], "db %g %g" % (one, more))


def test_loss_alone_and_rows_of_one_target():
    """lse without loss and loss without lse; every row with the same target."""
    M, N, K = 200, 700, 64
    for t in TYPES:
        x, w, target, b, dloss, _ = make(M, N, K, t)
        target.fill_(699)
        loss, lse = check_forward(x, w, target, b, t)
        check_backward(dloss, None, x, w, target, lse, b, t)
        tag = "bf16" if t == torch.bfloat16 else "f16"
        ws = torch.empty(la.cross_entropy_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV)
        for keep in (0, 1):
            out = torch.zeros(M, device=DEV)
            args = [x.data_ptr(), K, w.data_ptr(), K, b.data_ptr(), target.data_ptr()] + [None, None]
            args[6 + keep] = out.data_ptr()
            rc = getattr(la._lib(), "linear_%s_cross_entropy" % tag)(*args, M, N, K, ws.data_ptr(), ws.numel(),
                                                                      torch.cuda.current_stream().cuda_stream)
            assert rc == la.LINEAR_OK and torch.equal(out, lse if keep else loss)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(5, 129, 192), (20, 4099, 520), (100, 3001, 776), (130, 515, 93), (300, 8201, 264), (1024, 1024, 768),
                                   (2100, 1032, 520), (20000, 8300, 64)])
def test_what_the_workspace_and_the_outputs_held_does_not_matter(M, N, K, t):
    """All bits set: NaN as words and as floats, -1 as counts and places."""
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    loss, lse = fn("", t)(x, w, target, b, workspace=torch.zeros(la.cross_entropy_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV))
    size = la.cross_entropy_backward_workspace_bytes(M, N, K)
    for name in ("_backward", "_backward_f32out"):
        clean = fn(name, t)(dloss, x, w, target, lse, b, dlse=dlse, workspace=torch.zeros(size, dtype=torch.uint8, device=DEV))
        full = [torch.full_like(g, float("nan")) for g in clean]
        got = fn(name, t)(dloss, x, w, target, lse, b, dlse=dlse, dx=full[0], dw=full[1], db=full[2],
                          workspace=torch.full((size,), 255, dtype=torch.uint8, device=DEV))
        assert all(torch.equal(u, v) for u, v in zip(clean, got))
    again = fn("", t)(x, w, target, b, workspace=torch.full((la.cross_entropy_workspace_bytes(M, N, K),), 255, dtype=torch.uint8, device=DEV))
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("M", [9, 1500])
def test_targets_of_any_64_bit_value(M):
    """Words whose lower halves look like columns do not count."""
    t, N, K = torch.bfloat16, 300, 72
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    strange = torch.tensor([2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, -2 ** 63, -2 ** 32 + 7, 2 ** 31, -1], device=DEV)
    target[1:8] = strange
    _, lse = check_forward(x, w, target, b, t)
    check_backward(dloss, dlse, x, w, target, lse, b, t)


def test_two_calls_at_once():
    """Two host threads, each with a stream, inputs and workspaces of its own."""
    import threading
    t = torch.bfloat16
    sets = [make(300, 2049, 264, t, seed=s) for s in (0, 50)]
    want = []
    for x, w, target, b, dloss, dlse in sets:
        loss, lse = fn("", t)(x, w, target, b)
        want.append((loss, lse) + fn("_backward", t)(dloss, x, w, target, lse, b, dlse=dlse))
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        x, w, target, b, dloss, dlse = sets[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(8):
                loss, lse = fn("", t)(x, w, target, b)
                got[i] = (loss, lse) + fn("_backward", t)(dloss, x, w, target, lse, b, dlse=dlse)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    for g, v in zip(got, want):
        assert g is not None and all(torch.equal(a, b) for a, b in zip(g, v))


# weight gradients of three and four slices on the few rows' kernel: column tiles and row blocks of every
# remainder, one block a workgroup and many
@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(129, 4096, 264), (200, 4099, 520), (193, 16500, 72), (255, 9001, 1032), (256, 1100, 2008),
                                   (256, 70001, 256), (256, 3000, 776), (256, 524300, 8),
                                   (256, 16500, 2048), (161, 33000, 1024), (200, 131200, 256), (130, 53001, 640), (200, 33001, 520), (256, 17001, 1000)])
def test_some_hundred_rows_and_a_large_vocabulary(M, N, K, t):
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    _, lse = check_forward(x, w, target, b, t)
    got = check_backward(dloss, dlse, x, w, target, lse, b, t)
    check_backward(dloss, dlse, x, w, target, lse, b, t, f32=True)
    again = fn("_backward", t)(dloss, x, w, target, lse, b, dlse=dlse, bias=True)
    assert all(torch.equal(u, v) for u, v in zip(got, again))
    dw, flat = padded(torch.zeros_like(w), 8, 8, 9.0)
    fn("_backward", t)(dloss, x, w, target, lse, b, dlse=dlse, dw=dw)
    assert torch.equal(dw, got[1])
    dw.fill_(9.0)
    assert bool((flat == 9.0).all()), "written outside"


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(40, 66000, 2049), (300, 33100, 4099)])
def test_copied_weights_in_pieces(M, N, K, t):
    """Rows of odd length, more than are copied at a time."""
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    _, lse = check_forward(x, w, target, b, t)
    check_backward(dloss, dlse, x, w, target, lse, b, t)
    check_backward(dloss, None, x, w, target, lse, b, t, f32=True)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("size", [1e-30, 1e-34, 3e-35, 1e-36, 1e-38, 1e-42])
def test_row_weights_that_are_all_small(size, t):
    """Weights down to FP32's subnormals: the factor that dz is rounded under, and its inverse, stay numbers."""
    M, N, K = 33, 300, 72
    x, w, target, b, dloss, _ = make(M, N, K, t)
    _, lse = fn("", t)(x, w, target, b)
    d = dloss * 10 * size
    for dlse in (None, d * 0.5, d * -0.25):
        want, bound = ref.backward64(d, dlse, x, w, target, b, t, True)
        got = fn("_backward_f32out", t)(d, x, w, target, lse, b, dlse=dlse, bias=True)
        # the factor ends at 2^125: half a spacing of binary16's subnormals, 2^-25, is 2^-150 of dz (with what
        # the matrix unit makes of such words, as in backward64, 2^11 times that under its sums' error); outputs and the
        # partial sums of up to 16 splits are rounded to multiples of FP32's 2^-149
        dz = 2.0 ** -150 if t == torch.float16 else 0.0
        for g, v, e, n, count, factor in zip(got, want, bound, ("dx", "dw", "db"), (N, M, M), (w, x, torch.ones(1, device=DEV))):
            most = float(factor.double().abs().amax())
            room = count * most * dz * (1 + 2 ** 11 * (count / 16 + 48) * 2.0 ** -23) + 17 * 2.0 ** -150
            inside(g, v, e + room, "%s %g" % (n, size))


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_row_weights_near_the_largest_number(t):
    """|d + dlse| + |d| past FP32's range, d + dlse and the outputs inside it."""
    M, N, K = 33, 300, 72
    x, w, target, _, dloss, _ = make(M, N, K, t, bias=False)
    x = x * 2.0 ** -8
    _, lse = fn("", t)(x, w, target)
    target = torch.where(ref.counted(target, N), target, 5)
    one = dloss.sign() * (0.6 + dloss.abs().clamp(max=0.4))
    for d, dlse in ((3.3e38 * one, None), (3e38 * one.sign(), None), (1.9e38 * one.sign(), 1.4e38 * one), (3.3e38 * one, -1e38 * one)):
        want, bound = ref.backward64(d, dlse, x, w, target, None, t, True)
        got = fn("_backward_f32out", t)(d, x, w, target, lse, None, dlse=dlse, need_dx=False, bias=False)
        inside(got[1], want[1], bound[1], "dw")


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N", [(3, 64), (70, 1000), (300, 9001)])
@pytest.mark.parametrize("base,gap", [(12, 8), (28, 12), (296, 10), (304, 14), (1992, 8), (1984, 16), (-2016, 16), (30464, 12)])
def test_confident_rows_keep_their_loss(base, gap, M, N, t):
    """Rows decided by their target (logits base + gap and base): a loss far under a step of lse has an
    error that lse's size has no part in.  The logits are sums of two whole numbers, so they are exact."""
    x, w = torch.zeros(M, 8, dtype=t, device=DEV), torch.zeros(N, 8, dtype=t, device=DEV)
    x[:, 0], w[:, 0] = 1, base
    target = (torch.arange(M, device=DEV) * 37) % N
    group = 1 + torch.arange(M, device=DEV) % 7       # the rows of a group share the columns that are up
    x[torch.arange(M, device=DEV), group] = 1
    w[target, group] = gap
    z = x.double() @ w.double().t()
    assert float(w[0, 0]) == base
    y = z - z.amax(1, keepdim=True)
    want = torch.logsumexp(y, 1) - y.gather(1, target[:, None])[:, 0]
    loss, _ = fn("", t)(x, w, target)
    # the sum of the exponentials: up to 90 + N / 8192 additions (loss_refs) of half a step of FP32, relative to
    # a sum of exp(want), and S (|y| + 8) on three factors of each term but the largest (exp 0 is 1); the
    # logarithm and the addition
    p = torch.where(y == 0, 0.0, torch.exp(y) * 3 * 2.0 ** -23 * (y.abs() + 8)).sum(1)
    inside(loss, want, p + (90 + N / 8192) * 2.0 ** -24 + 4 * 2.0 ** -24 * want.abs(), "loss")


def test_calls_without_the_bindings_module(monkeypatch):
    """The same bits where tensors are read by the binding itself: the loss, its gradients, an AdamW step."""
    t = torch.bfloat16
    x, w, target, b, dloss, dlse = make(70, 300, 72, t)

    def calls():
        loss, lse = fn("", t)(x, w, target, b)
        grads = fn("_backward", t)(dloss, x, w, target, lse, b, dlse=dlse)
        wide = fn("_backward_f32out", t)(dloss, x, w, target, lse, b)
        p, m, v = w.clone(), la.adamw_state(w, 8), la.adamw_state(w, 8)
        la.linear_adamw([p], [grads[1]], [m], [v], lr=1e-2, step=1)
        return [loss, lse, *grads, *wide, p, m, v, *la.linear_adamw_values([m], False, like=[p])]

    want = calls()
    monkeypatch.setattr(la, "_marshal", lambda: la._NoMarshal)
    assert all(torch.equal(u, v) for u, v in zip(calls(), want))


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(1, 8200, 4096), (20, 4099, 520), (300, 1030, 96), (1024, 1024, 768), (2100, 1032, 520), (20000, 8300, 64)])
def test_workspaces_of_the_size_that_calls_in_place_need(M, N, K, t):
    """The same bits as with a larger workspace, and nothing written past its end."""
    x, w, target, b, dloss, dlse = make(M, N, K, t)
    loss, lse = fn("", t)(x, w, target, b, workspace=torch.empty(la.cross_entropy_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV))
    full = torch.empty(la.cross_entropy_backward_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV)
    want = fn("_backward", t)(dloss, x, w, target, lse, b, dlse=dlse, workspace=full)
    tight = la.cross_entropy_workspace_bytes(M, N, K, True)
    ws = torch.full((tight + 4096,), 77, dtype=torch.uint8, device=DEV)
    got = fn("", t)(x, w, target, b, workspace=ws[:tight])
    assert torch.equal(got[0], loss) and torch.equal(got[1], lse) and bool((ws[tight:] == 77).all())
    tight = la.cross_entropy_backward_workspace_bytes(M, N, K, True)
    ws = torch.full((tight + 4096,), 77, dtype=torch.uint8, device=DEV)
    for gx in (x, padded(x, 3, 1, float("nan"))[0]):   # x is gathered from any layout
        got = fn("_backward", t)(dloss, gx, w, target, lse, b, dlse=dlse, workspace=ws[:tight])
        assert all(torch.equal(u, v) for u, v in zip(got, want)) and bool((ws[tight:] == 77).all())


def test_a_call_in_place_takes_no_room_for_copies():
    t = torch.bfloat16
    x, w, target, b, dloss, dlse = make(4, 40000, 1024, t)
    torch.cuda.synchronize()
    for call in (lambda: fn("", t)(x, w, target, b), lambda: fn("", t)(x, w, target, b, loss=torch.empty(4, device=DEV))):
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        call()
        assert torch.cuda.max_memory_allocated() - before < 8 << 20
