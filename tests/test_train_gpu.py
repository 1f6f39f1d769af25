"""The gated block, its gradients and the layer's gradients on the GPU against 64-bit forms."""
import pytest
import torch

import linear_amd as la
import train_refs as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float16, torch.bfloat16]
IDS = ["f16", "bf16"]
ACTS = list(ref.ACTS)

# one token and a few, odd sizes, tile edges, row counts past each kernel's tile, long rows
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 1024, 768), (1, 4096, 4096), (1, 24, 40000), (2, 40, 72), (5, 129, 192), (7, 33, 65),
          (16, 256, 128), (16, 2048, 1536), (17, 520, 264), (64, 64, 64), (65, 127, 130), (128, 512, 256), (130, 72, 4096),
          (200, 300, 520), (257, 264, 1032), (300, 1000, 768), (512, 768, 512), (1000, 328, 2056), (2050, 200, 264),
          (1040, 2560, 1288)]
# enough tiles for each of the larger tile sizes to be the choice
LARGE = [(4100, 2056, 136), (128, 8200, 264), (2100, 1032, 520), (4100, 1032, 72), (120, 16392, 200), (600, 520, 264)]


def fn(name, t):
    return getattr(la, "linear_%s_%s" % ("bf16" if t == torch.bfloat16 else "f16", name))


def data(seed, *shapes, scale=None):
    """Normal words, each divided by the square root of its last size unless told otherwise."""
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=gen) * (s[-1] ** -0.5 if scale is None else scale) for s in shapes]


def padded(t, pad, shift=0, fill=9.0):
    """The matrix t with `pad` extra columns and a base `shift` words further on, in a sea of `fill`."""
    if pad < 0:
        pad = -t.shape[1] % 8 + 8
    flat = torch.full((t.shape[0] * (t.shape[1] + pad) + shift + 64,), fill, dtype=t.dtype, device=t.device)
    v = flat[shift:].as_strided(t.shape, (t.shape[1] + pad, 1))
    v.copy_(t)
    return v, flat


def make(M, N, K, t, seed=0):
    x, wg, wu, dh = data(seed + M + 3 * N + 7 * K, (M, K), (N, K), (N, K), (M, N))
    x, dh = x * K ** 0.5, dh * N ** 0.5 * 0.1
    return [v.to(t).to(DEV) for v in (x, wg, wu, dh)]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("i", range(len(SHAPES + LARGE)), ids=["%dx%dx%d" % s for s in SHAPES + LARGE])
def test_gated(i, t):
    M, N, K = (SHAPES + LARGE)[i]
    act = ACTS[i % 3]
    x, wg, wu, _ = make(M, N, K, t)
    want, bound = ref.gated64(x, wg, wu, act, t)
    h = fn("gated", t)(x, wg, wu, act)
    ref.inside(h, want[0], bound[0], "h")
    kept = fn("gated", t)(x, wg, wu, act, keep=True)
    for got, w, b, n in zip(kept, want, bound, ("h", "gate", "up")):
        ref.inside(got, w, b, n)
    assert torch.equal(kept[0], h)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("act", ACTS, ids=list(ref.ACTS.values()))
@pytest.mark.parametrize("M", [1, 3, 300])
def test_gated_wide_range_of_sums(M, act, t):
    """Sums from far below to far above the activation's bend, both signs (|g| up to 256)."""
    N, K = 264, 64
    x, wg, wu, _ = make(M, N, K, t)
    x = (x.float() * torch.logspace(-3, 2, M, device=DEV)[:, None]).to(t) if M > 1 else x * 20
    want, bound = ref.gated64(x, wg, wu, act, t)
    got = fn("gated", t)(x, wg, wu, act, keep=True)
    for o, w, b, n in zip(got, want, bound, ("h", "gate", "up")):
        ref.inside(o, w, b, n)


LAYOUTS = [(0, 8, 0), (8, 16, 8), (8, 8, 1), (3, 5, 0), (1, 0, 3), (-1, 8, 0)]   # pads of rows (-1: to a multiple of 8), and the bases' shift in words


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("M,N,K", [(1, 72, 512), (9, 72, 512), (150, 264, 136), (300, 77, 93)])
def test_gated_strides_bases_and_untouched_surroundings(M, N, K, layout, t):
    p, q, s = layout
    x, wg, wu, _ = make(M, N, K, t)
    want, bound = ref.gated64(x, wg, wu, la.EPI_SILU, t)
    # NaN around the inputs: nothing read there may reach an output
    xs, ws, us = (padded(v, p, s, float("nan"))[0] for v in (x, wg, wu))
    outs = [padded(torch.full((M, N), 5.0, dtype=t, device=DEV), q, s) for _ in range(3)]
    fn("gated", t)(xs, ws, us, la.EPI_SILU, keep=True, out=outs[0][0], gate=outs[1][0], up=outs[2][0])
    for (v, flat), w, b, n in zip(outs, want, bound, ("h", "gate", "up")):
        ref.inside(v, w, b, n)
        v.fill_(9.0)
        assert bool((flat == 9.0).all()), "%s: written outside" % n


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_gated_halves_of_one_weight(t):
    M, N, K = 33, 136, 256
    x, wg, wu, _ = make(M, N, K, t)
    w = torch.cat([wg, wu])
    assert torch.equal(fn("gated", t)(x, w[:N], w[N:]), fn("gated", t)(x, wg, wu))
    one = fn("gated", t)(x, wg, wg, keep=True)
    assert torch.equal(one[1], one[2])


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_gated_specials_stay_in_their_rows_and_columns(M, t):
    N, K = 264, 256
    x, wg, wu, _ = make(M, N, K, t)
    clean = fn("gated", t)(x, wg, wu)
    wg[5, 3] = float("nan")
    wu[200, 255] = float("inf")
    got = fn("gated", t)(x, wg, wu)
    keep = torch.ones(N, dtype=torch.bool, device=DEV)
    keep[[5, 200]] = False
    assert torch.equal(got[:, keep], clean[:, keep])
    assert bool(got[:, 5].isnan().all()) and bool((~got[:, 200].isfinite()).all())
    x[M - 1, 7] = float("nan")
    got = fn("gated", t)(x, wg, wu)
    assert bool(got[M - 1].isnan().all())
    assert torch.equal(got[:M - 1][:, keep], clean[:M - 1][:, keep])


def infinite(signs):
    """Infinities of these signs, NaN where the factor is zero."""
    return signs.double() * float("inf")


def same(got, want):
    got = got.double()
    return bool(((got == want) | (got.isnan() & want.isnan())).all())


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,K", [(1, 8), (1, 264), (1, 768), (1, 4100), (1, 9000), (2, 520), (9, 72), (40, 776), (300, 1000)])
def test_gated_infinite_input(M, K, t):
    """One infinity in x: each projection of its row is infinite, with its weight's sign, and
    nothing that a kernel reads past the ends meets it."""
    x, wg, wu, _ = make(M, 72, K, t)
    clean = fn("gated", t)(x, wg, wu, keep=True)
    for k in (0, K // 2, K - 1):
        v = x.clone()
        v[M - 1, k] = float("inf")
        h, g, u = fn("gated", t)(v, wg, wu, keep=True)
        assert same(g[M - 1], infinite(wg[:, k].sign())), k
        assert same(u[M - 1], infinite(wu[:, k].sign())), k
        for a, b in zip((h, g, u), clean):
            assert torch.equal(a[:M - 1], b[:M - 1])


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(1, 72, 136), (9, 200, 264), (65, 65, 65), (130, 1000, 72), (300, 520, 328), (1000, 72, 520)])
def test_gradients_infinite_input(M, N, K, t):
    x, w, _, dy = make(M, N, K, t)
    clean = fn("backward_input", t)(dy, w)
    dw0, db0 = fn("backward_weight", t)(dy, x, bias=True)
    for m, n in ((0, 0), (M - 1, N - 1), (M // 2, N // 2)):
        v = dy.clone()
        v[m, n] = float("-inf")
        rest = torch.arange(M, device=DEV) != m
        dx = fn("backward_input", t)(v, w)
        assert same(dx[m], infinite(-w[n].sign())) and torch.equal(dx[rest], clean[rest])
        rest = torch.arange(N, device=DEV) != n
        dw, db = fn("backward_weight", t)(v, x, bias=True)
        assert same(dw[n], infinite(-x[m].sign())) and torch.equal(dw[rest], dw0[rest])
        assert float(db[n]) == float("-inf") and torch.equal(db[rest], db0[rest])


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(1, 72, 136), (65, 65, 65), (200, 344, 136), (517, 264, 1000)])
def test_gated_backward_infinite_input(M, N, K, t):
    x, wg, wu, dh = make(M, N, K, t)
    _, g, u = fn("gated", t)(x, wg, wu, keep=True)
    clean = fn("gated_backward", t)(dh, x, wg, wu, g, u)
    for m, n in ((0, 0), (M - 1, N - 1)):
        v = dh.clone()
        v[m, n] = float("inf")
        dx, dwg, dwu = fn("gated_backward", t)(v, x, wg, wu, g, u)
        rest = torch.arange(M, device=DEV) != m
        assert torch.equal(dx[rest], clean[0][rest]) and not bool(dx[m].isfinite().any())
        rest = torch.arange(N, device=DEV) != n
        assert torch.equal(dwg[rest], clean[1][rest]) and torch.equal(dwu[rest], clean[2][rest])
        assert same(dwu[n], infinite((x[m].double() * g[m, n].double()).sign()))


@pytest.mark.parametrize("act", ACTS, ids=list(ref.ACTS.values()))
def test_gated_gradients_of_large_gates(act):
    """Far out act is 0 or g and act' is 0 or 1, also where g^2 and g^3 overflow binary32."""
    g = torch.tensor([[1e3, -1e3, 1e10, -1e10, 1e14, -1e14, 1e20, -1e20, 3e38, -3e38]], dtype=torch.bfloat16, device=DEV)
    N = g.shape[1]
    one = torch.ones(1, 8, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(N, 8, dtype=torch.bfloat16, device=DEV)
    row = torch.ones_like(g)
    dx, dwg, dwu = la.linear_bf16_gated_backward(row, one, w, w, g, row, act)
    assert torch.equal(dwg[:, 0], (g[0] > 0).to(dwg.dtype))
    assert torch.equal(dwu[:, 0], torch.where(g[0] > 0, g[0], torch.zeros_like(g[0])))


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_empty_and_zero_sums(t):
    z = lambda *s: torch.zeros(*s, dtype=t, device=DEV)          # noqa: E731
    h, g, u = fn("gated", t)(z(5, 0), z(7, 0), z(7, 0), keep=True)
    assert h.shape == (5, 7) and not h.any() and not g.any() and not u.any()
    assert fn("gated", t)(z(0, 8), z(7, 8), z(7, 8)).shape == (0, 7)
    assert fn("gated", t)(z(5, 8), z(0, 8), z(0, 8)).shape == (5, 0)
    full = lambda *s: torch.full(s, 3.0, dtype=t, device=DEV)    # noqa: E731
    dx, dwg, dwu = fn("gated_backward", t)(z(0, 7), z(0, 8), z(7, 8), z(7, 8), z(0, 7), z(0, 7), dwg=full(7, 8),
                                           dwu=full(7, 8))
    assert dx.shape == (0, 8) and not dwg.any() and not dwu.any()
    dx, dwg, dwu = fn("gated_backward", t)(z(5, 0), z(5, 8), z(0, 8), z(0, 8), z(5, 0), z(5, 0), dx=full(5, 8))
    assert not dx.any() and dwg.shape == (0, 8)
    assert not fn("backward_input", t)(z(5, 0), z(0, 8), out=full(5, 8)).any()
    assert not fn("backward_input", t)(z(5000, 0), z(0, 8), out=full(5000, 8)).any()
    assert not fn("gated", t)(z(1, 0), z(7, 0), z(7, 0), out=full(1, 7)).any()
    dw, db = fn("backward_weight", t)(z(0, 7), z(0, 8), out=full(7, 8), db=full(7))
    assert not dw.any() and not db.any()
    dw, db = fn("backward_weight", t)(z(5, 7), z(5, 0), db=full(7))
    assert dw.shape == (7, 0) and not db.any()
    w32, b32 = torch.full((7, 8), 3.0, device=DEV), torch.full((7,), 3.0, device=DEV)
    fn("backward_weight_f32out", t)(z(0, 7), z(0, 8), out=w32, db=b32, accumulate=True)
    assert bool((w32 == 3).all()) and bool((b32 == 3).all())
    fn("backward_weight_f32out", t)(z(0, 7), z(0, 8), out=w32, db=b32)
    assert not w32.any() and not b32.any()


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=["%dx%dx%d" % s for s in SHAPES])
def test_gated_backward(i, t):
    M, N, K = SHAPES[i]
    act = ACTS[(i + 1) % 3]
    x, wg, wu, dh = make(M, N, K, t)
    _, g, u = (v.to(t) for v in ref.gated64(x, wg, wu, act, t)[0])
    want, bound, (dg, du) = ref.gated_backward64(dh, x, wg, wu, g, u, act, t)
    got = fn("gated_backward", t)(dh, x, wg, wu, g, u, act)
    for o, w, b, n in zip(got, want, bound, ("dx", "dwg", "dwu")):
        ref.inside(o, w, b, n)
    # against the products of the rounded dg and du, the outputs are off by their own rounding
    # (at most u in every value, so in the 2-norm) and by the few dg and du that FP32 rounds the
    # other way (a share of about S (4 |z| + 16) / u of them, 2^-9 in binary16: 2 u sqrt(2^-9) < 0.1 u)
    dg, du = dg.to(t).double(), du.to(t).double()
    near = (dg @ wg.double() + du @ wu.double(), dg.t() @ x.double(), du.t() @ x.double())
    if min(M * K, N * K) >= 4096:
        for o, w, n in zip(got, near, ("dx", "dwg", "dwu")):
            assert float((o.double() - w).norm()) <= 1.1 * ref.half_step(t) * float(w.norm()) + 1e-30, n
    # either group alone gives the same words
    only = fn("gated_backward", t)(dh, x, wg, wu, g, u, act, need_dw=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], got[0])
    only = fn("gated_backward", t)(dh, x, wg, wu, g, u, act, need_dx=False)
    assert only[0] is None and torch.equal(only[1], got[1]) and torch.equal(only[2], got[2])


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("act", ACTS, ids=list(ref.ACTS.values()))
def test_gated_gradients_against_differences(act, t):
    """Directional derivatives of sum(dh * h) in 64 bits by central differences: e = 2^-13 has a
    truncation of e^2 / 6 times a third derivative (relative 1e-8 here) and a rounding of 2^-52 / e."""
    M, N, K = 24, 40, 48
    x, wg, wu, dh = make(M, N, K, t)
    X, G, U, D = (v.double() for v in (x, wg, wu, dh))

    def loss(a, b, c):
        return float((D * (ref.act64(act, a @ b.t())[0] * (a @ c.t()))).sum())

    # g and u rounded to t move act' and u by a half step (relative, |g| act'' <= 1.2 |act'| + 1.2)
    g, u = (X @ G.t()).to(t), (X @ U.t()).to(t)
    grads = fn("gated_backward", t)(dh, x, wg, wu, g, u, act)
    want, bound, (dg, du) = ref.gated_backward64(dh, x, wg, wu, g, u, act, t)
    eg = ref.half_step(t) * ((D * (X @ U.t())).abs() * (1.2 + 1.2 * (X @ G.t()).abs()) + dg.abs())
    eu = ref.half_step(t) * 1.13 * (D * (X @ G.t())).abs()
    extra = (eg @ G.abs() + eu @ U.abs(), eg.t() @ X.abs(), eu.t() @ X.abs())
    e = 2.0 ** -13
    for k, v in enumerate((X, G, U)):
        step = data(k, v.shape, scale=1.0)[0].double().to(DEV)
        plus, minus = [X, G, U], [X, G, U]
        plus[k], minus[k] = v + e * step, v - e * step
        diff = (loss(*plus) - loss(*minus)) / (2 * e)
        got = float((grads[k].double() * step).sum())
        allowed = float(((bound[k] + extra[k]) * step.abs()).sum()) + 1e-5 * abs(diff) + 1e-6
        assert abs(got - diff) <= allowed
        # the bound is a sum of magnitudes; the errors' signs are random, so the sum of squares holds too
        loose = float(((bound[k] + extra[k]) * step).norm())
        assert abs(got - diff) <= 6 * loose + 1e-5 * abs(diff) + 1e-6


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("wide", [False, True], ids=["rounded", "f32out"])
@pytest.mark.parametrize("M,N,K", SHAPES + [(136, 2568, 2560), (200, 4104, 4100), (4104, 136, 4100), (1100, 2568, 2560),
                                            (2568, 1100, 2560)])
def test_linear_backward(M, N, K, wide, t):
    x, w, _, dy = make(M, N, K, t)
    want, bound = ref.linear_backward64(dy, x, w, t, wide)
    dx = fn("backward_input", t)(dy, w)
    ref.inside(dx, want[0], bound[0], "dx")
    weight = fn("backward_weight_f32out" if wide else "backward_weight", t)
    dw, db = weight(dy, x, bias=True)
    ref.inside(dw, want[1], bound[1], "dw")
    ref.inside(db, want[2], bound[2], "db")
    alone, none = weight(dy, x)
    assert none is None and torch.equal(alone, dw)
    if wide:
        base, bb = torch.full_like(dw, 0.5), torch.full_like(db, -0.25)
        got = base.clone(), bb.clone()
        weight(dy, x, out=got[0], db=got[1], accumulate=True)
        assert torch.equal(got[0], base + dw) and torch.equal(got[1], bb + db)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (3, 64, 136), (70, 65, 33), (128, 256, 256), (300, 1000, 264), (520, 264, 776),
                                   (1030, 2056, 520), (4100, 300, 328),
                                   (200, 2568, 2560), (333, 4104, 4100), (4100, 333, 4104), (2568, 200, 2560), (2564, 2568, 24),
                                   (4100, 4104, 72)])
def test_linear_backward_of_small_integers_is_exact(M, N, K, t):
    """Words -2 .. 2: every sum is an integer far below 2^24, so FP32 holds it exactly in any order."""
    gen = torch.Generator().manual_seed(M)
    ints = lambda *s: torch.randint(-2, 3, s, generator=gen).to(t).to(DEV)   # noqa: E731
    dy, x, w = ints(M, N), ints(M, K), ints(N, K)
    D, X, W = dy.double(), x.double(), w.double()
    assert torch.equal(fn("backward_input", t)(dy, w), (D @ W).to(t))
    dw, db = fn("backward_weight", t)(dy, x, bias=True)
    assert torch.equal(dw, (D.t() @ X).to(t)) and torch.equal(db, D.sum(0).to(t))
    dw, db = fn("backward_weight_f32out", t)(dy, x, bias=True)
    assert torch.equal(dw, (D.t() @ X).float()) and torch.equal(db, D.sum(0).float())


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("M,N,K", [(1, 72, 512), (150, 264, 136), (300, 77, 93), (520, 328, 264)])
def test_backward_strides_bases_and_untouched_surroundings(M, N, K, layout, t):
    p, q, s = layout
    x, wg, wu, dh = make(M, N, K, t)
    _, g, u = (v.to(t) for v in ref.gated64(x, wg, wu, la.EPI_SILU, t)[0])
    ins = [padded(v, p, s, float("nan"))[0] for v in (dh, x, wg, wu, g, u)]

    def outputs(*specs):
        return [padded(torch.full(sh, 5.0, dtype=o, device=DEV), q, s) for sh, o in specs]

    def check(outs, want, bound):
        for (v, flat), w, b in zip(outs, want, bound):
            ref.inside(v, w.reshape(v.shape), b.reshape(v.shape), "output")
            v.fill_(9.0)
            assert bool((flat == 9.0).all()), "written outside"

    outs = outputs(((M, K), t), ((N, K), t), ((N, K), t))
    fn("gated_backward", t)(*ins, dx=outs[0][0], dwg=outs[1][0], dwu=outs[2][0])
    check(outs, *ref.gated_backward64(dh, x, wg, wu, g, u, la.EPI_SILU, t)[:2])
    for wide in (False, True):
        o = torch.float32 if wide else t
        outs = outputs(((M, K), t), ((N, K), o), ((1, N), o))
        fn("backward_input", t)(ins[0], ins[2], out=outs[0][0])
        fn("backward_weight_f32out" if wide else "backward_weight", t)(ins[0], ins[1], out=outs[1][0], db=outs[2][0][0])
        check(outs, *ref.linear_backward64(dh, x, wg, t, wide))


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_large_views_of_odd_strides(t):
    """Even sizes in rows of odd stride, enough of them for the larger tile of the any-layout kernel."""
    for M, N, K in ((2050, 2056, 72), (72, 2056, 2056), (2056, 72, 2056)):
        x, wg, wu, dh = make(M, N, K, t)
        xs, gs, us, ds = (padded(v, 3, 1, float("nan"))[0] for v in (x, wg, wu, dh))
        want, bound = ref.gated64(x, wg, wu, la.EPI_SILU, t)
        ref.inside(fn("gated", t)(xs, gs, us), want[0], bound[0], "h")
        for wide in (False, True):
            want, bound = ref.linear_backward64(dh, x, wg, t, wide)
            ref.inside(fn("backward_input", t)(ds, gs), want[0], bound[0], "dx")
            dw, db = fn("backward_weight_f32out" if wide else "backward_weight", t)(ds, xs, bias=True)
            ref.inside(dw, want[1], bound[1], "dw")
            ref.inside(db, want[2], bound[2], "db")


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(40, 72, 64), (300, 264, 520), (300, 77, 93)])
def test_backward_specials_stay_in_their_rows_and_columns(M, N, K, t):
    x, w, _, dy = make(M, N, K, t)
    dx, (dw, _) = fn("backward_input", t)(dy, w), fn("backward_weight", t)(dy, x)
    dy[M - 1, N - 1] = float("nan")
    rows, cols = torch.arange(M, device=DEV) != M - 1, torch.arange(N, device=DEV) != N - 1
    bx, (bw, bb) = fn("backward_input", t)(dy, w), fn("backward_weight", t)(dy, x, bias=True)
    assert bool(bx[M - 1].isnan().all()) and torch.equal(bx[rows], dx[rows])
    assert bool(bw[N - 1].isnan().all()) and torch.equal(bw[cols], dw[cols])
    assert bool(bb[N - 1].isnan()) and bool(bb[:N - 1].isfinite().all())
    dy[M - 1, N - 1] = 0.5
    w[0, K - 1] = float("inf")
    bx = fn("backward_input", t)(dy, w)
    assert bool((~bx[:, K - 1].isfinite() | (dy[:, 0] == 0)).all())
    assert torch.equal(bx[:M - 1, :K - 1], dx[:M - 1, :K - 1])


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_reruns_streams_and_workspaces(t):
    """The same words from reruns, from a stream of the caller's, and from a workspace full of NaN."""
    M, N, K = 300, 1000, 776
    x, wg, wu, dh = make(M, N, K, t)
    h, g, u = fn("gated", t)(x, wg, wu, keep=True)
    one = fn("gated_backward", t)(dh, x, wg, wu, g, u)
    dx, (dw, db) = fn("backward_input", t)(dh, wg), fn("backward_weight", t)(dh, x, bias=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        ws = torch.full((la.gated_workspace_bytes(M, N, K),), 255, dtype=torch.uint8, device=DEV)
        wb = torch.full((la.backward_workspace_bytes(M, N, K),), 255, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        two = fn("gated_backward", t)(dh, x, wg, wu, g, u, workspace=ws, stream=handle)
        three = fn("gated_backward", t)(dh, x, wg, wu, g, u, stream=handle)
        h2 = fn("gated", t)(x, wg, wu, stream=handle)
        dx2 = fn("backward_input", t)(dh, wg, workspace=wb, stream=handle)
        dw2, db2 = fn("backward_weight", t)(dh, x, bias=True, workspace=wb, stream=handle)
        s.synchronize()
        for a, b, c in zip(one, two, three):
            assert torch.equal(a, b) and torch.equal(a, c)
        assert torch.equal(h, h2) and torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(1, 264, 512), (300, 264, 520), (700, 1032, 264)])
def test_graph_replays(M, N, K, t):
    """A captured forward and backward replays to the eager calls' words on new inputs."""
    x, wg, wu, dh = make(M, N, K, t)
    s = torch.cuda.Stream()
    bufs = {n: torch.empty(sh, dtype=t, device=DEV) for n, sh in
            (("out", (M, N)), ("gate", (M, N)), ("up", (M, N)), ("dx", (M, K)), ("dwg", (N, K)), ("dwu", (N, K)),
             ("dy", (M, K)), ("dw", (N, K)), ("db", (N,)))}
    ws = torch.empty(la.gated_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV)
    wb = torch.empty(la.backward_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV)
    names = ("out", "gate", "up"), ("dx", "dwg", "dwu")

    def step(stream=None, **o):
        fn("gated", t)(x, wg, wu, keep=True, stream=stream, **{n: o[n] for n in names[0]})
        fn("gated_backward", t)(dh, x, wg, wu, o["gate"], o["up"], workspace=ws, stream=stream, **{n: o[n] for n in names[1]})
        fn("backward_input", t)(dh, wg, out=o["dy"], workspace=wb, stream=stream)
        fn("backward_weight", t)(dh, x, out=o["dw"], db=o["db"], workspace=wb, stream=stream)

    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step(**bufs)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(**bufs)
    for i in range(3):
        nx, _, _, nh = make(M, N, K, t, seed=100 + i)
        x.copy_(nx)
        dh.copy_(nh)
        for b in bufs.values():
            b.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        got = {n: b.clone() for n, b in bufs.items()}
        step(**bufs)
        torch.cuda.synchronize()
        for n, b in bufs.items():
            assert torch.equal(got[n], b), n


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_one_training_step(t):
    """Forward, down projection, backward through both and the clip, as a user runs them together."""
    M, N, K = 130, 344, 136
    x, wg, wu, _ = make(M, N, K, t)
    wd, dy = (v.to(t).to(DEV) for v in data(9, (K, N), (M, K)))
    h, g, u = fn("gated", t)(x, wg, wu, keep=True)
    y = la.linear(h, wd)
    dh = fn("backward_input", t)(dy, wd)
    dwd, _ = fn("backward_weight", t)(dy, h)
    dx, dwg, dwu = fn("gated_backward", t)(dh, x, wg, wu, g, u)
    grads = [dwg, dwu, dwd]
    norm = la.linear_grad_norm(grads)
    clipped = la.linear_grad_clip(grads, norm, 0.5, out=[torch.empty_like(v) for v in grads])
    # the same step in 64 bits with the intermediate words (h, g, u, dh) as they were stored
    want, bound = ref.gated64(x, wg, wu, la.EPI_SILU, t)
    ref.inside(h, want[0], bound[0], "h")
    b, e = ref.linear_backward64(dy, h, wd, t, False)
    ref.inside(dh, b[0], e[0], "dh")
    ref.inside(dwd, b[1], e[1], "dwd")
    b, e, _ = ref.gated_backward64(dh, x, wg, wu, g, u, la.EPI_SILU, t)
    for o, w, c in zip((dx, dwg, dwu), b, e):
        ref.inside(o, w, c, "gated gradient")
    total = torch.sqrt(sum(v.double().square().sum() for v in grads))
    assert abs(float(norm) - float(total)) <= 2.0 ** -24 * float(total)
    scale = min(1.0, 0.5 / (float(total) + 1e-6))
    for o, v in zip(clipped, grads):
        ref.inside(o, v.double() * scale, ref.rounded(v.double() * scale, 4 * ref.S * v.double().abs() * scale, t), "clipped")
    p = h.double() @ wd.double().t()
    ref.inside(y, p, ref.rounded(p, ref.acc(N, h.double().abs() @ wd.double().abs().t()), t), "y")


def test_long_rows_past_32_bits():
    """A gradient and an input whose rows lie more than 2^31 words apart from first to last."""
    t = torch.float16
    M, N, K = 5, 16, 24
    ld = (1 << 29) + 8
    x, w, _, dy = make(M, N, K, t)
    store = torch.empty((M - 1) * ld + K, dtype=t, device=DEV)
    far = store.as_strided((M, K), (ld, 1))
    far.copy_(x)
    assert torch.equal(fn("gated", t)(far, w, w), fn("gated", t)(x, w, w))
    assert torch.equal(fn("backward_weight", t)(dy, far)[0], fn("backward_weight", t)(dy, x)[0])
    del far
    far = store.as_strided((M, N), (ld, 1))
    far.copy_(dy)
    assert torch.equal(fn("backward_input", t)(far, w), fn("backward_input", t)(dy, w))
    assert torch.equal(fn("backward_weight", t)(far, x)[0], fn("backward_weight", t)(dy, x)[0])


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_operands_past_2_31_words(t):
    """Streamed operands whose last rows lie past 2^31 words (and 4 GiB): the contraction over
    530000 rows, and rows of output that far.  Words -2 .. 2, so FP32 sums are exact (|sum| <=
    4 * 530000 < 2^24)."""
    M, W, n = 530000, 4104, 16
    gen = torch.Generator(device=DEV).manual_seed(7)
    ints = lambda *s: torch.randint(-2, 3, s, generator=gen, device=DEV, dtype=torch.int8).to(t)   # noqa: E731
    big, thin, w = ints(M, W), ints(M, n), ints(n, W)

    def chunks(f, *ts):
        return [f(*(v[i:i + 65536].double() for v in ts)) for i in range(0, M, 65536)]

    dw, db = fn("backward_weight_f32out", t)(thin, big, bias=True)
    assert torch.equal(dw, sum(chunks(lambda a, b: a.t() @ b, thin, big)).float())
    assert torch.equal(db, sum(chunks(lambda a: a.sum(0), thin)).float())
    dw, db = fn("backward_weight_f32out", t)(big, thin, bias=True)
    assert torch.equal(dw, sum(chunks(lambda a, b: a.t() @ b, big, thin)).float())
    assert torch.equal(db, sum(chunks(lambda a: a.sum(0), big)).float())
    wt = w.t().contiguous()                                     # [W, n]: dx [M, n] from dy [M, W]
    dx = fn("backward_input", t)(big, wt)
    assert torch.equal(dx, torch.cat(chunks(lambda a: (a @ wt.double()).to(t), big)))
    dx = fn("backward_input", t)(thin, w)                       # dx [M, W]: the output is the large one
    for i in range(0, M, 65536):
        assert torch.equal(dx[i:i + 65536], (thin[i:i + 65536].double() @ w.double()).to(t))
    _, g, u = fn("gated", t)(big, w, w, keep=True)
    assert torch.equal(g, torch.cat(chunks(lambda a: (a @ w.double().t()).to(t), big))) and torch.equal(g, u)


def test_random_sweep():
    """Random sizes, types, activations, row pads and base shifts over every call."""
    import random
    rng = random.Random(2024)
    for case in range(60):
        t = rng.choice(TYPES)
        M, N, K = (int(round(2 ** rng.uniform(0, 10.5))) for _ in range(3))
        if rng.random() < 0.6:
            N, K = (max(8, v // 8 * 8) for v in (N, K))
        pad, shift, act = rng.choice([0, 8, 16, 3, -1]), rng.choice([0, 0, 0, 8, 1]), rng.choice(ACTS)
        print("case", case, t, (M, N, K), pad, shift, act, flush=True)
        x, wg, wu, dh = make(M, N, K, t, seed=case)
        xs, gs, us, ds = (padded(v, pad, shift, float("nan"))[0] for v in (x, wg, wu, dh))
        want, bound = ref.gated64(x, wg, wu, act, t)
        for o, w, b in zip(fn("gated", t)(xs, gs, us, act, keep=True), want, bound):
            ref.inside(o, w, b, "gated")
        g, u = want[1].to(t), want[2].to(t)
        want, bound, _ = ref.gated_backward64(dh, x, wg, wu, g, u, act, t)
        for o, w, b in zip(fn("gated_backward", t)(ds, xs, gs, us, g, u, act), want, bound):
            ref.inside(o, w, b, "gated backward")
        for wide in (False, True):
            want, bound = ref.linear_backward64(dh, x, wg, t, wide)
            ref.inside(fn("backward_input", t)(ds, gs), want[0], bound[0], "dx")
            dw, db = fn("backward_weight_f32out" if wide else "backward_weight", t)(ds, xs, bias=True)
            ref.inside(dw, want[1], bound[1], "dw")
            ref.inside(db, want[2], bound[2], "db")


def test_calls_from_four_threads():
    """Each thread on a stream of its own, without workspaces of the caller's: the words of one thread."""
    import threading
    t = torch.bfloat16
    sets = [make(M, N, K, t, seed=M) for M, N, K in ((300, 1000, 776), (17, 520, 264), (130, 1001, 769), (1, 2048, 1536))]

    def step(x, wg, wu, dh, stream=None):
        h, g, u = fn("gated", t)(x, wg, wu, keep=True, stream=stream)
        grads = list(fn("gated_backward", t)(dh, x, wg, wu, g, u, stream=stream))
        grads += list(fn("backward_weight", t)(dh, x, bias=True, stream=stream))
        grads.append(fn("backward_input", t)(dh, wg, stream=stream))
        return [h, *grads, la.linear_grad_norm(grads, stream=stream)]

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(10):
                got[i] = step(*sets[i], stream=s)
            s.synchronize()
        except Exception as e:                                   # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors
    for a, b in zip(got, want):
        for o, w in zip(a, b):
            assert torch.equal(o, w)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(2, 40, 72), (65, 127, 130), (300, 264, 136)])
def test_projections_and_gradients_side_by_side(M, N, K, t):
    x, wg, wu, dh = make(M, N, K, t)
    both, dw = torch.full((M, 2 * N), 5.0, dtype=t, device=DEV), torch.full((N, 2 * K), 5.0, dtype=t, device=DEV)
    h, g, u = fn("gated", t)(x, wg, wu, keep=True)
    got = fn("gated", t)(x, wg, wu, keep=True, gate=both[:, :N], up=both[:, N:])
    assert torch.equal(got[0], h) and torch.equal(both, torch.cat([g, u], 1))
    dx, dwg, dwu = fn("gated_backward", t)(dh, x, wg, wu, g, u)
    got = fn("gated_backward", t)(dh, x, wg, wu, both[:, :N], both[:, N:], dwg=dw[:, :K], dwu=dw[:, K:])
    assert torch.equal(got[0], dx) and torch.equal(dw, torch.cat([dwg, dwu], 1))


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(1, 72, 136), (1, 4168, 88), (3, 129, 65), (9, 2720, 1024), (17, 264, 2056), (31, 136, 4096),
                                   (32, 344, 136), (32, 8192, 512)])
@pytest.mark.parametrize("aligned", [True, False])
def test_few_rows_lose_nothing_to_the_inner_rounding(M, N, K, t, aligned):
    """Up to 32 rows dg and du keep two words (relative u^2, or where the second is subnormal the
    smallest subnormal's half): against the gradients of the unrounded dg and du the outputs are off
    by their own rounding, u at most in every value, and FP32's."""
    x, wg, wu, dh = make(M, N, K, t)
    if not aligned:
        x, wg, wu = (padded(v, 1, 1)[0] for v in (x, wg, wu))
    _, g, u = fn("gated", t)(x, wg, wu, la.EPI_GELU_ERF, keep=True)
    got = fn("gated_backward", t)(dh, x, wg, wu, g, u, la.EPI_GELU_ERF)
    X, G, U, D, pg, pu = (v.double() for v in (x, wg, wu, dh, g, u))
    act, slope, r, es = ref.act64(la.EPI_GELU_ERF, pg)
    dg, du = D * pu * slope, D * act
    # their FP32 evaluation, and what two words leave
    left = [e + ref.half_step(t) ** 2 * v.abs() + ref.tiny(t)
            for v, e in ((dg, (D * pu).abs() * es + 2 * ref.S * dg.abs()), (du, (r + ref.S) * du.abs() + D.abs() * ref.FLOOR))]
    pieces = [((dg, G, left[0]), (du, U, left[1])), ((dg.t(), X, left[0].t()),), ((du.t(), X, left[1].t()),)]
    for o, terms, n in zip(got, pieces, ("dx", "dwg", "dwu")):
        want = sum(a @ b for a, b, _ in terms)
        size = sum(a.abs() @ b.abs() for a, b, _ in terms)
        bound = sum(r @ b.abs() for _, b, r in terms) + ref.acc(2 * (2 * N if n == "dx" else M), size)
        ref.inside(o, want, ref.rounded(want, bound, t), n)
