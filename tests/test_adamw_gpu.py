"""AdamW steps on the GPU against 64-bit forms; 8-bit moments byte for byte."""
import math

import pytest
import torch

import linear_amd as la
import optim_refs as ref
from train_refs import inside

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float16, torch.bfloat16, torch.float32]
OPTIONS = dict(lr=1e-2, beta1=0.9, beta2=0.97, eps=1e-8, weight_decay=0.1)

SETS = {
    "one": [(1,)],
    "edges": [(1,), (2,), (7,), (8,), (9,), (31,), (32,), (33,), (255,), (2047,), (2048,), (2049,), (4096,), (4097,)],
    "matrices": [(257, 515), (64, 64), (3, 1), (1, 9), (1000, 1001)],
    "more_than_a_table": [(1 + (37 * i) % 300,) for i in range(97)],
    "exactly_a_table": [(9 + i,) for i in range(40)],
    "some_empty": [(0,), (5,), (0, 7), (11, 3), (4, 0)],
    "large": [(3000, 1111), (4099,), (2048, 2048)],
}


def make(sizes, ptypes, gtypes, seed=0):
    gen = torch.Generator().manual_seed(seed)
    p = [(torch.randn(*s, generator=gen) * 0.1).to(ptypes[i % len(ptypes)]).to(DEV) for i, s in enumerate(sizes)]
    g = [(torch.randn(*s, generator=gen) * 10.0 ** -(i % 4)).to(gtypes[i % len(gtypes)]).to(DEV) for i, s in enumerate(sizes)]
    return p, g


def states(params, bits):
    return [la.adamw_state(p, bits) for p in params], [la.adamw_state(p, bits) for p in params]


def values(states, params, second):
    """The moments in 64 bits."""
    return [ref.decode(s, p.numel(), second).reshape(p.shape) if s.dtype == torch.uint8 else s.double()
            for s, p in zip(states, params)]


def check_step(p, g, m, v, step, scale=1.0, copies=None, **kw):
    """One step, checked against the form in 64 bits from the same weights and moments."""
    old, om, ov = [t.clone() for t in p], values(m, p, False), values(v, p, True)
    keep = [t.clone() for t in g]
    assert la.linear_adamw(p, g, m, v, step=kw.pop("step_tensor", step), copies=copies, **{**OPTIONS, **kw}) is not None
    for i in range(len(p)):
        want, bound = ref.step64(old[i], g[i], om[i], ov[i], OPTIONS, step, scale)
        inside(p[i], want[0], ref.stored(want[0], bound[0], p[i].dtype), "p %d" % i)
        if copies is not None:
            inside(copies[i], want[0], ref.stored(want[0], bound[0], copies[i].dtype), "copy %d" % i)
        if m[i].dtype == torch.uint8:
            assert ref.same_state(m[i], ref.encode(want[1], False), p[i].numel(), False), "m %d" % i
            assert ref.same_state(v[i], ref.encode(want[2], True), p[i].numel(), True), "v %d" % i
        else:
            inside(m[i], want[1], bound[1], "m %d" % i)
            inside(v[i], want[2], bound[2], "v %d" % i)
        assert torch.equal(g[i], keep[i])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("name", SETS)
def test_steps(name, bits):
    sizes = SETS[name]
    p, g = make(sizes, TYPES, [torch.bfloat16, torch.float32, torch.float16, torch.bfloat16])
    m, v = states(p, bits)
    for step in (1, 2, 3):
        check_step(p, g, m, v, step)
        g = make(sizes, TYPES, [torch.bfloat16, torch.float32, torch.float16, torch.bfloat16], seed=step)[1]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gt", TYPES, ids=["gf16", "gbf16", "gf32"])
@pytest.mark.parametrize("pt", TYPES, ids=["pf16", "pbf16", "pf32"])
def test_types_clipping_and_copies(pt, gt, bits):
    sizes = [(70, 33), (2050,), (5,)]
    p, g = make(sizes, [pt], [gt])
    m, v = states(p, bits)
    norm = la.linear_grad_norm(g)
    for step, most in ((1, 0.5), (2, 1e6)):
        copies = [torch.empty(s, dtype=[torch.float16, torch.bfloat16][i % 2], device=DEV) for i, s in enumerate(sizes)]
        check_step(p, g, m, v, step, ref.clip_scale(norm, most), copies, norm=norm, max_norm=most)


def rows(t, pad, fill=9.0):
    flat = torch.full((t.shape[0] * (t.shape[1] + pad) + 8,), fill, dtype=t.dtype, device=DEV)
    v = flat.as_strided(t.shape, (t.shape[1] + pad, 1), 4)
    v.copy_(t)
    return v, flat


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pads", [(3, 0, 0), (0, 5, 0), (0, 0, 1), (8, 2, 3)], ids=str)
def test_rows_with_gaps(pads, bits):
    """Strided weights, gradients and copies: the same bits as without gaps, and nothing between rows written."""
    sizes = [(40, 33), (1, 77), (300, 5), (7, 1)]
    p, g = make(sizes, TYPES, TYPES[::-1])
    m, v = states(p, bits)
    q, h = [rows(t, pads[0]) for t in p], [rows(t, pads[1]) for t in g]
    c = [rows(torch.zeros(s, dtype=torch.bfloat16, device=DEV), pads[2]) for s in sizes]
    mm, vv = states(p, bits)
    plain = [torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in sizes]
    for step in (1, 2):
        la.linear_adamw(p, g, m, v, step=step, copies=plain, **OPTIONS)
        la.linear_adamw([t[0] for t in q], [t[0] for t in h], mm, vv, step=step, copies=[t[0] for t in c], **OPTIONS)
    for a, b in ((p, q), (g, h), (plain, c)):
        for x, (y, flat) in zip(a, b):
            assert torch.equal(x, y)
            y.fill_(9.0)
            assert bool((flat == 9.0).all())
    assert all(torch.equal(a, b) for a, b in zip(m + v, mm + vv))


@pytest.mark.parametrize("bits", [32, 8])
def test_addresses_of_any_alignment(bits):
    sizes = [(1000,), (33, 65)]
    p, g = make(sizes, [torch.bfloat16, torch.float32], [torch.float32, torch.float16])
    m, v = states(p, bits)

    def shifted(t):
        flat = torch.zeros(t.numel() + 9, dtype=t.dtype, device=DEV)
        out = flat[3:3 + t.numel()].view(t.shape)
        out.copy_(t)
        return out, flat

    q, h, mm, vv = ([shifted(t) for t in ts] for ts in (p, g, m, v))
    for step in (1, 2, 3):
        la.linear_adamw(p, g, m, v, step=step, **OPTIONS)
        la.linear_adamw([t[0] for t in q], [t[0] for t in h], [t[0] for t in mm], [t[0] for t in vv], step=step, **OPTIONS)
    for a, b in ((p, q), (m, mm), (v, vv)):
        for x, (y, flat) in zip(a, b):
            assert torch.equal(x, y) and not bool(flat[:3].any()) and not bool(flat[3 + x.numel():].any())


def test_8_bit_borders():
    """Values on and beside every border between codes, block maxima on and beside the borders where the
    unit changes, blocks of zeros, tiny and huge values: the state after a step with beta 0 is the
    gradient's (m) and its square's (v), here from float32 words."""
    lv = ref.levels(False)
    mid = (lv[1:] + lv[:-1]) / 2
    near = torch.cat([mid, torch.nextafter(mid.float(), torch.tensor(0.0)).double(),
                      torch.nextafter(mid.float(), torch.tensor(1e9)).double(), lv])
    blocks = []
    for top in (448.0, 463.99997, 464.0, 464.00003, 500.0, 232.0, 231.99998):
        for chunk in near[near < top].split(31):
            block = torch.zeros(32, dtype=torch.float64)
            block[0] = top
            block[1:1 + chunk.numel()] = chunk
            blocks += [block, -block, block * 2.0 ** -50, block * 2.0 ** 40]
    for size in (0.0, 1e-45, 1e-38, 1e-31, 2.0 ** -100, 3e38, 1.9375 * 2.0 ** 127, 3.4e38):
        blocks.append(torch.full((32,), size, dtype=torch.float64) * torch.linspace(-1, 1, 32, dtype=torch.float64))
    g = torch.cat(blocks)[:-5].float().to(DEV)
    p = torch.zeros_like(g)
    m, v = la.adamw_state(p, 8), la.adamw_state(p, 8)
    la.linear_adamw([p], [g], [m], [v], step=1, lr=0.0, beta1=0.0, beta2=0.0)
    assert ref.same_state(m, ref.encode(g.double(), False), g.numel(), False)
    assert ref.same_state(v, ref.encode(g.double() * g.double(), True), g.numel(), True)


def test_8_bit_second_moments_borders():
    lv = ref.levels(True)
    mid = (lv[1:] + lv[:-1]) / 2
    roots = torch.cat([mid, lv]).sqrt().float()
    near = torch.cat([roots, torch.nextafter(roots, torch.tensor(0.0)), torch.nextafter(roots, torch.tensor(1e9))])
    blocks = []
    for top in (61440.0 ** 0.5, 63487.99 ** 0.5, 63488.0 ** 0.5, 63488.01 ** 0.5, 65000.0 ** 0.5):
        for chunk in near[near < top].split(31):
            block = torch.zeros(32)
            block[0] = top
            block[1:1 + chunk.numel()] = chunk
            blocks += [block, block * 2.0 ** -30, block * 2.0 ** 30]
    g = torch.cat(blocks).to(DEV)
    p = torch.zeros_like(g)
    m, v = la.adamw_state(p, 8), la.adamw_state(p, 8)
    la.linear_adamw([p], [g], [m], [v], step=1, lr=0.0, beta1=0.0, beta2=0.0)
    assert ref.same_state(v, ref.encode(g.double() * g.double(), True), g.numel(), True)
    stands = ref.decode(v, g.numel(), True)
    assert bool((stands[g != 0] > 0).all()), "a moment over zero is never stored as zero"


def test_every_code_is_read_back():
    """Every code in blocks of several units, through a step that keeps the moments (beta near 1 keeps no
    code exactly, so the values are read instead) and as bfloat16 and float32."""
    for second in (False, True):
        codes = torch.arange(256, dtype=torch.uint8).repeat(3)
        units = torch.tensor([27] * 8 + [127] * 8 + [200] * 8, dtype=torch.uint8)
        state = torch.cat([codes, units]).to(DEV)
        want = ref.decode(state, 768, second)
        for t in (torch.bfloat16, torch.float32):
            out = [torch.empty(768, dtype=t, device=DEV)]
            got = la.linear_adamw_values([state], second, out=out)[0].double()
            ok = ~want.isnan()
            assert torch.equal(got[ok], want[ok]) and bool(got[~ok].isnan().all())
    with pytest.raises(ValueError):
        la.linear_adamw_values([state], True, out=[torch.empty(768, dtype=torch.float16, device=DEV)])


def test_values_of_many_states():
    sizes = [(1 + (53 * i) % 400, 1 + i % 3) for i in range(150)] + [(0,), (2049,)]
    p, g = make(sizes, [torch.float32], [torch.bfloat16])
    m, v = states(p, 8)
    la.linear_adamw(p, g, m, v, step=1, **OPTIONS)
    for s, second in ((m, False), (v, True)):
        got = la.linear_adamw_values(s, second, like=p)
        for a, b, q in zip(got, values(s, p, second), p):
            assert a.shape == q.shape and a.dtype == torch.bfloat16 and torch.equal(a.double(), b)
    wide, flat = rows(torch.zeros(sizes[0], device=DEV), 3)
    la.linear_adamw_values(m[:1], False, out=[wide])
    assert torch.equal(wide.double(), values(m[:1], p[:1], False)[0])
    wide.fill_(9.0)
    assert bool((flat == 9.0).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_not_finite_gradients_stay_in_their_places(bits):
    p, g = make([(300,)], [torch.float32], [torch.float32])
    m, v = states(p, bits)
    la.linear_adamw(p, g, m, v, step=1, **OPTIONS)
    clean = [[t.clone() for t in s] for s in (p, m, v)]
    la.linear_adamw(clean[0], g, clean[1], clean[2], step=2, **OPTIONS)
    g[0][5], g[0][40], g[0][299] = float("nan"), float("inf"), float("-inf")
    la.linear_adamw(p, g, m, v, step=2, **OPTIONS)
    bad = torch.zeros(300, dtype=torch.bool, device=DEV)
    bad[[5, 40, 299]] = True
    assert torch.equal(p[0][~bad], clean[0][0][~bad]) and bool(p[0][bad].isnan().all())
    mv, vv = values(m, p, False)[0], values(v, p, True)[0]
    cm, cv = values(clean[1], p, False)[0], values(clean[2], p, True)[0]
    same = ~bad if bits == 32 else torch.zeros_like(bad)
    if bits == 8:                                     # a block whose largest value is lost may count in other units
        same[:] = ~bad.reshape(-1)[torch.arange(300, device=DEV)]
        for lo in (0, 32, 288):
            same[lo:lo + 32] = False
    assert torch.equal(mv[same], cm[same]) and torch.equal(vv[same], cv[same])
    assert bool(mv[~bad].isfinite().all()) and bool(vv[~bad].isfinite().all())
    assert bool((~mv[bad].isfinite()).all()) and bool((~vv[bad].isfinite()).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_norms_that_are_not_finite(bits):
    for value in (float("nan"), float("inf")):
        p, g = make([(100,)], [torch.float32], [torch.float32])
        m, v = states(p, bits)
        before = p[0].clone()
        la.linear_adamw(p, g, m, v, step=1, norm=torch.tensor([value], device=DEV), max_norm=1.0, **OPTIONS)
        if math.isnan(value):
            assert bool(p[0].isnan().all())
        else:                                         # gradients of zero: the decay alone
            want = before.double() * (1 - OPTIONS["lr"] * OPTIONS["weight_decay"])
            assert bool(((p[0].double() - want).abs() <= 4 * ref.H * want.abs()).all())


def test_tiny_gradients_keep_their_ratio():
    """Second moments under the normal range of FP32: m / sqrt(v) is still near one (eps small beside it).
    v is off by half a subnormal spacing, 2^-150, of at least 2^-133 here."""
    g = torch.full((64,), 2.0 ** -64, device=DEV) * torch.linspace(1, 2, 64, device=DEV)
    p, m, v = torch.zeros(64, device=DEV), torch.zeros(64, device=DEV), torch.zeros(64, device=DEV)
    la.linear_adamw([p], [g], [m], [v], lr=1.0, step=1, beta1=0.9, beta2=0.97, eps=1e-30, weight_decay=0.0)
    assert bool(((p.double() + 1).abs() <= 2.0 ** -17 + 20 * ref.H).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_follows_device_scalars(bits):
    p, g = make([(70, 33), (2050,)], [torch.bfloat16, torch.float32], [torch.bfloat16])
    m, v = states(p, bits)
    q, mm, vv = ([t.clone() for t in s] for s in (p, m, v))
    lr, step = torch.tensor([1e-2], device=DEV), torch.ones(1, dtype=torch.int64, device=DEV)
    norm = torch.tensor([3.0], device=DEV)
    options = {k: o for k, o in OPTIONS.items() if k != "lr"}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.linear_adamw(p, g, m, v, lr=lr, step=step, norm=norm, max_norm=1.0, **options)
    for i in range(1, 5):
        rate = 10.0 ** -i
        lr.fill_(rate)
        step.fill_(i)
        norm.fill_(float(i))
        for t, new in zip(g, make([(70, 33), (2050,)], [torch.bfloat16], [torch.bfloat16], seed=i)[1]):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        la.linear_adamw(q, g, mm, vv, lr=float(lr), step=i, norm=norm, max_norm=1.0, **options)
        # the same formula; the device's power of beta may be a step of FP64 off
        for a, b in zip(p, q):
            inside(a, b.double(), ref.stored(b.double(), 8 * ref.H * (b.double().abs() + rate), a.dtype) * 2, "p")
            b.copy_(a)
        assert all(torch.equal(a, b) for a, b in zip(m + v, mm + vv))


def test_another_stream():
    p, g = make([(500, 33)], [torch.float32], [torch.float32])
    m, v = states(p, 32)
    q, mm, vv = ([t.clone() for t in s] for s in (p, m, v))
    la.linear_adamw(p, g, m, v, step=1, **OPTIONS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    la.linear_adamw(q, g, mm, vv, step=1, stream=side, **OPTIONS)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(p + m + v, q + mm + vv))


def test_values_past_2_31():
    """A tensor of more than 2^31 values: its ends take part."""
    n = 2 ** 31 + 4099
    p = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    for lo in (0, 2 ** 31 - 100, n - 300):
        p[lo:lo + 300], g[lo:lo + 300] = 1.0, 0.5
    m, v = la.adamw_state(p, 8), la.adamw_state(p, 8)
    la.linear_adamw([p], [g], [m], [v], step=1, lr=0.25, beta1=0.5, beta2=0.5, weight_decay=0.0)
    for lo in (0, 2 ** 31 - 100, n - 300):
        assert bool((p[lo:lo + 300] == 0.75).all())
    assert int((p != 0).sum()) == 900 and int((m[:n] != 0).sum()) == 900 and int((v[:n] != 0).sum()) == 900
    out = la.linear_adamw_values([m], False, like=[p])[0]
    assert float(out[n - 1]) == 0.25 and float(out[2 ** 31]) == 0.25 and int((out != 0).sum()) == 900


@pytest.mark.parametrize("bits", [32, 8])
def test_a_training_step_of_a_small_model(bits):
    """The gated block, the head's cross entropy, all gradients, their norm and the update, as a training
    program runs them; two steps against the same in 64 bits with the library's own gradients, and the
    loss against its plain form."""
    import loss_refs
    t = torch.bfloat16
    M, K, F, N = 96, 64, 136, 517
    gen = torch.Generator().manual_seed(4)
    wg, wu, wo, head = ((torch.randn(*s, generator=gen) * s[1] ** -0.5).to(t).to(DEV) for s in ((F, K), (F, K), (K, F), (N, K)))
    params = [wg, wu, wo, head]
    m, v = states(params, bits)
    for step in (1, 2):
        x = torch.randn(M, K, generator=gen).to(t).to(DEV)
        target = torch.randint(0, N, (M,), generator=gen).to(DEV)
        target[::7] = -100
        h, gate, up = la.linear_bf16_gated(x, wg, wu, keep=True)
        y = la.linear_bf16_nobias(h, wo)
        loss, lse = la.linear_bf16_cross_entropy(y, head, target)
        want, bound = loss_refs.forward64(y, head, target)
        inside(loss, want[0], bound[0], "loss")
        dloss = (target >= 0).float() / (target >= 0).sum()
        dy, dhead, _ = la.linear_bf16_cross_entropy_backward(dloss, y, head, target, lse)
        grads64, gb = loss_refs.backward64(dloss, None, y, head, target, None, t)
        inside(dy, grads64[0], gb[0], "dy")
        inside(dhead, grads64[1], gb[1], "dhead")
        dh = la.linear_bf16_backward_input(dy, wo)
        dwo, _ = la.linear_bf16_backward_weight(dy, h)
        _, dwg, dwu = la.linear_bf16_gated_backward(dh, x, wg, wu, gate, up, need_dx=False)
        grads = [dwg, dwu, dwo, dhead]
        norm = la.linear_grad_norm(grads)
        check_step(params, grads, m, v, step, ref.clip_scale(norm, 0.1), norm=norm, max_norm=0.1)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("with_copies", [False, True], ids=["plain", "copies"])
@pytest.mark.parametrize("count", [39, 40, 41, 71, 72, 73, 145])
def test_tables_of_every_fill(count, with_copies, bits):
    """Tensors that fill a launch's table, one less and one more, in the plain form and with copies; empty
    tensors among them take no place."""
    sizes = [(1 + (53 * i) % 97,) for i in range(count)]
    sizes[3:3] = [(0,), (0, 5)]
    p, g = make(sizes, TYPES, TYPES[::-1])
    m, v = states(p, bits)
    copies = [torch.empty_like(t, dtype=torch.bfloat16) for t in p] if with_copies else None
    check_step(p, g, m, v, 1, copies=copies)


@pytest.mark.parametrize("bits", [32, 8])
def test_one_tensor_with_gaps_among_plain_ones(bits):
    sizes = [(1 + (53 * i) % 97, 3) for i in range(75)]
    p, g = make(sizes, [torch.float32], [torch.bfloat16])
    m, v = states(p, bits)
    wide = torch.full((sizes[50][0], 8), 7.0, device=DEV)
    wide[:, :3] = p[50]
    p[50] = wide[:, :3]
    check_step(p, g, m, v, 1)
    assert bool((wide[:, 3:] == 7.0).all())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-37, 1e-39, 1e-44, 1e-60, 1e-300])
def test_an_eps_of_any_size_over_zero(eps, bits):
    """Values with zero moments stay where they are (0 / eps is 0); the others take the formula's step."""
    o = {**OPTIONS, "eps": eps, "weight_decay": 0.0}
    p, g = make([(70, 33), (5,)], TYPES, TYPES[::-1])
    for t in g:
        t[::2] = 0
    m, v = states(p, bits)
    for step in (1, 2):
        old, om, ov = [t.clone() for t in p], values(m, p, False), values(v, p, True)
        la.linear_adamw(p, g, m, v, step=step, **o)
        for i in range(len(p)):
            want, bound = ref.step64(old[i], g[i], om[i], ov[i], o, step)
            inside(p[i][1::2], want[0][1::2], ref.stored(want[0], bound[0], p[i].dtype)[1::2], "p %d" % i)
            assert torch.equal(p[i][::2], old[i][::2])
