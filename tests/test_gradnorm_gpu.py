"""The global gradient norm and clipping on the GPU against 64-bit forms.

Bounds: the sum of squares is FP64, so the norm is its FP32 rounding, half a step (2^-24) plus
2^-40 for some 2^20 FP64 additions' rounding at the sizes here; the scale is two FP32 operations
(a sum and a quotient) of that norm, 4 half steps; the scaled value one product, then the rounding
to its type."""
import math

import pytest
import torch

import linear_amd as la

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float16, torch.bfloat16, torch.float32]
H = 2.0 ** -24


def tensors(sizes, types, seed=0, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(*s, generator=gen) * scale).to(types[i % len(types)]).to(DEV) for i, s in enumerate(sizes)]


def total(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def check(grads, max_norm, out=None):
    want = total(grads)
    keep = [g.clone() for g in grads]
    norm = la.linear_grad_norm(grads)
    assert norm.shape == (1,) and norm.dtype == torch.float32
    # below 2^-126 FP32 values lie 2^-149 apart, so the rounding there is off by up to 2^-150
    # (1e-44 twice: 1.38721e-44 rounds to 10 * 2^-149 = 1.40130e-44, off by 1.4e-46 < 7.0e-46)
    assert abs(float(norm) - want) <= (H + 2.0 ** -40) * want + 2.0 ** -150
    got = la.linear_grad_clip(grads, norm, max_norm, out=out)
    scale = min(1.0, max_norm / (want + 1e-6))
    for o, g in zip(got, keep):
        w = g.double() * scale
        u = 0.0 if o.dtype == torch.float32 else torch.finfo(o.dtype).eps / 2
        tiny = torch.finfo(o.dtype).smallest_normal * torch.finfo(o.dtype).eps / 2
        bound = w.abs() * (8 * H + u * (1 + 8 * H)) + tiny
        assert bool(((o.double() - w).abs() <= bound).all())
        if scale == 1.0:
            assert torch.equal(o, g)
    if out is not None:
        for g, k in zip(grads, keep):
            assert torch.equal(g, k)
    return norm, got


SETS = {
    "one": [(1,)],
    "one_row": [(7,)],
    "edges": [(1,), (2,), (3,), (8,), (255,), (256,), (257,), (2047,), (8191,), (8192,), (8193,), (16384,), (16385,)],
    "matrices": [(257, 515), (64, 64), (3, 1), (1, 9), (1000, 1001)],
    "more_than_a_table": [(1 + (37 * i) % 300,) for i in range(150)],
    "exactly_a_table": [(9 + i,) for i in range(64)],
    "some_empty": [(0,), (5,), (0, 7), (11, 3), (4, 0)],
    "large": [(5000, 4099), (1 << 22,)],
    "cubes": [(3, 5, 7), (2, 3, 4, 5)],
}


@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("types", [[t] for t in TYPES] + [TYPES], ids=["f16", "bf16", "f32", "mixed"])
@pytest.mark.parametrize("place", ["in_place", "out"])
def test_norm_and_clip(name, types, place):
    grads = tensors(SETS[name], types, seed=len(name))
    out = [torch.full_like(g, 7.0) for g in grads] if place == "out" else None
    check(grads, 0.75, out)
    check(tensors(SETS[name], types, seed=1), 1e9, out)         # no clipping: the words stay


@pytest.mark.parametrize("t", TYPES, ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 3, 4])
def test_bases_that_are_not_aligned(t, shift):
    flat = tensors([(40000,)], [t])[0]
    parts = [flat[shift:shift + 9001], flat[10000 + shift:10000 + shift + 64], flat[20001:20002], flat[30000:39999]]
    guard = flat.clone()
    out = [torch.empty(p.numel() + 8, dtype=t, device=DEV)[s:s + p.numel()] for p, s in zip(parts, (0, 1, 2, 3))]
    check(parts, 2.0, out)
    check(parts, 2.0)
    keep = torch.ones_like(flat, dtype=torch.bool)
    for a, n in ((shift, 9001), (10000 + shift, 64), (20001, 1), (30000, 9999)):
        keep[a:a + n] = False
    assert torch.equal(flat[keep], guard[keep])                 # only the tensors were written


@pytest.mark.parametrize("t", TYPES, ids=["f16", "bf16", "f32"])
def test_padded_rows(t):
    wide = tensors([(70, 9000)], [t])[0]
    guard = wide.clone()
    a, b = wide[:, 16:8700], wide[3:9, :8]
    assert not a.is_contiguous()
    check([a[10:]], 1.5)
    check([b], 1.5, out=[torch.empty(6, 24, dtype=t, device=DEV)[:, 3:11]])
    check([b.contiguous()], 1.5, out=[b])
    assert torch.equal(wide[:, :8][9:], guard[:, :8][9:]) and torch.equal(wide[:, 8700:], guard[:, 8700:])


def test_ranges():
    """FP32 gradients whose squares overflow or vanish in FP32, binary16 and bfloat16 extremes."""
    big = torch.tensor([3e38, -3e38, 1.0], device=DEV)
    assert float(la.linear_grad_norm([big])) == float("inf")     # 4.2e38 is past FP32
    for v in ([1e30, 2e30], [1e-30, 3e-30], [1e-44, 1e-44], [2e38, 2e38]):
        check([torch.tensor(v, device=DEV)], 1.0, out=[torch.empty(2, device=DEV)])
    check([torch.full((1000,), 65504.0, dtype=torch.float16, device=DEV)], 1.0)
    check([torch.full((1000,), 6e-8, dtype=torch.float16, device=DEV)], 1e-7)
    check([torch.full((10,), 1e38, dtype=torch.bfloat16, device=DEV)], 1.0)


def test_specials():
    g = torch.tensor([1.0, float("inf"), 2.0], device=DEV)
    norm = la.linear_grad_norm([g])
    assert float(norm) == float("inf")
    o = la.linear_grad_clip([g], norm, 1.0, out=[torch.empty_like(g)])[0]
    assert float(o[0]) == 0.0 and bool(o[1].isnan()) and float(o[2]) == 0.0
    g = torch.tensor([1.0, float("nan"), 2.0], dtype=torch.bfloat16, device=DEV)
    norm = la.linear_grad_norm([g, torch.ones(5, device=DEV)])
    assert bool(norm.isnan())
    for o in la.linear_grad_clip([g, torch.ones(5, device=DEV)], norm, 1.0):
        assert bool(o.isnan().all())
    z = torch.zeros(33, dtype=torch.float16, device=DEV)
    norm = la.linear_grad_norm([z])
    assert float(norm) == 0.0
    assert not la.linear_grad_clip([z], norm, 1.0)[0].any()
    assert not la.linear_grad_clip([torch.ones(3, device=DEV)], torch.ones(1, device=DEV), 0.0)[0].any()


def test_no_tensors_and_all_empty():
    out = torch.full((1,), 5.0, device=DEV)
    assert float(la.linear_grad_norm([], out=out)) == 0.0
    assert la.linear_grad_clip([], out, 1.0) == []
    e = [torch.empty(0, device=DEV), torch.empty(3, 0, dtype=torch.float16, device=DEV)]
    assert float(la.linear_grad_norm(e)) == 0.0
    la.linear_grad_clip(e, out, 1.0)


def test_the_same_tensor_twice():
    g = tensors([(100, 30)], [torch.bfloat16])[0]
    norm = la.linear_grad_norm([g, g])
    assert abs(float(norm) - math.sqrt(2) * total([g])) <= 2 * H * float(norm)
    with pytest.raises(la.LinearArgumentError):
        la.linear_grad_clip([g, g], norm, 1.0)
    a, b = la.linear_grad_clip([g, g], norm, 1.0, out=[torch.empty_like(g), torch.empty_like(g)])
    assert torch.equal(a, b)


def test_reruns_streams_and_graphs():
    grads = tensors([(300, 700), (513,), (64, 64)], TYPES)
    a = la.linear_grad_norm(grads)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ws = torch.full((la.grad_workspace_bytes(3),), 255, dtype=torch.uint8, device=DEV)
    out = [torch.empty_like(g) for g in grads]
    norm = torch.empty(1, device=DEV)
    torch.cuda.synchronize()
    b = la.linear_grad_norm(grads, workspace=ws, stream=s)
    c = la.linear_grad_norm(grads, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        la.linear_grad_norm(grads, out=norm, workspace=ws)
        la.linear_grad_clip(grads, norm, 0.3, out=out)
    for i in range(3):
        for g, n in zip(grads, tensors([(300, 700), (513,), (64, 64)], TYPES, seed=10 + i)):
            g.copy_(n)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        want = la.linear_grad_norm(grads)
        assert torch.equal(norm, want)
        for o, e in zip(out, la.linear_grad_clip(grads, want, 0.3, out=[torch.empty_like(g) for g in grads])):
            assert torch.equal(o, e)
