"""AdamW's entry points without a GPU: every refusal comes from the host before anything is enqueued,
so fake device addresses never reach a kernel; and the 8-bit forms of the tests."""
import array
import ctypes
import os

import pytest
import torch

import linear_amd as la
import optim_refs as ref

needs_lib = pytest.mark.skipif(not os.path.exists(la.LIB_PATH), reason="liblinear_amd.so not built")
cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")

BASE = 0x7F0000000000
STEP = 0x1000000000
P, G, M, V, C, NORM, LR, N, P2, G2, M2, V2 = (BASE + i * STEP for i in range(12))
NODEV, OK = la.LINEAR_E_DEVICE, la.LINEAR_OK
NULL, SHAPE, STRIDE, ALIAS, VALUE = (la.LINEAR_E_NULL, la.LINEAR_E_SHAPE, la.LINEAR_E_STRIDE, la.LINEAR_E_ALIAS,
                                     la.LINEAR_E_VALUE)


def table(rows):
    return None if rows is None else array.array("q", [x for r in rows for x in r])


def address(t):
    return None if t is None else t.buffer_info()[0]


PT, GT = (P, 4, 8, 8, 2), (G, 4, 8, 8, 1)


def adamw(params=(PT,), grads=(GT,), m=(M,), v=(V,), copies=None, count=None, options=True, **kw):
    o = la._AdamwOptions(**{**dict(lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, state_bits=32), **kw})
    t = [table(params), table(grads), table([(x,) for x in m]), table([(x,) for x in v]), table(copies)]
    return la._lib().linear_adamw(*map(address, t), len(params) if count is None else count,
                                  ctypes.byref(o) if options else None, None)


@needs_lib
@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), SHAPE), (dict(count=la.GRAD_MAX_TENSORS + 1), SHAPE), (dict(options=False), NULL),
    (dict(state_bits=16), VALUE), (dict(state_bits=0), VALUE), (dict(lr=-1.0), VALUE), (dict(lr=float("nan")), VALUE),
    (dict(lr=float("inf")), VALUE), (dict(beta1=1.0), VALUE), (dict(beta1=-0.1), VALUE), (dict(beta2=1.5), VALUE),
    (dict(beta2=float("nan")), VALUE), (dict(eps=-1e-9), VALUE), (dict(weight_decay=-1.0), VALUE), (dict(step=0), VALUE),
    (dict(step=-3), VALUE), (dict(norm=NORM, max_norm=-1.0), VALUE), (dict(norm=NORM, max_norm=float("nan")), VALUE),
    (dict(params=((P, -1, 8, 8, 2),)), SHAPE), (dict(grads=((G, 4, 7, 7, 1),)), SHAPE), (dict(grads=((G, 1, 32, 32, 1),)), SHAPE),
    (dict(params=((P, 4, 8, 8, 3),)), VALUE), (dict(grads=((G, 4, 8, 8, -1),)), VALUE),
    (dict(params=((0, 4, 8, 8, 2),)), NULL), (dict(grads=((0, 4, 8, 8, 1),)), NULL), (dict(m=(0,)), NULL), (dict(v=(0,)), NULL),
    (dict(params=((P, 4, 8, 7, 2),)), STRIDE), (dict(grads=((G, 4, 8, 1 << 31, 1),)), STRIDE),
    (dict(copies=((C, 4, 8, 8, 2),)), VALUE), (dict(copies=((C, 4, 9, 9, 1),)), SHAPE), (dict(copies=((0, 4, 8, 8, 1),)), NULL),
    (dict(grads=((P, 4, 8, 8, 1),)), ALIAS), (dict(m=(P + 4 * 31,)), ALIAS), (dict(m=(V - 4,)), ALIAS),
    (dict(v=(G + 60,)), ALIAS), (dict(copies=((P, 4, 8, 8, 1),)), ALIAS), (dict(copies=((V, 4, 8, 8, 1),)), ALIAS),
    (dict(norm=M, max_norm=1.0), ALIAS), (dict(device_lr=V + 124), ALIAS), (dict(device_step=P), ALIAS),
    (dict(state_bits=8, m=(M,), v=(M + 32,)), ALIAS),
])
def test_refusals(kw, code):
    assert adamw(**kw) == code


@needs_lib
@cpu_only
def test_calls_that_pass_the_checks():
    assert adamw() == NODEV and adamw(state_bits=8) == NODEV and adamw(copies=((C, 4, 8, 8, 1),)) == NODEV
    assert adamw(state_bits=8, v=(M + 33,)) == NODEV                 # 32 codes and a block's byte
    assert adamw(step=0, device_step=N) == NODEV and adamw(device_lr=LR) == NODEV
    assert adamw(norm=NORM, max_norm=0.0) == NODEV and adamw(max_norm=-1.0) == NODEV
    assert adamw(params=(), grads=(), m=(), v=()) == OK
    assert adamw(params=(PT, (0, 0, 3, 3, 0)), grads=(GT, (0, 0, 3, 3, 0)), m=(M, 0), v=(V, 0)) == NODEV
    # a gradient listed twice is only read; a parameter listed twice is not
    two = dict(m=(M, M2), v=(V, V2))
    assert adamw(params=(PT, (P2, 4, 8, 8, 0)), grads=(GT, GT), **two) == NODEV
    assert adamw(params=(PT, PT), grads=(GT, (G2, 4, 8, 8, 0)), **two) == ALIAS


@needs_lib
@pytest.mark.parametrize("out,state,code", [
    ((P, 4, 8, 8, 0), M, VALUE), ((P, 4, 8, 8, 5), M, VALUE), ((0, 4, 8, 8, 1), M, NULL), ((P, 4, 8, 8, 1), 0, NULL),
    ((P, 4, 8, 7, 1), M, STRIDE), ((P, 4, 8, 8, 1), P + 30, ALIAS), ((P, 4, 8, 8, 2), P - 20, ALIAS),
])
def test_values_refusals(out, state, code):
    t, s = table([out]), table([(state,)])
    assert la._lib().linear_adamw_values(address(t), address(s), 0, 1, None) == code


@needs_lib
def test_state_sizes():
    f = la._lib().linear_adamw_state_bytes
    assert [f(n, 8) for n in (0, 1, 32, 33, 4096)] == [0, 2, 33, 35, 4224] and f(5, 32) == 20
    assert f(-1, 8) == f(5, 16) == f(1 << 62, 32) == -1
    p = torch.zeros(5, 7)
    assert la.adamw_state(p).shape == (5, 7) and la.adamw_state(p, 8).shape == (37,)
    with pytest.raises(ValueError):
        la.adamw_state(p, 4)


def test_wrong_arguments_are_refused_before_the_library():
    p, g = [torch.zeros(4, 8)], [torch.zeros(4, 8)]
    m, v = [torch.zeros(4, 8)], [torch.zeros(4, 8)]
    o = dict(lr=0.1, step=1)
    bad = [lambda: la.linear_adamw(p, g, m, v, **o),                                 # on the host
           lambda: la.linear_adamw(p, [], m, v, **o), lambda: la.linear_adamw(p, [g[0].t()], m, v, **o),
           lambda: la.linear_adamw(p, [g[0][:3]], m, v, **o), lambda: la.linear_adamw(p, g, m, [v[0].half()], **o),
           lambda: la.linear_adamw(p, g, m, [torch.zeros(33, dtype=torch.uint8)], **o),
           lambda: la.linear_adamw(p, g, [torch.zeros(32, dtype=torch.uint8)], [torch.zeros(33, dtype=torch.uint8)], **o),
           lambda: la.linear_adamw(p, g, m, v, norm=torch.zeros(1), **o), lambda: la.linear_adamw(p, g, m, v, max_norm=1.0, **o),
           lambda: la.linear_adamw(p, g, m, v, lr=torch.zeros(2), step=1),
           lambda: la.linear_adamw(p, g, m, v, lr=0.1, step=torch.zeros(1)),
           lambda: la.linear_adamw(p, g, m, v, copies=[], **o),
           lambda: la.linear_adamw_values([torch.zeros(33, dtype=torch.uint8)], False),
           lambda: la.linear_adamw_values([torch.zeros(32, dtype=torch.uint8)], False, out=p)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        la.linear_adamw([p[0].double()], g, m, v, **o)


@pytest.mark.parametrize("second", [False, True])
def test_the_8_bit_forms(second):
    """Every code's value encodes to itself in a block that holds the largest, and no value is further than
    half a step from what its code stands for."""
    lv = ref.levels(second)
    assert bool((lv[1:] > lv[:-1]).all()) and float(lv[-1]) == (61440.0 if second else 448.0)
    blocks = [torch.cat([lv[-1:], part]) for part in lv[:-1].split(31)]
    x = torch.cat([torch.nn.functional.pad(b, (0, 32 - b.numel())) for b in blocks])
    state = ref.encode(x, second)
    assert torch.equal(ref.decode(state, x.numel(), second), x)
    gen = torch.Generator().manual_seed(0)
    y = torch.randn(4099, generator=gen).double() ** (2 if second else 1)
    z = ref.decode(ref.encode(y, second), y.numel(), second)
    least = y.abs().max() * 2.0 ** (-31 if second else -17)
    assert bool(((z - y).abs() <= 2.0 ** -4 * y.abs() + least).all())


def test_the_native_tables_leave_what_is_not_plain_to_the_checks():
    """Anything but lists of contiguous GPU tensors of the right types and sizes gives None (here: host
    tensors, wrong objects, lists of other lengths)."""
    if not os.path.exists(la.MARSHAL_PATH):
        pytest.skip("_marshal.so not built")
    n, t = la._marshal(), [torch.zeros(4, 8)]
    for args in ((t, t, t, t, None), (t, t, t, t, t), ([], [], [], [], None), (t, [], t, t, None), ([1], t, t, t, None),
                 (t, t, t, "x", None), (t, t, t, t), (None,) * 5, ([t[0].to_sparse()], t, t, t, None)):
        assert n.adamw(*args) is None
    for args in ((t, t), ([], []), (t, None), (t,), ([3], [4])):
        assert n.states(*args) is None
