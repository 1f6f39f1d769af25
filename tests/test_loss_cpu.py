"""The cross entropy's entry points without a GPU: every refusal comes from the host before anything
is enqueued, so fake device addresses never reach a kernel; and the gradients' formula against
differences of the loss's."""
import os

import pytest
import torch

import linear_amd as la
import loss_refs as ref

needs_lib = pytest.mark.skipif(not os.path.exists(la.LIB_PATH), reason="liblinear_amd.so not built")
cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")

BASE = 0x7F0000000000
STEP = 0x1000000000
X, W, B, T, LOSS, LSE, DLOSS, DLSE, DX, DW, DB, WS = (BASE + i * STEP for i in range(12))
NODEV, OK = la.LINEAR_E_DEVICE, la.LINEAR_OK
BIG = 1 << 40


def forward(x=X, ldx=64, w=W, ldw=64, b=B, t=T, loss=LOSS, lse=LSE, M=8, N=32, K=64, ws=WS, nws=BIG, tag="f16"):
    return getattr(la._lib(), "linear_%s_cross_entropy" % tag)(x, ldx, w, ldw, b, t, loss, lse, M, N, K, ws, nws, None)


def backward(dloss=DLOSS, dlse=DLSE, x=X, ldx=64, w=W, ldw=64, b=B, t=T, lse=LSE, dx=DX, lddx=64, dw=DW, lddw=64, db=DB,
             acc=None, M=8, N=32, K=64, ws=WS, nws=BIG, tag="f16"):
    fn = getattr(la._lib(), "linear_%s_cross_entropy_backward%s" % (tag, "" if acc is None else "_f32out"))
    return fn(dloss, dlse, x, ldx, w, ldw, b, t, lse, dx, lddx, dw, lddw, db, *(() if acc is None else (acc,)), M, N, K, ws,
              nws, None)


NULL, SHAPE, STRIDE, ALIAS, SPACE = (la.LINEAR_E_NULL, la.LINEAR_E_SHAPE, la.LINEAR_E_STRIDE, la.LINEAR_E_ALIAS,
                                     la.LINEAR_E_WORKSPACE)


@needs_lib
@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(N=1 << 31), SHAPE), (dict(K=1 << 22), SHAPE), (dict(M=(1 << 24) + 1), SHAPE),
    (dict(x=0), NULL), (dict(w=0), NULL), (dict(t=0), NULL), (dict(loss=0, lse=0), NULL), (dict(ws=0), NULL),
    (dict(ldx=63), STRIDE), (dict(ldw=63), STRIDE), (dict(ldw=1 << 31), STRIDE),
    (dict(nws=100), SPACE), (dict(ws=WS + 8), SPACE),
    (dict(loss=X + 4), ALIAS), (dict(lse=W), ALIAS), (dict(loss=B), ALIAS), (dict(lse=T + 56), ALIAS), (dict(lse=LOSS + 28), ALIAS),
    (dict(ws=X, nws=BIG), ALIAS), (dict(ws=LOSS), ALIAS), (dict(ws=T), ALIAS),
])
def test_forward_refusals(tag, kw, code):
    assert forward(tag=tag, **kw) == code


@needs_lib
@cpu_only
def test_forward_calls_that_pass_the_checks():
    assert forward() == NODEV and forward(b=0) == NODEV and forward(loss=0) == NODEV and forward(lse=0) == NODEV
    assert forward(M=0, x=0, t=0, loss=0, lse=0, ws=0, nws=0) == OK
    assert forward(N=0, w=0, b=0) == NODEV and forward(K=0, x=0, w=0, ldx=0, ldw=0) == NODEV
    assert forward(M=1, ldx=10 ** 9) == NODEV           # one row has no stride


@needs_lib
@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("acc", [None, 0, 1])
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(K=1 << 22), SHAPE),
    (dict(dloss=0), NULL), (dict(x=0), NULL), (dict(w=0), NULL), (dict(t=0), NULL), (dict(lse=0), NULL), (dict(ws=0), NULL),
    (dict(dx=0, dw=0, db=0), NULL),
    (dict(ldx=63), STRIDE), (dict(ldw=63), STRIDE), (dict(lddx=63), STRIDE), (dict(lddw=63), STRIDE),
    (dict(nws=100), SPACE), (dict(ws=WS + 8), SPACE),
    (dict(dx=X), ALIAS), (dict(dw=W), ALIAS), (dict(dw=DX + 64), ALIAS), (dict(db=DW + 2), ALIAS), (dict(db=DLOSS), ALIAS),
    (dict(dx=LSE), ALIAS), (dict(dx=DLSE), ALIAS), (dict(dw=T), ALIAS), (dict(ws=DX), ALIAS), (dict(ws=LSE), ALIAS),
])
def test_backward_refusals(tag, acc, kw, code):
    assert backward(tag=tag, acc=acc, **kw) == code


@needs_lib
@cpu_only
def test_backward_calls_that_pass_the_checks():
    for acc in (None, 0, 1):
        assert backward(acc=acc) == NODEV and backward(acc=acc, dlse=0, b=0) == NODEV
        assert backward(acc=acc, dx=0) == NODEV and backward(acc=acc, dw=0, db=0) == NODEV and backward(acc=acc, dx=0, dw=0) == NODEV
        assert backward(acc=acc, N=0, x=0, w=0, b=0, dw=0, db=0) == NODEV      # dx is zeroed
        assert backward(acc=acc, K=0, x=0, w=0, dx=0, dw=0) == NODEV           # db alone
        assert backward(acc=acc, K=0, x=0, w=0, dx=0, dw=0, db=0) == OK
        assert backward(acc=acc, M=0, N=0, x=0, w=0, b=0, t=0, lse=0, dloss=0, dlse=0, dx=0, dw=0, db=0, ws=0, nws=0) == OK
    # no rows: dw and db are zeroed, or left alone where they are added to
    empty = dict(M=0, x=0, w=0, t=0, lse=0, dloss=0, dlse=0, dx=0)
    assert backward(**empty) == NODEV and backward(acc=0, **empty) == NODEV and backward(acc=1, **empty) == OK


@needs_lib
def test_workspace_sizes():
    for f in (la.cross_entropy_workspace_bytes, la.cross_entropy_backward_workspace_bytes):
        for M in (0, 1, 63, 5000, 1 << 24):
            for N in (0, 1, 777, 130000, (1 << 31) - 65536):
                for K in (0, 1, 4096, (1 << 22) - 8):
                    assert f(M, N, K) >= 0
        for bad in ((-1, 2, 3), ((1 << 24) + 1, 2, 3), (1, 1 << 31, 3), (1, 2, 1 << 22)):
            with pytest.raises(ValueError):
                f(*bad)
    # far under the logits' 2 M N bytes once the vocabulary is taken in pieces
    assert la.cross_entropy_backward_workspace_bytes(16384, 131072, 4096) < 2 * 16384 * 131072 // 4


def test_wrong_arguments_are_refused_before_the_library():
    x, w, t, v = torch.zeros(4, 8).half(), torch.zeros(6, 8).half(), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    bad = [lambda: la.linear_f16_cross_entropy(x, w, t),                             # on the host
           lambda: la.linear_f16_cross_entropy_backward(v, x, w, t, v),
           lambda: la.linear_f16_cross_entropy(x, w[:, :7], t), lambda: la.linear_f16_cross_entropy(x, w, t.int()),
           lambda: la.linear_f16_cross_entropy(x, w, t[:3]), lambda: la.linear_f16_cross_entropy(x, w, t, b=v.half()),
           lambda: la.linear_f16_cross_entropy_backward(v[:1].expand(4), x, w, t, v),  # a broadcast gradient
           lambda: la.linear_f16_cross_entropy_backward(v, x, w, t, v.double()),
           lambda: la.linear_f16_cross_entropy_backward(v, x, w, t, v, need_dx=False, need_dw=False),
           lambda: la.linear_f16_cross_entropy_backward_f32out(v, x, w, t, v, accumulate=True)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        la.linear_bf16_cross_entropy(x, w, t)


def test_the_gradients_formula_against_differences():
    gen = torch.Generator().manual_seed(0)
    M, N, K = 5, 11, 6
    x, w, b = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((M, K), (N, K), (N,)))
    target = torch.tensor([3, -100, 10, 11, 0])
    dloss, dlse = torch.randn(M, generator=gen).double(), torch.randn(M, generator=gen).double()

    def total(x, w, b):
        loss, lse, _ = ref.forward64(x, w, target, b)[0]
        return float((loss * dloss + lse * dlse).sum())

    got = ref.backward64(dloss, dlse, x, w, target, b, torch.float32)[0]
    h = 1e-5
    for i, v in enumerate((x, w, b)):
        for at in range(v.numel()):
            step = torch.zeros_like(v)
            step.view(-1)[at] = h
            args = [[x, w, b], [x, w, b]]
            args[0][i], args[1][i] = v + step, v - step
            slope = (total(*args[0]) - total(*args[1])) / (2 * h)
            # third derivatives of a few units times h^2 / 6, and 2^-52 of sums of some 20 over 2 h
            assert abs(slope - float(got[i].view(-1)[at])) <= 10 * h * h + 20 * 2.0 ** -52 / h


def test_the_bounds_catch_mistakes():
    """A loss or a gradient computed with a small mistake is outside its bound."""
    from train_refs import inside
    gen = torch.Generator().manual_seed(1)
    M, N, K = 12, 300, 64
    x, w = torch.randn(M, K, generator=gen).bfloat16(), (torch.randn(N, K, generator=gen) / 4).bfloat16()
    target = torch.randint(0, N, (M,), generator=gen)
    dloss = torch.ones(M)
    (loss, lse, _), (eo, el, _) = ref.forward64(x, w, target)
    inside(lse.float(), lse, el, "lse")
    short = ref.forward64(x, w[:-1], target % (N - 1))[0]
    for got, want, bound in ((short[1].float(), lse, el), ((loss * 1.0001).float(), loss, eo)):
        with pytest.raises(AssertionError):
            inside(got, want, bound, "planted")
    want, bound = ref.backward64(dloss, None, x, w, target, None, torch.bfloat16)
    other = ref.backward64(dloss, None, x, w, (target + 1) % N, None, torch.bfloat16)[0]
    for got, v, e in zip(other, want, bound):
        with pytest.raises(AssertionError):
            inside(got.bfloat16(), v, e, "planted")
    for v, e in zip(want, bound):
        inside(v.bfloat16(), v, e, "right")
        with pytest.raises(AssertionError):
            inside((v * 1.03).bfloat16(), v, e, "planted")


def test_the_native_tables_leave_what_is_not_plain_to_the_checks():
    """Anything but contiguous GPU tensors of the right types and sizes gives None (here: host tensors and
    wrong objects)."""
    if not os.path.exists(la.MARSHAL_PATH):
        pytest.skip("_marshal.so not built")
    n, x, f, target = la._marshal(), torch.zeros(4, 8, dtype=torch.float16), torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    for args in ((x, x, target, None, False), (x, x, target, x[0], True), (None, x, target, None, False), (x, 3, target, None, False),
                 (x, x, None, None, False), (x.to_sparse(), x, target, None, False), (x, x, target), ()):
        assert n.cross_entropy(*args) is None
    good = [f, x, x, target, f, None, None, True, True, False, False, False]
    for i, v in ((0, f), (0, None), (1, "x"), (3, f), (4, None), (5, 1)):
        assert n.cross_entropy_backward(*good[:i], v, *good[i + 1:]) is None
    assert n.cross_entropy_backward(*good[:5]) is None


@needs_lib
def test_workspaces_without_copies():
    """Operands that are read in place need no room for copies; others are refused with less."""
    fwd, bwd = la.cross_entropy_workspace_bytes, la.cross_entropy_backward_workspace_bytes
    assert fwd(1, 128259, 4096, True) < 1 << 16 and fwd(1, 128259, 4096) > 1 << 27
    assert bwd(20, 32000, 4096) - bwd(20, 32000, 4096, True) > 1 << 27
    for M in (0, 1, 63, 5000, 1 << 24):
        for N in (0, 1, 777, 130000, (1 << 31) - 65536):
            for K in (0, 1, 8, 4096, 4097, (1 << 22) - 8):
                for f in (fwd, bwd):
                    assert 0 <= f(M, N, K, True) <= f(M, N, K) and (K % 8 == 0 or f(M, N, K, True) == f(M, N, K))
    for bad in ((-1, 2, 8), (1, 1 << 31, 8), (1, 2, 1 << 22), (1, 2, -8)):
        for f in (fwd, bwd):
            with pytest.raises(ValueError):
                f(*bad, True)
    for call, size in ((forward, fwd(8, 32, 64, True)), (backward, bwd(8, 32, 64, True))):
        assert call(nws=size - 1) == SPACE
        for kw in (dict(w=W + 2), dict(ldw=65), dict(ldw=(1 << 22) + 8), *((dict(x=X + 8), dict(ldx=68)) if call is forward else ())):
            assert call(nws=size, **kw) == SPACE, kw
        if not torch.cuda.is_available():
            assert call(nws=size) == NODEV and call(nws=size, ldw=72, ldx=80) == NODEV
            if call is backward:                       # x is gathered from any layout
                assert call(nws=size, x=X + 2, ldx=65) == NODEV
