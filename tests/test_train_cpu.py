"""The gated block's, gradients' and norm's entry points without a GPU: every refusal comes from
the host before anything is enqueued, so fake device addresses never reach a kernel."""
import array
import os

import pytest
import torch

import linear_amd as la

needs_lib = pytest.mark.skipif(not os.path.exists(la.LIB_PATH), reason="liblinear_amd.so not built")
pytestmark = needs_lib

BASE = 0x7F0000000000
STEP = 0x1000000000
X, WG, WU, H, G, U, DH, DX, DWG, DWU, WS, DY, DB = (BASE + i * STEP for i in range(13))
NODEV = la.LINEAR_E_DEVICE
cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")


def gated(x=X, ldx=64, wg=WG, ldwg=64, wu=WU, ldwu=64, act=la.EPI_SILU, h=H, ldh=32, g=0, ldg=0, u=0, ldu=0, M=8, N=32,
          K=64, ws=0, nws=0, tag="f16"):
    fn = getattr(la._lib(), "linear_%s_gated" % tag)
    return fn(x, ldx, wg, ldwg, wu, ldwu, act, h, ldh, g, ldg, u, ldu, M, N, K, ws, nws, None)


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), la.LINEAR_E_SHAPE), (dict(N=1 << 31), la.LINEAR_E_SHAPE), (dict(K=(1 << 31) - 1), la.LINEAR_E_SHAPE),
    (dict(act=0), la.LINEAR_E_VALUE), (dict(act=la.EPI_MUL), la.LINEAR_E_VALUE), (dict(act=7), la.LINEAR_E_VALUE),
    (dict(x=0), la.LINEAR_E_NULL), (dict(wg=0), la.LINEAR_E_NULL), (dict(wu=0), la.LINEAR_E_NULL),
    (dict(h=0), la.LINEAR_E_NULL),
    (dict(ldx=63), la.LINEAR_E_STRIDE), (dict(ldwg=63), la.LINEAR_E_STRIDE), (dict(ldwu=1), la.LINEAR_E_STRIDE),
    (dict(ldh=31), la.LINEAR_E_STRIDE), (dict(g=G, ldg=31), la.LINEAR_E_STRIDE), (dict(u=U, ldu=31), la.LINEAR_E_STRIDE),
    (dict(ldx=1 << 31), la.LINEAR_E_STRIDE),
    (dict(h=X + 10), la.LINEAR_E_ALIAS), (dict(h=WU - 2), la.LINEAR_E_ALIAS), (dict(g=H, ldg=32), la.LINEAR_E_ALIAS),
    (dict(g=G, ldg=32, u=G + 64, ldu=32), la.LINEAR_E_ALIAS), (dict(u=X, ldu=32), la.LINEAR_E_ALIAS),
    (dict(K=63), la.LINEAR_E_NULL), (dict(K=63, ws=WS, nws=64), la.LINEAR_E_WORKSPACE),
    (dict(K=63, ws=WS + 8, nws=1 << 20), la.LINEAR_E_WORKSPACE), (dict(K=63, ws=H, nws=1 << 20), la.LINEAR_E_ALIAS),
])
def test_gated_refusals(tag, kw, code):
    assert gated(tag=tag, **kw) == code


@cpu_only
def test_gated_calls_that_pass_the_checks():
    assert gated() == NODEV
    assert gated(wu=WG) == NODEV                       # one weight for both projections is only read
    assert gated(g=G, ldg=32) == NODEV                 # one projection kept
    assert gated(x=0, wg=0, wu=0, K=0, ldx=0, ldwg=0, ldwu=0) == NODEV
    assert gated(K=63, ws=WS, nws=1 << 20) == NODEV and gated(K=63, M=3) == NODEV
    assert gated(M=0, x=0, h=0) == la.LINEAR_OK
    assert gated(N=0, wg=0, h=0) == la.LINEAR_OK


def gated_backward(dh=DH, lddh=32, x=X, ldx=64, wg=WG, ldwg=64, wu=WU, ldwu=64, g=G, ldg=32, u=U, ldu=32, act=la.EPI_SILU,
                   dx=DX, lddx=64, dwg=DWG, lddwg=64, dwu=DWU, lddwu=64, M=8, N=32, K=64, ws=WS, nws=1 << 20, tag="f16"):
    fn = getattr(la._lib(), "linear_%s_gated_backward" % tag)
    return fn(dh, lddh, x, ldx, wg, ldwg, wu, ldwu, g, ldg, u, ldu, act, dx, lddx, dwg, lddwg, dwu, lddwu, M, N, K, ws, nws,
              None)


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), la.LINEAR_E_SHAPE), (dict(K=1 << 31), la.LINEAR_E_SHAPE), (dict(act=1), la.LINEAR_E_VALUE),
    (dict(dh=0), la.LINEAR_E_NULL), (dict(x=0), la.LINEAR_E_NULL), (dict(wg=0), la.LINEAR_E_NULL),
    (dict(g=0), la.LINEAR_E_NULL), (dict(u=0), la.LINEAR_E_NULL), (dict(dwg=0), la.LINEAR_E_NULL),
    (dict(dwu=0), la.LINEAR_E_NULL), (dict(dx=0, dwg=0, dwu=0), la.LINEAR_E_NULL), (dict(ws=0), la.LINEAR_E_NULL),
    (dict(lddh=31), la.LINEAR_E_STRIDE), (dict(ldg=31), la.LINEAR_E_STRIDE), (dict(lddwu=63), la.LINEAR_E_STRIDE),
    (dict(nws=10), la.LINEAR_E_WORKSPACE), (dict(ws=WS + 8), la.LINEAR_E_WORKSPACE),
    (dict(dx=DWG, lddx=64), la.LINEAR_E_ALIAS), (dict(dwu=DWG + 64), la.LINEAR_E_ALIAS), (dict(dwg=WG), la.LINEAR_E_ALIAS),
    (dict(ws=DX), la.LINEAR_E_ALIAS), (dict(ws=DH), la.LINEAR_E_ALIAS), (dict(dx=X), la.LINEAR_E_ALIAS),
])
def test_gated_backward_refusals(tag, kw, code):
    assert gated_backward(tag=tag, **kw) == code


@cpu_only
def test_gated_backward_calls_that_pass_the_checks():
    assert gated_backward() == NODEV
    assert gated_backward(dx=0, wg=0, wu=0) == NODEV           # weight gradients alone do not read the weights
    assert gated_backward(dwg=0, dwu=0, x=0) == NODEV
    assert gated_backward(K=0) == la.LINEAR_OK
    assert gated_backward(M=0, dh=0, x=0, g=0, u=0, dx=0) == NODEV      # dwg and dwu are zeroed
    assert gated_backward(N=0, dh=0, wg=0, wu=0, g=0, u=0, dwg=0, dwu=0) == NODEV


# a size whose contraction is split, so that the call needs a workspace
SPLIT = dict(M=16, N=4096, lddy=4096)


def backward_input(dy=DY, lddy=32, w=WG, ldw=64, dx=DX, lddx=64, M=8, N=32, K=64, ws=WS, nws=1 << 20):
    return la._lib().linear_f16_backward_input(dy, lddy, w, ldw, dx, lddx, M, N, K, ws, nws, None)


def backward_weight(dy=DY, lddy=32, x=X, ldx=64, dw=DWG, lddw=64, db=DB, M=8, N=32, K=64, ws=WS, nws=1 << 20):
    return la._lib().linear_bf16_backward_weight(dy, lddy, x, ldx, dw, lddw, db, M, N, K, ws, nws, None)


def backward_weight_f32(acc=0, dw=DWG, db=DB, **kw):
    return la._lib().linear_f16_backward_weight_f32out(DY, 32, X, 64, dw, 64, db, acc, 8, 32, 64, WS, 1 << 20, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), la.LINEAR_E_SHAPE), (dict(dy=0), la.LINEAR_E_NULL), (dict(w=0), la.LINEAR_E_NULL),
    (dict(dx=0), la.LINEAR_E_NULL), (dict(lddy=31), la.LINEAR_E_STRIDE), (dict(ldw=63), la.LINEAR_E_STRIDE),
    (dict(lddx=63), la.LINEAR_E_STRIDE), (dict(dx=DY), la.LINEAR_E_ALIAS), (dict(dx=WG + 64), la.LINEAR_E_ALIAS),
    (dict(nws=0, **SPLIT), la.LINEAR_E_WORKSPACE), (dict(ws=WS + 4, **SPLIT), la.LINEAR_E_WORKSPACE),
    (dict(ws=DX, **SPLIT), la.LINEAR_E_ALIAS), (dict(ws=0, **SPLIT), la.LINEAR_E_NULL),
])
def test_backward_input_refusals(kw, code):
    assert backward_input(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), la.LINEAR_E_SHAPE), (dict(dy=0), la.LINEAR_E_NULL), (dict(x=0), la.LINEAR_E_NULL),
    (dict(dw=0), la.LINEAR_E_NULL), (dict(lddy=31), la.LINEAR_E_STRIDE), (dict(ldx=63), la.LINEAR_E_STRIDE),
    (dict(lddw=63), la.LINEAR_E_STRIDE), (dict(dw=X), la.LINEAR_E_ALIAS), (dict(db=DY + 62), la.LINEAR_E_ALIAS),
    (dict(db=DWG + 128), la.LINEAR_E_ALIAS), (dict(M=4096, nws=100), la.LINEAR_E_WORKSPACE),
    (dict(M=4096, ws=DB), la.LINEAR_E_ALIAS), (dict(M=4096, ws=0), la.LINEAR_E_NULL),
])
def test_backward_weight_refusals(kw, code):
    assert backward_weight(**kw) == code


@cpu_only
def test_backward_calls_that_pass_the_checks():
    assert backward_input() == NODEV and backward_weight() == NODEV and backward_weight(db=0) == NODEV
    assert backward_weight_f32() == NODEV and backward_weight_f32(acc=1) == NODEV
    assert backward_input(M=0, dx=0) == la.LINEAR_OK and backward_input(K=0, dx=0) == la.LINEAR_OK
    assert backward_input(N=0, dy=0, w=0) == NODEV                     # dx is zeroed
    assert backward_weight(N=0, dw=0, db=0) == la.LINEAR_OK
    assert backward_weight(M=0, dy=0, x=0) == NODEV                    # dw and db are zeroed
    assert backward_weight(K=0, x=0, dw=0) == NODEV                    # db alone
    assert backward_weight(K=0, x=0, dw=0, db=0) == la.LINEAR_OK


def table(*rows):
    return array.array("q", [v for r in rows for v in r])


def norm(rows, count=None, out=H, ws=WS, nws=1 << 20):
    t = table(*rows)
    return la._lib().linear_grad_norm(t.buffer_info()[0], len(rows) if count is None else count, out, ws, nws, None)


def clip(rows, out=None, norm_=H, max_norm=1.0, count=None):
    t = table(*rows)
    o = None if out is None else table(*out)
    return la._lib().linear_grad_clip(t.buffer_info()[0], o.buffer_info()[0] if o else None,
                                      len(rows) if count is None else count, norm_, max_norm, None)


A = (X, 4, 8, 8, 0)
B = (WG, 1, 100, 100, 2)


@pytest.mark.parametrize("rows,kw,code", [
    ([A], dict(count=-1), la.LINEAR_E_SHAPE), ([A], dict(count=la.GRAD_MAX_TENSORS + 1), la.LINEAR_E_SHAPE),
    ([(X, -1, 8, 8, 0)], {}, la.LINEAR_E_SHAPE), ([(X, 1 << 31, 8, 8, 0)], {}, la.LINEAR_E_SHAPE),
    ([(X, 4, 8, 8, 3)], {}, la.LINEAR_E_VALUE), ([(X, 4, 8, 8, -1)], {}, la.LINEAR_E_VALUE),
    ([A, (0, 4, 8, 8, 0)], {}, la.LINEAR_E_NULL), ([A], dict(out=0), la.LINEAR_E_NULL), ([A], dict(ws=0), la.LINEAR_E_NULL),
    ([(X, 4, 8, 7, 0)], {}, la.LINEAR_E_STRIDE), ([A], dict(nws=8), la.LINEAR_E_WORKSPACE),
    ([A], dict(ws=WS + 8), la.LINEAR_E_WORKSPACE), ([A], dict(out=X + 4), la.LINEAR_E_ALIAS),
    ([A], dict(ws=X - 16), la.LINEAR_E_ALIAS), ([A], dict(out=WS), la.LINEAR_E_ALIAS),
])
def test_norm_refusals(rows, kw, code):
    assert norm(rows, **kw) == code


@pytest.mark.parametrize("rows,kw,code", [
    ([A], dict(max_norm=-1.0), la.LINEAR_E_VALUE), ([A], dict(max_norm=float("nan")), la.LINEAR_E_VALUE),
    ([A], dict(norm_=0), la.LINEAR_E_NULL), ([A], dict(count=-1), la.LINEAR_E_SHAPE),
    ([A], dict(out=[(H, 4, 8, 8, 1)], norm_=WS), la.LINEAR_E_VALUE),
    ([A], dict(out=[(H, 4, 7, 8, 0)], norm_=WS), la.LINEAR_E_SHAPE),
    ([A], dict(out=[(0, 4, 8, 8, 0)]), la.LINEAR_E_NULL),
    ([A], dict(norm_=X), la.LINEAR_E_ALIAS),
    ([A, A], {}, la.LINEAR_E_ALIAS),                               # the same tensor twice, in place
    ([A, (X + 62, 1, 4, 4, 0)], {}, la.LINEAR_E_ALIAS),            # the tail of one is the head of another
    ([A, B], dict(out=[(H, 4, 8, 8, 0), (H + 60, 1, 100, 100, 2)], norm_=WS), la.LINEAR_E_ALIAS),
    ([A, B], dict(out=[(WG + 8, 4, 8, 8, 0), (U, 1, 100, 100, 2)]), la.LINEAR_E_ALIAS),
    ([A], dict(out=[(X + 2, 4, 8, 8, 0)]), la.LINEAR_E_ALIAS),     # shifted onto itself
    ([A], dict(out=[(X, 4, 8, 9, 0)]), la.LINEAR_E_ALIAS),         # same start, other stride
    ([A], dict(out=[(H, 4, 8, 8, 0)]), la.LINEAR_E_ALIAS),         # the norm inside an output
])
def test_clip_refusals(rows, kw, code):
    assert clip(rows, **kw) == code


@cpu_only
def test_norm_and_clip_calls_that_pass_the_checks():
    assert norm([A, B]) == NODEV and norm([A, A]) == NODEV and norm([], nws=0) == NODEV
    assert norm([(0, 0, 8, 8, 0), A]) == NODEV
    assert clip([A, B]) == NODEV and clip([]) == la.LINEAR_OK
    assert clip([A, A], out=[(U, 4, 8, 8, 0), (G, 4, 8, 10, 0)]) == NODEV
    assert clip([A, B], out=[A, (U, 1, 100, 100, 2)]) == NODEV     # one in place, one not
    assert clip([A], max_norm=float("inf")) == NODEV and clip([A], max_norm=0.0) == NODEV


def test_workspace_sizes():
    assert la.gated_workspace_bytes(5, 65, 7) >= 5 * 128 * 2 * 2
    assert la.backward_workspace_bytes(4096, 1000, 8) >= 1000 * 4
    assert la.grad_workspace_bytes(0) == 0 and la.grad_workspace_bytes(65) >= 2 * 8
    assert la.gated_forward_workspace_bytes(4096, 14336, 4096) == 0
    assert la.gated_forward_workspace_bytes(30, 20, 9) >= (30 + 40) * 16 * 2
    assert la.backward_workspace_bytes(100, 90, 81) >= (100 * 96 + 90 * 88) * 2
    for f in (la.gated_forward_workspace_bytes, la.gated_workspace_bytes, la.backward_workspace_bytes):
        for zero in range(3):                     # any size may be zero, beside large ones
            for other in (1, 63, 5000, 70000):
                sizes = [other] * 3
                sizes[zero] = 0
                assert f(*sizes) >= 0
        assert f(0, 0, 0) >= 0
    for f in (la.gated_forward_workspace_bytes, la.gated_workspace_bytes, la.backward_workspace_bytes):
        with pytest.raises(ValueError):
            f(-1, 2, 3)
    with pytest.raises(ValueError):
        la.gated_workspace_bytes(1 << 31, 8, 8)
    with pytest.raises(ValueError):
        la.grad_workspace_bytes(la.GRAD_MAX_TENSORS + 1)
    for code in (la.LINEAR_E_VALUE, la.LINEAR_E_MEMORY):
        assert la.linear_status_string(code) != "unknown status"


def test_host_tensors_and_wrong_arguments_are_refused_before_the_library():
    x, w, h = torch.zeros(4, 8).half(), torch.zeros(6, 8).half(), torch.zeros(4, 6).half()
    calls = [lambda: la.linear_f16_gated(x, w, w), lambda: la.linear_f16_gated_backward(h, x, w, w, h, h),
             lambda: la.linear_f16_backward_input(h, w), lambda: la.linear_f16_backward_weight(h, x),
             lambda: la.linear_f16_backward_weight_f32out(h, x, bias=True), lambda: la.linear_grad_norm([x, w]),
             lambda: la.linear_grad_clip([x], torch.zeros(1), 1.0)]
    for c in calls:
        with pytest.raises(ValueError):
            c()
    with pytest.raises(TypeError):
        la.linear_bf16_gated(x, w, w)
    with pytest.raises(ValueError):
        la.linear_f16_gated(x, w, w[:5])
    with pytest.raises(ValueError):
        la.linear_f16_gated_backward(h, x, w, w, h, h[:3])
    with pytest.raises(ValueError):
        la.linear_f16_gated_backward(h, x, w, w, h, h, need_dx=False, need_dw=False)
    with pytest.raises(ValueError):
        la.linear_f16_backward_weight_f32out(h, x, accumulate=True)
    with pytest.raises(TypeError):
        la.linear_grad_norm([x.double()])
    with pytest.raises(ValueError):
        la.linear_grad_norm([x.t()])
    with pytest.raises(ValueError):
        la.linear_grad_norm([])
    with pytest.raises(ValueError):
        la.linear_grad_clip([x], torch.zeros(1), 1.0, out=[w])


@cpu_only
def test_columns_side_by_side_in_one_tensor():
    """Matrices of one row stride that share rows but no column do not overlap; one column in
    common, or rows of another length, do."""
    half = dict(ldg=64, ldu=64)
    assert gated(g=G, u=G + 64, **half) == NODEV and gated(u=G, g=G + 64, **half) == NODEV
    assert gated(h=X + 128, ldh=96, ldx=96) == NODEV                      # behind x's columns
    assert gated(g=G, u=G + 62, **half) == la.LINEAR_E_ALIAS and gated(u=G, g=G + 62, **half) == la.LINEAR_E_ALIAS
    assert gated(g=G, u=G + 66, **half) == la.LINEAR_E_ALIAS              # into the next row's first column
    assert gated(g=G, u=G + 64, ldg=64, ldu=65) == la.LINEAR_E_ALIAS
    assert gated(g=G, u=G + 64 + 128 * 3, **half) == NODEV                # three rows further down
    assert gated_backward(dwg=DWG, dwu=DWG + 128, lddwg=128, lddwu=128) == NODEV
    assert gated_backward(ws=DWG + 128, nws=10 ** 6, lddwg=10 ** 6) == la.LINEAR_E_ALIAS
