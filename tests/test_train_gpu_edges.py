"""Edges of the gated block's and the gradients' calls on the GPU."""
import pytest
import torch

import linear_amd as la
import train_refs as ref
from test_train_gpu import DEV, IDS, TYPES, fn, infinite, make, padded, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_gradients_of_an_empty_batch_with_one_group_wanted(t):
    z = lambda *s: torch.zeros(*s, dtype=t, device=DEV)          # noqa: E731
    back = fn("gated_backward", t)
    dx, dwg, dwu = back(z(0, 7), z(0, 8), z(7, 8), z(7, 8), z(0, 7), z(0, 7), need_dw=False)
    assert dx.shape == (0, 8) and dwg is None and dwu is None
    dx, dwg, dwu = back(z(5, 0), z(5, 8), z(0, 8), z(0, 8), z(5, 0), z(5, 0), need_dx=False)
    assert dx is None and dwg.shape == dwu.shape == (0, 8)
    dx, dwg, dwu = back(z(0, 7), z(0, 8), z(7, 8), z(7, 8), z(0, 7), z(0, 7), need_dx=False,
                        dwg=torch.full((7, 8), 3.0, dtype=t, device=DEV), dwu=torch.full((7, 8), 3.0, dtype=t, device=DEV))
    assert dx is None and not dwg.any() and not dwu.any()
    dx, dwg, dwu = back(z(5, 0), z(5, 8), z(0, 8), z(0, 8), z(5, 0), z(5, 0), need_dw=False,
                        dx=torch.full((5, 8), 3.0, dtype=t, device=DEV))
    assert not dx.any() and dwg is None and dwu is None


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_adding_an_empty_batch_leaves_the_sums(t):
    z = lambda *s: torch.zeros(*s, dtype=t, device=DEV)          # noqa: E731
    dw, db = torch.full((7, 8), -0.0, device=DEV), torch.full((7,), -0.0, device=DEV)
    fn("backward_weight_f32out", t)(z(0, 7), z(0, 8), bias=True, out=dw, db=db, accumulate=True)
    assert bool(dw.signbit().all()) and bool(db.signbit().all())


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(1, 72, 136), (9, 264, 136), (32, 1032, 264), (16, 4104, 72), (20, 77, 93), (33, 72, 136),
                                   (300, 264, 136)])
@pytest.mark.parametrize("aligned", [True, False])
def test_infinite_weights_and_inputs_of_the_gated_gradients(M, N, K, t, aligned):
    """An infinity of a weight or of x gives its column of dx, or of dwg and dwu, infinities of the
    gradient's sign, whatever the number of rows; other columns keep their words."""
    x, wg, wu, dh = make(M, N, K, t)
    _, g, u = fn("gated", t)(x, wg, wu, keep=True)
    dh.fill_(0.5)
    u = u + torch.where(u < 0, -1.0, 1.0).to(t)             # no gradient is zero
    if not aligned:
        x, wg, wu = (padded(v, 1, 1)[0] for v in (x, wg, wu))
    back = lambda: fn("gated_backward", t)(dh, x, wg, wu, g, u)          # noqa: E731
    clean = back()
    _, slope, _, _ = ref.act64(la.EPI_SILU, g.double())
    act = ref.act64(la.EPI_SILU, g.double())[0]
    signs = (dh.double() * u.double() * slope).sign(), (dh.double() * act).sign()
    assert all(bool(s.all()) for s in signs)
    k = K // 2
    cols = torch.arange(K, device=DEV) != k
    for w, s, n in ((wg, signs[0], 0), (wu, signs[1], N - 1)):
        kept = w[n, k].clone()
        w[n, k] = float("-inf")
        dx = back()[0]
        assert same(dx[:, k], infinite(-s[:, n])) and torch.equal(dx[:, cols], clean[0][:, cols])
        w[n, k] = kept
    x[M - 1, k] = float("inf")
    _, dwg, dwu = back()
    for got, c, s in ((dwg, clean[1], signs[0]), (dwu, clean[2], signs[1])):
        assert same(got[:, k], infinite(s[M - 1])) and torch.equal(got[:, cols], c[:, cols])
    x[M - 1, k] = float("nan")
    _, dwg, dwu = back()
    assert bool(dwg[:, k].isnan().all()) and bool(dwu[:, k].isnan().all())
