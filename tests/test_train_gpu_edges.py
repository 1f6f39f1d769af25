"""Edges of the gated block's and the gradients' calls on the GPU."""
import pytest
import torch

import linear_amd as la
from test_train_gpu import DEV, IDS, TYPES, fn

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
