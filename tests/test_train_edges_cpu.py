"""Edges of the gated block's and the gradients' entry points that need no GPU: sizes of zero, the
largest sizes, and operands that a call does not read."""
import pytest

import linear_amd as la
from test_train_cpu import DB, DWG, gated_backward, needs_lib

pytestmark = needs_lib


@pytest.mark.parametrize("tag", ["f16", "bf16"])
def test_gradients_of_an_empty_batch_with_one_group_wanted(tag):
    """An empty output has no address, like one that is not wanted: nothing is left to compute."""
    none = dict(dx=0, dwg=0, dwu=0, tag=tag)
    assert gated_backward(M=0, dh=0, x=0, g=0, u=0, **none) == la.LINEAR_OK
    assert gated_backward(N=0, dh=0, wg=0, wu=0, g=0, u=0, **none) == la.LINEAR_OK
    assert gated_backward(K=0, x=0, wg=0, wu=0, **none) == la.LINEAR_OK
    assert gated_backward(**none) == la.LINEAR_E_NULL                       # every output has elements
    assert gated_backward(M=0, dh=0, x=0, g=0, u=0, dx=0, dwg=0, tag=tag) == la.LINEAR_E_NULL   # one of a pair


@pytest.mark.parametrize("tag", ["f16", "bf16"])
def test_adding_an_empty_batch_leaves_the_sums(tag):
    """Nothing is enqueued: adding a zero would turn a -0 into +0."""
    fn = getattr(la._lib(), "linear_%s_backward_weight_f32out" % tag)
    assert fn(0, 32, 0, 64, DWG, 64, DB, 1, 0, 32, 64, 0, 0, None) == la.LINEAR_OK
    assert fn(0, 32, 0, 64, 0, 64, DB, 1, 0, 32, 64, 0, 0, None) == la.LINEAR_E_NULL


def test_sizes_of_the_gated_backward_workspace():
    """dg | du is a matrix of twice N columns (N in whole slices of 64), each row below 2^31 words: the
    workspace call refuses the sizes that the backward call refuses."""
    top = (1 << 30) - 64
    for M in (1, 5000):
        assert la.gated_workspace_bytes(M, top, 1) > 4 * M * top
        for N in (top + 1, 1 << 30, (1 << 31) - 65536):
            with pytest.raises(ValueError):
                la.gated_workspace_bytes(M, N, 1)
            assert gated_backward(M=M, N=N, K=1, ldx=1, ldwg=1, ldwu=1, lddx=1, lddwg=1, lddwu=1, lddh=N, ldg=N, ldu=N,
                                  nws=1 << 62) == la.LINEAR_E_SHAPE
