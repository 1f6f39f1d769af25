"""Outputs with more columns than one launch's threads can count (2^32 of them), in every kernel that
takes few rows.  Words -2 .. 2, so every sum is exact, and every output is compared."""
import pytest
import torch

import linear_amd as la
import train_refs as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
K = 8


def ints(gen, *shape):
    return torch.randint(-2, 3, shape, generator=gen, device=DEV, dtype=torch.int8).half()


def each_part(N, step=1 << 24):
    return (slice(n, min(n + step, N)) for n in range(0, N, step))


@pytest.mark.parametrize("shift", [0, 1], ids=["aligned", "any layout"])
def test_one_row_of_many_outputs(shift):
    N = (1 << 26) + 72                         # 64 threads an output in the one-row kernels
    gen = torch.Generator(device=DEV).manual_seed(1)
    store = ints(gen, 1, K + shift)
    x, w, b = store[:, shift:], ints(gen, N, K), ints(gen, N)
    y, p, s = la.linear_f16(x, w, b), la.linear_f16_nobias(x, w), la.linear_f16_f32out(x, w)
    e = la.linear_f16_epilogue(x, w, [la.EPI_BIAS, la.EPI_MUL], bias=b, mul=p)
    h, g, u = la.linear_f16_gated(x, w, w, keep=True)
    for n in each_part(N):
        want = (x.double() @ w[n].double().t())
        assert torch.equal(p[:, n].double(), want) and torch.equal(s[:, n].double(), want)
        assert torch.equal(y[:, n].double(), want + b[n].double())
        assert torch.equal(e[:, n].double(), (want + b[n].double()) * want)
        assert torch.equal(g[:, n].double(), want) and torch.equal(u[:, n], g[:, n])
        # g and u are exact: h is off by the activation's FP32 evaluation, the product's (S) and its own
        # rounding (u relative, or half the spacing of the subnormals, 2^-25: SiLU of -16 is 2e-6)
        act, _, r, _ = ref.act64(la.EPI_SILU, want)
        bound = ((r + ref.S) * act.abs() + ref.FLOOR) * want.abs()
        ref.inside(h[:, n], act * want, ref.rounded(act * want, bound, h.dtype), "h")


def test_few_rows_of_more_outputs():
    M, N = 2, (1 << 28) + 72                   # 32 threads an output in the 16-row kernels
    gen = torch.Generator(device=DEV).manual_seed(2)
    x, w = ints(gen, M, K), ints(gen, N, K)
    y = la.linear_f16_nobias(x, w)
    _, g, _ = la.linear_f16_gated(x, w, w, keep=True)
    for n in each_part(N):
        want = x.double() @ w[n].double().t()
        assert torch.equal(y[:, n].double(), want) and torch.equal(g[:, n].double(), want)


def test_bias_gradient_of_many_columns():
    M, N = 3, (1 << 28) + 72                   # 16 threads a column
    gen = torch.Generator(device=DEV).manual_seed(3)
    dy = ints(gen, M, N)
    _, db = la.linear_f16_backward_weight(dy, dy[:, :0], bias=True)
    out = torch.empty(N, 0, device=DEV)
    wide = torch.ones(N, device=DEV)
    la.linear_f16_backward_weight_f32out(dy, dy[:, :0], bias=True, accumulate=True, out=out, db=wide)
    for n in each_part(N):
        want = dy[:, n].double().sum(0)
        assert torch.equal(db[n].double(), want) and torch.equal(wide[n].double(), want + 1)
