"""The one-row kernel at infinite inputs."""
import pytest
import torch

import linear_amd as la

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 8), (1, 768), (1, 4096), (1, 4104), (1, 9000), (2, 520), (16, 776), (300, 1000)])
def test_infinite_input(M, K, t):
    """One infinity in x: its row of y is infinite, with the weights' signs, NaN where a weight is 0."""
    gen = torch.Generator().manual_seed(K)
    x, w = (torch.randn(*s, generator=gen).to(t).cuda() for s in ((M, K), (72, K)))
    tag = "bf16" if t == torch.bfloat16 else "f16"
    for k in (0, K // 2, K - 1):
        v = x.clone()
        v[M - 1, k] = float("inf")
        want = w[:, k].double().sign() * float("inf")
        for name in ("nobias", "f32out"):
            got = getattr(la, "linear_%s_%s" % (tag, name))(v, w)[M - 1].double()
            assert bool(((got == want) | (got.isnan() & want.isnan())).all()), (name, k)
