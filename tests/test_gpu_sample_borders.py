"""Sampling where its ways through a row change: floors at zero, and rows that its sample and lists do not settle, in
clusters of every size (checked as in test_gpu_sample)."""
import pytest
import torch

from test_gpu_sample import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(1, 8193), (7, 9000), (1, 50257), (160, 9000), (3, 262144)])
def test_the_floor_of_min_p_at_zero(R, V, dtype):
    """Rows whose largest value is 0 or -0 and min_p 1: the zeros are kept, of either sign, wherever top_p would cut."""
    g = torch.Generator().manual_seed(V + R)
    x = torch.randn(R, V, generator=g)
    x = (x - x.amax(1, keepdim=True)).to(dtype)
    zeros = torch.randint(0, V, (R, 5), generator=g)
    signs = torch.where(torch.rand(R, 5, generator=g) < 0.5, 0.0, -0.0).to(dtype)
    x.scatter_(1, zeros, signs)
    x[0] = torch.where(x[0] == 0, -0.0, x[0])
    u = torch.rand(R, generator=g)
    for p in (0.5, 0.7, 0.9, 0.99, 1.0):
        tok, lp, kept = check(x, u, p=p, mp=1.0)
        if p == 1.0:
            assert torch.equal(kept, (x == 0).sum(1).int())
        assert bool((x.gather(1, tok.long()[:, None]) == 0).all())
    # floors just below zero, and settings of each row's own
    check(x, u, T=0.5, p=0.9, mp=1 - 2.0 ** -24)
    check(x, u, T=1e-12, p=0.999999, mp=0.5)
    R2 = torch.arange(R)
    check(x, u, p=torch.where(R2 % 2 == 0, 0.9, 1.0), mp=torch.where(R2 % 3 == 0, 1.0, 0.25))
