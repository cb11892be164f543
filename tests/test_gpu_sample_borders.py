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


def clumped(g, R, V, dtype):
    """Logits of some 20 values: runs of equal ones longer than any list."""
    return (torch.randn(R, V, generator=g) * 4).round().div(4).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(160, 40000), (160, 8193), (100, 32000), (100, 40000), (153, 65536), (9, 50257), (2, 262144)])
def test_cuts_that_no_list_holds(R, V, dtype):
    """The border by count, by mass and by both in clumps of equal values and among more values than the lists hold, with
    one CTA to a row and with clusters of 2 to 16."""
    g = torch.Generator().manual_seed(R + V)
    u = torch.rand(R, generator=g)
    some = torch.arange(R)
    k = torch.where(some % 4 == 0, 0, (V * (0.3 + 0.6 * torch.rand(R, generator=g))).int()).int()
    p = torch.where(some % 4 == 1, 1.0, 0.2 + 0.79 * torch.rand(R, generator=g))
    mp = torch.where(some % 3 == 2, 0.01 * torch.rand(R, generator=g), 0.0)
    for x in (clumped(g, R, V, dtype), torch.randn(R, V, generator=g).to(dtype)):
        first = check(x, u, k=k, p=p, mp=mp)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(check(x[:8], u[:8], k=k[:8], p=p[:8], mp=mp[:8]),
                                                         [t[:8] for t in first]))


@pytest.mark.parametrize("R,V", [(160, 8193), (256, 16385), (256, 32769), (160, 50257), (160, 65536), (100, 32000)])
def test_sampled_rows_of_one_cta(R, V):
    g = torch.Generator().manual_seed(R + 2 * V)
    x = torch.randn(R, V, generator=g) * torch.exp(2.4 * torch.rand(R, 1, generator=g) - 0.7)
    some = torch.arange(R)
    k = torch.where(some % 4 == 0, (2 ** (9 * torch.rand(R, generator=g))).int(), 0).int()
    p = torch.where(some % 4 < 3, 0.5 + 0.499 * torch.rand(R, generator=g), 1.0)
    mp = torch.where(some % 3 == 0, 0.1 * torch.rand(R, generator=g) ** 2, 0.0)
    u = torch.rand(R, generator=g)
    check(x, u, k=k, p=p, mp=mp)
    check(x.to(torch.bfloat16), u, k=k, p=p, mp=mp)
    # every other 128 values higher: a sample of every second misses the border
    high = 0.3 * torch.randn(R, V, generator=g) + 4.0 * (torch.arange(V) // 128 % 2 == 1)
    check(high, u, p=p, mp=torch.where(some % 2 == 0, 2.0 ** -9, 0.0))
