"""Lengths and counts at the ends of int32: reported, and nothing of those sequences is read or written."""
import pytest
import torch

import kv8_ref
from block_diffusion_text_gb300 import dg
from test_gpu_kv8 import filled, rows, state

pytestmark = pytest.mark.gpu

LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("hd", [32, 128])
@pytest.mark.parametrize("row0", [0, 1, 70])
def test_read_of_lengths_out_of_range(hd, row0):
    """A negative length leaves its sequence's rows as they are, one past the capacity reads up to it."""
    g = torch.Generator().manual_seed(60)
    c = filled(g, 5, 2, 100, hd, [100] * 5)
    K, V, Ke, Ve, _ = state(c)
    c.len = torch.tensor([LOW, 100, -1, LOW + 40, HIGH], dtype=torch.int32)
    out = [torch.full((5, 2, 120, hd), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dg.kv8_read(c, row0, 120, out=out)
    assert c.status() == dg.DG_ERR_CAPACITY
    for o, codes, exps in zip(out, (K, V), (Ke, Ve)):
        want = torch.full((5, 2, 120, hd), 7.0, dtype=torch.float64)
        for b in (1, 4):
            want[b, :, :100 - row0] = kv8_ref.values(codes, exps)[b, :, row0:]
        assert torch.equal(o.cpu().double(), want)


def test_append_of_lengths_and_counts_out_of_range():
    g = torch.Generator().manual_seed(61)
    c = filled(g, 6, 2, 100, 64, [10] * 6)
    before = state(c)
    c.len = torch.tensor([LOW, HIGH, 10, 10, HIGH - 3, 95], dtype=torch.int32)
    counts = torch.tensor([5, 5, LOW, HIGH, HIGH, 5], dtype=torch.int32).cuda()
    k, v = rows(g, 6, 2, 5, 64), rows(g, 6, 2, 5, 64)
    dg.kv8_append(c, k.cuda(), v.cuda(), counts=counts)
    assert c.status() in (dg.DG_ERR_CAPACITY, dg.DG_ERR_ARG)
    after = state(c)
    for x, y in zip(before[:4], after[:4]):
        assert torch.equal(x[:5], y[:5])
    wK, _ = kv8_ref.append(before[0], before[2], k, after[4], [0, 0, 0, 0, 0, 5])
    assert torch.equal(after[0], wK)


@pytest.mark.parametrize("C,cap", [(1, 100), (1, 5000), (200, 100), (200, 3000), (40, 20000)])
def test_attention_of_lengths_out_of_range(C, cap):
    """A negative length counts as none and one past the capacity as the capacity, with the status word set."""
    g = torch.Generator().manual_seed(62)
    c = filled(g, 3, 1, cap, 64, [cap] * 3)
    q, k, v = rows(g, 3, 2, C, 64).cuda(), rows(g, 3, 1, C, 64).cuda(), rows(g, 3, 1, C, 64).cuda()
    c.len = torch.tensor([0, cap, 60], dtype=torch.int32)
    want = dg.kv8_attention(c, q, k, v)
    assert c.status() == 0
    c.len = torch.tensor([LOW, HIGH, 60], dtype=torch.int32)
    assert torch.equal(dg.kv8_attention(c, q, k, v), want)
    assert c.status() == dg.DG_ERR_CAPACITY
