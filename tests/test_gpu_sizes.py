"""Sizes beyond 32 bits are refused: cut to 32 bits they would name another, smaller call."""
import pytest
import torch

from test_gpu_moe_tokens import drawn
from block_diffusion_text_gb300 import dg

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def refused(call):
    with pytest.raises(dg.DgError) as e:
        call()
    assert e.value.code == dg.DG_ERR_SHAPE


def test_logits():
    u = torch.zeros(1, device="cuda")
    refused(lambda: dg.sample(torch.empty(1, (1 << 32) + 5, dtype=BF, device="cuda"), u))
    R = (1 << 32) + 1
    refused(lambda: dg.sample(torch.empty(R, 1, dtype=BF, device="cuda"), torch.empty(R, device="cuda")))


def test_matrices_and_experts():
    refused(lambda: dg.w4_quantize(torch.empty(1, (1 << 32) + 64, dtype=BF, device="cuda")))
    for N, K, group in (((1 << 32) + 16, 64, 64), (16, (1 << 32) + 64, 64), (16, 64, (1 << 32) + 64)):
        refused(lambda: dg.W4Matrix(N, K, group))
    w = [t.cuda() for t in drawn(torch.Generator().manual_seed(1), 256, 8, 128)]
    refused(lambda: dg.MoeFfn(*w, top_k=(1 << 32) + 2))
    refused(lambda: dg.MoeFfn(*w, top_k=2).workspace_bytes((1 << 32) + 3))
