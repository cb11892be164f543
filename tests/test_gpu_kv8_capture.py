"""Captured attention calls that bring neither an output nor a workspace: both come from the graph's pool, and must
not be the same memory."""
import pytest
import torch

from block_diffusion_text_gb300 import dg
from test_gpu_kv8 import filled, rows

pytestmark = pytest.mark.gpu

CASES = [
    # B, C, Hq, Hkv, hd, lens, cap, causal: outputs above 1 MiB (the allocator's large blocks, as the workspace) ..
    (8, 250, 8, 2, 128, [5000, 1, 333, 4097, 64, 0, 2000, 2500], 5120, True),
    (2, 256, 16, 8, 128, [4000, 777], 4096, False),
    (4, 128, 16, 2, 64, [8000, 64, 1, 4000], 8000, True),
    # .. and both below it
    (1, 1, 2, 1, 32, [69999], 70000, True),
    (3, 1, 2, 2, 64, [40000, 0, 65], 70000, True),
]


@pytest.mark.parametrize("case", CASES, ids=[f"b{c[0]}c{c[1]}q{c[2]}h{c[4]}" for c in CASES])
def test_captured_output_lies_beside_the_workspace(case):
    B, C, Hq, Hkv, hd, lens, cap, causal = case
    g = torch.Generator().manual_seed(cap + C)
    c = filled(g, B, Hkv, cap, hd, lens)
    assert c.workspace_bytes(C, Hq) > 0
    x = [rows(g, B, h, C, hd).cuda() for h in (Hq, Hkv, Hkv)]
    want = dg.kv8_attention(c, *x, causal=causal)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        o = dg.kv8_attention(c, *x, causal=causal)
        # a second call in the same graph, whose buffers come from the same pool
        o2 = dg.kv8_attention(c, *x, causal=causal)
    for _ in range(5):
        o.zero_()
        o2.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(o2, want)
