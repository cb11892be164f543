"""What the expert block's workspace says, and what comes after it has said so."""
import pytest
import torch

import moe_tokens_ref
from test_gpu_moe_tokens import BF, check, drawn, ffn_of
from block_diffusion_text_gb300 import dg

pytestmark = pytest.mark.gpu

ARRIVALS = 256  # byte of the workspace at which the grid's barrier counts


def spoil(ws):
    """A count that the arrivals never bring to the last of a round: the wait runs out (two seconds each barrier)."""
    ws[ARRIVALS:ARRIVALS + 4] = torch.tensor([255, 255, 255, 127], dtype=torch.uint8, device="cuda")


def test_a_wait_that_runs_out_is_told():
    g = torch.Generator().manual_seed(1)
    f = ffn_of(drawn(g, 256, 8, 128), 2)
    h = torch.randn(3, 256, generator=g).to(BF).cuda()
    want = dg.moe_tokens(f, h)
    ws = torch.zeros(f.workspace_bytes(3), dtype=torch.uint8, device="cuda")
    spoil(ws)
    dg.moe_tokens(f, h, ws=ws)
    assert int(ws[:4].view(torch.int32)) == dg.DG_ERR_TIMEOUT
    ws.zero_()
    assert torch.equal(dg.moe_tokens(f, h, ws=ws), want) and int(ws[:4].view(torch.int32)) == dg.DG_OK


def test_the_kept_workspace_is_let_go_of_after_a_timeout():
    g = torch.Generator().manual_seed(2)
    f = ffn_of(drawn(g, 256, 8, 128), 2)
    h = torch.randn(3, 256, generator=g).to(BF).cuda()
    dg.moe_release_workspaces()
    want = dg.moe_tokens(f, h)
    (kept,) = dg._moe_workspaces.values()
    spoil(kept)
    dg.moe_tokens(f, h)
    assert dg.moe_tokens_status() == dg.DG_ERR_TIMEOUT
    for _ in range(3):
        assert torch.equal(dg.moe_tokens(f, h), want)
    assert dg.moe_tokens_status() == dg.DG_OK


def test_the_barrier_goes_on_from_any_round():
    g = torch.Generator().manual_seed(3)
    f = ffn_of(drawn(g, 256, 8, 128), 2)
    h = torch.randn(5, 256, generator=g).to(BF).cuda()
    want = dg.moe_tokens(f, h)
    ws = torch.zeros(f.workspace_bytes(5), dtype=torch.uint8, device="cuda")
    ws[512:516] = 255  # the rounds' count is about to wrap
    for _ in range(3):
        assert torch.equal(dg.moe_tokens(f, h, ws=ws), want)
    assert int(ws[:4].view(torch.int32)) == dg.DG_OK


def test_what_a_call_met_outlives_a_larger_workspace():
    g = torch.Generator().manual_seed(4)
    f = ffn_of(drawn(g, 256, 8, 128), 2)
    h = torch.randn(32, 256, generator=g).to(BF).cuda()
    dg.moe_release_workspaces()
    want = dg.moe_tokens(f, h)
    dg.moe_release_workspaces()
    assert dg.moe_tokens_status() == dg.DG_OK
    dg.moe_tokens(f, h[:1] * float("nan"))
    assert torch.equal(dg.moe_tokens(f, h), want)
    assert dg.moe_tokens_status() == dg.DG_ERR_VALUE
    dg.moe_release_workspaces()
    assert torch.equal(dg.moe_tokens(f, h), want) and dg.moe_tokens_status() == dg.DG_OK


@pytest.mark.parametrize("d", [256, 16384])
@pytest.mark.parametrize("M", [2, 20])
def test_rows_whose_squares_leave_fp32_are_told(M, d):
    """2^56 is within the range at the widest row (2^14 squares of 2^112 at most); 2^70 is not."""
    g = torch.Generator().manual_seed(5)
    w = drawn(g, d, 8, 128)
    f = ffn_of(w, 2)
    h = torch.randn(M, d, generator=g).clamp(-1, 1).to(BF)
    h[1] *= 2.0 ** 56
    ws = torch.zeros(f.workspace_bytes(M), dtype=torch.uint8, device="cuda")
    check(w, h, 2, ffn=f, ws=ws)
    assert int(ws[:4].view(torch.int32)) == dg.DG_OK
    h[1] *= 2.0 ** 14
    got = dg.moe_tokens(f, h.cuda(), ws=ws)
    assert int(ws[:4].view(torch.int32)) == dg.DG_ERR_VALUE
    out, tol, *_ = moe_tokens_ref.block(h[:1], *w, 2)
    assert bool(((got[:1].double().cpu() - out).abs() <= tol).all())
