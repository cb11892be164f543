"""The mixture-of-experts block for a few tokens against its definition in 64 bits (tolerance in moe_tokens_ref)."""
import math

import pytest
import torch

import moe_tokens_ref
from block_diffusion_text_gb300 import dg, synth

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def drawn(g, d, n, Fe, router=None):
    Wr = (torch.randn(n, d, generator=g) / math.sqrt(d)).to(BF) if router is None else router
    We1 = (torch.randn(n + 1, Fe, d, generator=g) / math.sqrt(d)).to(BF)
    We2 = (torch.randn(n + 1, d, Fe, generator=g) / math.sqrt(Fe)).to(BF)
    return Wr, We1, We2


def ffn_of(w, top_k, eps=1e-6):
    return dg.MoeFfn(*[t.cuda() for t in w], top_k=top_k, rms_eps=eps)


def check(w, h, top_k, ffn=None, eps=1e-6, ws=None):
    M = h.shape[0]
    f = ffn or ffn_of(w, top_k, eps)
    idx = torch.full((M, top_k), -1, dtype=torch.int32, device="cuda")
    gate = torch.zeros(M, top_k, device="cuda")
    got = dg.moe_tokens(f, h.cuda(), routing=(idx, gate), ws=ws)
    # the experts that it took, if they are the largest within the logits' errors
    out, tol, _, wgate, fair = moe_tokens_ref.block(h, *w, top_k, eps, idx=idx.cpu().long())
    assert fair
    assert bool(((gate.double().cpu() - wgate).abs() <= 1e-4).all())
    assert bool((gate[:, 1:] <= gate[:, :-1]).all())
    err = (got.double().cpu() - out).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    return got


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 32])
@pytest.mark.parametrize("d,n,top_k,Fe", [(128, 1, 1, 128), (256, 5, 5, 128), (384, 17, 3, 256), (1024, 64, 8, 128)])
def test_against_64_bits(M, d, n, top_k, Fe):
    g = torch.Generator().manual_seed(M + d + n)
    h = (torch.randn(M, d, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(BF)
    check(drawn(g, d, n, Fe), h, top_k, eps=1e-5)
    assert dg.moe_tokens_status() == 0


@pytest.mark.parametrize("M,d,n,top_k,Fe", [(3, 2816, 128, 8, 768), (20, 2816, 40, 16, 384), (2, 4096, 256, 16, 128),
                                            (1, 128, 2, 1, 2048), (5, 8192, 3, 2, 128)])
def test_model_sizes(M, d, n, top_k, Fe):
    g = torch.Generator().manual_seed(M + d)
    check(drawn(g, d, n, Fe), torch.randn(M, d, generator=g).to(BF), top_k)


@pytest.mark.parametrize("M,d,n,top_k,Fe", [(32, 256, 256, 16, 128), (32, 128, 2, 2, 128), (25, 256, 3, 2, 1024), (32, 2816, 128, 8, 768)])
def test_experts_with_many_tokens_and_many_experts(M, d, n, top_k, Fe):
    """More than eight tokens to an expert, and as many parts as there can be."""
    g = torch.Generator().manual_seed(M + d + n)
    check(drawn(g, d, n, Fe), torch.randn(M, d, generator=g).to(BF), top_k)


def test_all_tokens_on_one_expert_and_ties():
    """A router of zeros but one row: that expert, then the lowest of the equal ones, for every token."""
    g = torch.Generator().manual_seed(3)
    d, n, Fe, M = 256, 40, 128, 32
    h = (1 + 0.2 * torch.randn(M, d, generator=g)).to(BF)     # of positive mean: row 37's logit is the largest
    Wr = torch.zeros(n, d, dtype=BF)
    Wr[37] = 0.1
    w = drawn(g, d, n, Fe, Wr)
    idx, gate = torch.zeros(M, 3, dtype=torch.int32, device="cuda"), torch.zeros(M, 3, device="cuda")
    got = dg.moe_tokens(ffn_of(w, 3), h.cuda(), routing=(idx, gate))
    assert idx.cpu().tolist() == [[37, 0, 1]] * M
    out, tol, widx, _, _ = moe_tokens_ref.block(h, *w, 3)
    assert widx.tolist() == [[37, 0, 1]] * M
    assert bool(((got.double().cpu() - out).abs() <= tol).all())


def test_in_place_and_again_on_the_same_workspace():
    g = torch.Generator().manual_seed(4)
    w = drawn(g, 512, 16, 256)
    f = ffn_of(w, 4)
    h = torch.randn(6, 512, generator=g).to(BF).cuda()
    want = dg.moe_tokens(f, h)
    ws = torch.zeros(f.workspace_bytes(6) + 256, dtype=torch.uint8, device="cuda")
    off = -ws.data_ptr() % 256
    for _ in range(20):
        assert torch.equal(dg.moe_tokens(f, h, ws=ws[off:]), want)
    assert int(ws[off:off + 4].view(torch.int32)) == 0
    x = h.clone()
    assert dg.moe_tokens(f, x, out=x) is x
    assert torch.equal(x, want)


def test_zero_token_and_rows_apart():
    """A row of zeros stays what the experts make of zero; NaN in one row stays in it and is reported."""
    g = torch.Generator().manual_seed(5)
    w = drawn(g, 256, 8, 128)
    f = ffn_of(w, 2)
    h = torch.randn(5, 256, generator=g).to(BF)
    h[2] = 0
    got = dg.moe_tokens(f, h.cuda())
    assert not bool(got[2].any()) and bool(got.isfinite().all())
    ws = torch.zeros(f.workspace_bytes(5), dtype=torch.uint8, device="cuda")
    h[2, 7] = float("nan")
    bad = dg.moe_tokens(f, h.cuda(), ws=ws)
    assert int(ws[:4].view(torch.int32)) == dg.DG_ERR_VALUE
    keep = [0, 1, 3, 4]
    out, tol, *_ = moe_tokens_ref.block(h[keep], *w, 2)
    assert bool(((bad[keep].double().cpu() - out).abs() <= tol).all())


def test_layers_of_a_model():
    dims = synth.Dims(V=64, d=256, C=16, B=1, Hq=2, Hkv=1, hd=64, F=64, P=16, L=2, n_exp=12, top_k=3, Fe=128)
    w = synth.make_weights(dims, 1)
    m = dg.Model(dims, {k: v.cuda() for k, v in w.items()})
    h = torch.randn(4, 256, generator=torch.Generator().manual_seed(6)).to(BF)
    for layer in range(2):
        check([w[k][layer] for k in ("Wr", "We1", "We2")], h, 3, ffn=dg.MoeFfn.of(m, layer))
    # the same layer through the model's own struct
    L, out = dg.load(), torch.empty(4, 256, dtype=BF, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    hc = h.cuda()
    rc = L.dg_moe_tokens(dg.ct.byref(m.s), 1, hc.data_ptr(), out.data_ptr(), 4, None, None, ws.data_ptr(), ws.numel(),
                         torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(out, dg.moe_tokens(dg.MoeFfn.of(m, 1), hc))


def test_streams_and_graphs():
    g = torch.Generator().manual_seed(7)
    w = drawn(g, 512, 16, 256)
    f = ffn_of(w, 4)
    hs = [torch.randn(3, 512, generator=g).to(BF).cuda() for _ in range(3)]
    want = [dg.moe_tokens(f, h) for h in hs]
    torch.cuda.synchronize()
    sts = [torch.cuda.Stream() for _ in range(3)]
    got = [[dg.moe_tokens(f, h, stream=s) for h, s in zip(hs, sts)] for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))
    x = hs[0].clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        a = dg.moe_tokens(f, x)
        b = dg.moe_tokens(f, a)
    for h in hs:
        x.copy_(h)
        gr.replay()
        torch.cuda.synchronize()
        ra = dg.moe_tokens(f, h)
        assert torch.equal(a, ra) and torch.equal(b, dg.moe_tokens(f, ra))
    dg.moe_release_workspaces()
    assert torch.equal(dg.moe_tokens(f, hs[1]), want[1])


def test_binding_refusals():
    w = [t.cuda() for t in drawn(torch.Generator().manual_seed(8), 256, 8, 128)]
    f = dg.MoeFfn(*w, top_k=2)
    h = torch.zeros(3, 256, dtype=BF, device="cuda")
    ok = dict(ffn=f, h=h)
    bad = (torch.zeros(3, 2, device="cuda"), torch.zeros(3, 2, device="cuda"))
    for kw in (dict(h=h.float()), dict(h=h.cpu()), dict(h=h[:, :128]), dict(h=h[0]), dict(out=h[:2]), dict(routing=bad),
               dict(h=h.T.contiguous().T), dict(ws=torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            dg.moe_tokens(**dict(ok, **kw))
    for kw in (dict(h=torch.zeros(33, 256, dtype=BF, device="cuda")), dict(h=h[:0]),
               dict(ws=torch.zeros(512, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(dg.DgError):
            dg.moe_tokens(**dict(ok, **kw))
    with pytest.raises(dg.DgError):
        dg.MoeFfn(*w, top_k=9)
    with pytest.raises(ValueError):
        dg.MoeFfn(w[0], w[1][:8], w[2], top_k=2)
