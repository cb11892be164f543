"""Norms of the heads with the rotation against their definition in 64 bits (tolerance derived in heads_ref)."""
import pytest
import torch

import heads_ref
from block_diffusion_text_gb300 import dg

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def check(qkv, pos, Hq, Hkv, gains=(None, None), cuda=None, **kw):
    g = [None if t is None else t.cuda() for t in gains]
    got = dg.qk_norm_rope(qkv.cuda() if cuda is None else cuda, pos.cuda(), Hq, Hkv, g[0], g[1], **kw)
    rkw = dict(eps=kw.get("rms_eps", 1e-6), base=kw.get("rope_base", 10000.0))
    (q, k, v), (tq, tk) = heads_ref.heads(qkv, pos, Hq, Hkv, gains, **rkw)
    for x, want, tol in ((got[0], q, tq), (got[1], k, tk)):
        err = (x.double().cpu() - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
    assert torch.equal(got[2].double().cpu(), v)
    return got


def packed(g, B, C, Hq, Hkv, hd):
    x = torch.randn(B, C, Hq + 2 * Hkv, hd, generator=g) * torch.exp(torch.randn(B, C, Hq + 2 * Hkv, 1, generator=g))
    return x.reshape(B, C, -1).to(BF)


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("B,C,Hq,Hkv", [(1, 1, 1, 1), (1, 1, 8, 2), (3, 5, 2, 1), (2, 33, 16, 8), (5, 1, 7, 7), (1, 700, 4, 4),
                                        (2, 2, 40, 8)])
def test_against_64_bits(hd, B, C, Hq, Hkv):
    g = torch.Generator().manual_seed(hd + B * C + Hq)
    pos = torch.randint(0, 5000, (B,), generator=g, dtype=torch.int32)
    gains = [(1 + 0.3 * torch.randn(hd, generator=g)).to(BF) for _ in range(2)]
    x = packed(g, B, C, Hq, Hkv, hd)
    check(x, pos, Hq, Hkv, gains)
    check(x, pos, Hq, Hkv, (gains[0], None), rope_base=500.0, rms_eps=1e-3)


def test_far_positions_keep_their_angle():
    g = torch.Generator().manual_seed(1)
    pos = torch.tensor([0, 131072, 1 << 20, (1 << 31) - 3, -5, 1 << 30], dtype=torch.int32)
    check(packed(g, 6, 2, 2, 1, 128), pos, 2, 1)
    check(packed(g, 6, 2, 2, 1, 64), pos, 2, 1, rope_base=1e6)
    check(packed(g, 6, 2, 2, 1, 32), pos, 2, 1, rope_base=1.0)


def test_strides_zero_heads_and_neighbours():
    """Tokens inside wider rows of a larger batch, NaN between them; heads of zeros stay zero; a NaN head is alone."""
    g = torch.Generator().manual_seed(2)
    B, C, Hq, Hkv, hd = 3, 7, 3, 1, 64
    W = (Hq + 2 * Hkv) * hd
    x = packed(g, B, C, Hq, Hkv, hd)
    x.view(B, C, -1, hd)[1, 2, 1] = 0
    wide = torch.full((B, C + 2, W + 24), float("nan"), dtype=BF, device="cuda")
    wide[:, 1:1 + C, 16:16 + W] = x.cuda()
    pos = torch.tensor([5, 0, 900], dtype=torch.int32)
    q, k, v = check(x, pos, Hq, Hkv, cuda=wide[:, 1:1 + C, 16:16 + W])
    assert not bool(q[1, 1, 2].any())
    y = x.clone()
    y.view(B, C, -1, hd)[0, 3, 1, 5] = float("nan")
    q2, k2, v2 = dg.qk_norm_rope(y.cuda(), pos.cuda(), Hq, Hkv)
    assert not bool(q2[0, 1, 3].isfinite().any())
    q2[0, 1, 3] = q[0, 1, 3]
    assert torch.equal(q2, q) and torch.equal(k2, k) and torch.equal(v2, v)


@pytest.mark.parametrize("B,C,Hq,Hkv,hd", [(3, 1701, 26, 3, 128), (1, 9733, 20, 2, 64), (5, 4001, 14, 1, 32)])
def test_several_tokens_to_a_block(B, C, Hq, Hkv, hd):
    g = torch.Generator().manual_seed(B + C)
    pos = torch.randint(0, 100000, (B,), generator=g, dtype=torch.int32)
    gains = [(1 + 0.3 * torch.randn(hd, generator=g)).to(BF) for _ in range(2)]
    check(packed(g, B, C, Hq, Hkv, hd), pos, Hq, Hkv, gains)


def test_sequences_past_32_bits_apart():
    g = torch.Generator().manual_seed(9)
    B, C, Hq, Hkv, hd = 2, 3, 2, 1, 64
    x, W, sb = packed(g, B, C, Hq, Hkv, hd), (Hq + 2 * Hkv) * hd, 2 ** 31 + 8
    wide = torch.empty(sb + C * W, dtype=BF, device="cuda").as_strided((B, C, W), (sb, W, 1))
    wide.copy_(x)
    check(x, torch.tensor([7, 4000], dtype=torch.int32), Hq, Hkv, cuda=wide)


def test_out_stream_and_graph_follow_the_positions():
    g = torch.Generator().manual_seed(3)
    x = packed(g, 2, 3, 4, 2, 128)
    pos = torch.tensor([7, 70], dtype=torch.int32)
    want = check(x, pos, 4, 2)
    xc, pc = x.cuda(), pos.cuda()
    out = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    assert dg.qk_norm_rope(xc, pc, 4, 2, out=out, stream=st)[0] is out[0]
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = dg.qk_norm_rope(xc, pc, 4, 2)
    pc += 1
    gr.replay()
    torch.cuda.synchronize()
    ref = dg.qk_norm_rope(xc, pc, 4, 2)
    assert all(torch.equal(a, b) for a, b in zip(got, ref)) and not torch.equal(got[0], want[0])


def test_binding_refusals():
    x, p = torch.zeros(2, 3, 4 * 64, dtype=BF, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    gain = torch.ones(64, dtype=BF, device="cuda")
    ok = dict(qkv=x, pos=p, Hq=2, Hkv=1)
    for kw in (dict(qkv=x.float()), dict(qkv=x[0]), dict(Hkv=4), dict(Hq=0), dict(pos=p.long()), dict(pos=p[:1]), dict(pos=p.cpu()),
               dict(q_gain=gain[:32]), dict(k_gain=gain.float()), dict(qkv=x.transpose(1, 2)),
               dict(out=(x, x, x))):
        with pytest.raises(ValueError):
            dg.qk_norm_rope(**dict(ok, **kw))
    with pytest.raises(dg.DgError):   # a head dim that is not supported
        dg.qk_norm_rope(x, p, 14, 1)
    q, k, v = dg.qk_norm_rope(x[:, :0], p, 2, 1)
    assert q.shape == (2, 2, 0, 64) and k.shape == v.shape == (2, 1, 0, 64)
