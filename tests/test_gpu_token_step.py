"""A decoded token's whole step on the public entry points, as they are used together: packed 4-bit projection, norms
and rotation, the 8-bit cache's append and attention, 4-bit output projection with its residual, the experts, the 4-bit
LM head and the sampler, for a ragged batch over several tokens."""
import math

import pytest
import torch

import heads_ref
import kv8_ref
import moe_tokens_ref
import sample_ref
import w4_ref
from block_diffusion_text_gb300 import dg

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Layer:
    """One layer, an embedding and a head, with everything a step keeps between tokens."""

    def __init__(self, B, seed=0, d=256, Hq=4, Hkv=2, hd=64, n=12, top_k=3, Fe=128, V=1003, cap=200):
        g = torch.Generator().manual_seed(seed)
        self.B, self.d, self.Hq, self.Hkv, self.hd, self.top_k, self.V = B, d, Hq, Hkv, hd, top_k, V
        mat = lambda *s: (torch.randn(*s, generator=g) / math.sqrt(s[-1])).to(BF)  # noqa: E731
        self.E = torch.randn(V, d, generator=g).to(BF)
        self.W = dict(qkv=mat((Hq + 2 * Hkv) * hd, d), out=mat(d, Hq * hd), head=self.E)
        self.q = {k: w4_ref.quantize(w, 64) for k, w in self.W.items()}
        self.w4 = {k: dg.w4_quantize(w.cuda(), 64) for k, w in self.W.items()}
        self.gains = [(1 + 0.1 * torch.randn(hd, generator=g)).to(BF) for _ in range(2)]
        self.gcu = [t.cuda() for t in self.gains]
        self.moe = (mat(n, d), mat(n + 1, Fe, d), mat(n + 1, d, Fe))
        self.ffn = dg.MoeFfn(*[t.cuda() for t in self.moe], top_k=top_k)
        self.Ecu = self.E.cuda()
        self.cache = dg.Kv8Cache.empty(B, Hkv, cap, hd)
        self.cache.K_exp.fill_(127)
        self.cache.V_exp.fill_(127)
        self.tok = torch.randint(0, V, (B,), generator=g, dtype=torch.int32).cuda()
        self.u = torch.zeros(B, device="cuda")

    def step(self):
        """One token of every sequence; returns what each operator gave."""
        a = self.Ecu[self.tok.long()]
        r = dict(a=a, pos=self.cache.len.clone())
        r["qkv"] = dg.w4_matvec(self.w4["qkv"], a)
        r["q"], r["k"], r["v"] = dg.qk_norm_rope(r["qkv"].view(self.B, 1, -1), self.cache.len, self.Hq, self.Hkv, *self.gcu)
        r["o"] = dg.kv8_attention(self.cache, r["q"], r["k"], r["v"])
        dg.kv8_append(self.cache, r["k"], r["v"])
        self.cache.len += 1
        r["h"] = dg.w4_matvec(self.w4["out"], r["o"], resid=a)
        r["m"] = dg.moe_tokens(self.ffn, r["h"])
        r["logits"] = dg.w4_matvec(self.w4["head"], r["m"], coef=1 / math.sqrt(self.d), dtype=torch.float32)
        r["tok"], r["lp"], r["kept"] = dg.sample(r["logits"], self.u, temperature=0.8, top_k=50, top_p=0.9, min_p=0.01)
        self.tok.copy_(r["tok"])
        return r


def within(x, want, tol):
    err = (x.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def check_step(L, r, cached):
    c = {k: v.cpu() for k, v in r.items()}
    within(c["qkv"], *w4_ref.product(*L.q["qkv"], c["a"], dtype=BF))
    (q, k, v), (tq, tk) = heads_ref.heads(c["qkv"].view(L.B, 1, -1), c["pos"], L.Hq, L.Hkv, L.gains)
    within(c["q"], q, tq)
    within(c["k"], k, tk)
    assert torch.equal(c["v"].double(), v)
    o, tol = kv8_ref.attention(*cached, c["q"], c["k"], c["v"], False)
    within(c["o"], o, tol)
    within(c["h"], *w4_ref.product(*L.q["out"], c["o"], resid=c["a"], dtype=BF))
    within(c["m"], *moe_tokens_ref.block(c["h"], *L.moe, L.top_k)[:2])
    within(c["logits"], *w4_ref.product(*L.q["head"], c["m"], coef=1 / math.sqrt(L.d)))
    for b in range(L.B):
        f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
        why = sample_ref.check_row(c["logits"][b], float(L.u[b]), f32(0.8), 50, f32(0.9), f32(0.01), int(c["tok"][b]),
                                   float(c["lp"][b]), int(c["kept"][b]))
        assert why is None, why


@pytest.mark.parametrize("B", [1, 5, 32])
def test_each_operator_of_the_step(B):
    L = Layer(B, seed=B)
    g = torch.Generator().manual_seed(B)
    L.cache.len.copy_(torch.randint(0, 3, (B,), generator=g))  # ragged starts over rows of zeros
    for _ in range(4):
        cached = [t.cpu() for t in (L.cache.K, L.cache.V, L.cache.K_exp, L.cache.V_exp, L.cache.len)]
        L.u.copy_(torch.rand(B, generator=g))
        check_step(L, L.step(), cached)
    assert L.cache.status() == 0 and dg.moe_tokens_status() == 0


def test_a_captured_step_follows_the_growing_cache():
    g = torch.Generator().manual_seed(9)
    us = torch.rand(70, 3, generator=g).cuda()
    eager, toks = Layer(3, seed=1), []
    for u in us:
        eager.u.copy_(u)
        toks.append(eager.step()["tok"].clone())
    L = Layer(3, seed=1)
    tok0 = L.tok.clone()
    L.step()                                   # so that nothing is set up for the first time under capture
    L.cache.len.zero_()
    L.tok.copy_(tok0)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = L.step()
    for i, u in enumerate(us):
        L.u.copy_(u)
        gr.replay()
        assert torch.equal(out["tok"], toks[i]), i
    assert L.cache.len.tolist() == [70] * 3
    assert torch.equal(L.cache.K[:, :, :70], eager.cache.K[:, :, :70])
