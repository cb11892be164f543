"""Attention over the 8-bit cache at scores far beyond what an exponential spans: up to 2^23 in magnitude all weight is
on the row's largest and the output is that key's value; beyond, the status word says that the call does not take them."""
import pytest
import torch

import kv8_ref
from block_diffusion_text_gb300 import dg
from test_gpu_kv8 import filled, rows, state

pytestmark = pytest.mark.gpu

SIZES = [(1, 128, 400), (3, 32, 400), (2, 64, 5000), (16, 128, 400), (40, 128, 20000), (256, 128, 3000), (256, 64, 5000),
         (130, 128, 3000)]


@pytest.mark.parametrize("power", [10, 18, 21, 22, 26, 30, 40, 60, 100])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("C,hd,cap", SIZES, ids=[f"c{c}h{h}cap{n}" for c, h, n in SIZES])
def test_weight_is_on_the_largest_score(C, hd, cap, power, sign):
    """Scores up to 2^(power + 1) in magnitude, of either sign; neighbours in order of size are 2^-6 of the largest
    apart.  The largest is a cached key's in some rows and a new token's in others."""
    g = torch.Generator().manual_seed(90)
    B, Hq, Hkv, n = 2, 4, 2, 390
    c = filled(g, B, Hkv, cap, hd, [n, 65])
    q, k, v = rows(g, B, Hq, C, hd), rows(g, B, Hkv, C, hd), rows(g, B, Hkv, C, hd)
    # channel 0 carries the score: cached keys 1 to 1.75 (four codes, on scale 1) but for one of 2 (or 0.5), new ones
    # 1.875 but for one of 4 (or 0.25); channel 1 of a query turns the new ones off
    c.K_exp[:] = 127
    codes = torch.tensor([0x38, 0x3a, 0x3c, 0x3e], dtype=torch.uint8)  # 1, 1.25, 1.5, 1.75
    K = torch.zeros(B, Hkv, cap, hd, dtype=torch.uint8)
    K[..., 0] = codes[torch.randint(0, 4, (B, Hkv, cap), generator=g)]
    win = torch.randint(0, 65, (B, Hkv), generator=g)
    for b in range(B):
        for h in range(Hkv):
            K[b, h, win[b, h], 0] = 0x40 if sign > 0 else 0x30  # 2, or 0.5
    c.K.copy_(K)
    k[:] = 0
    k[..., 0] = 1.875
    wnew = C // 2
    k[:, :, wnew, 0] = 4 if sign > 0 else 0.25
    k[..., 1] = -4.0                                           # in rows with q[1] = |q[0]| no new token wins
    q[:] = 0
    f = sign * 2.0 ** (power - 2) * hd ** 0.5
    q[..., 0] = f
    off = torch.arange(C) % 2 == 0
    q[:, :, off, 1] = abs(f)
    got = dg.kv8_attention(c, q.cuda(), k.cuda(), v.cuda()).cpu().double().view(B, C, Hq, hd)
    if power > 23:
        assert c.status() == dg.DG_ERR_VALUE
        return
    assert c.status() == 0
    val = kv8_ref.values(c.V.cpu(), c.V_exp.cpu())
    for b in range(B):
        for h in range(Hq):
            cached, new = val[b, h // 2, win[b, h // 2]], v[b, h // 2, wnew].double()
            want = torch.where(off[:, None], cached, new)
            # the weight's f16 rounding, the output's to bf16, and other keys' below 2^-20 of it
            tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20) * want.abs() + 2.0 ** -20 * max(float(val[b, h // 2, :65].abs().max()), float(v.abs().max().double()))
            assert ((got[b, :, h] - want).abs() <= tol).all()
