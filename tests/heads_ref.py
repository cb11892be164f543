"""Norms of the heads with the rotation, restated in 64 bits."""
import torch

U = 2.0 ** -24


def heads(qkv, pos, Hq, Hkv, gains=(None, None), eps=1e-6, base=10000.0):
    """((q, k, v), (tolerance of q, of k)) in 64 bits.

    fp32 steps of a value: the sum of hd squares (hd / 2 additions in a row at most, hd 2^-24 has room), the mean,
    eps, root, quotient (5), products with 1 / rms and gain (2), the turn (3 more, and sine and cosine: off by 2^-23
    themselves, and by the angle's 2^-25 of half a turn, 2^-23 at most): all relative to |a| + |b| of the pair.  Then
    half a step of bf16."""
    B, C, W = qkv.shape
    hd = W // (Hq + 2 * Hkv)
    x = qkv.double().reshape(B, C, Hq + 2 * Hkv, hd).transpose(1, 2)
    at = pos.double()[:, None] + torch.arange(C, dtype=torch.float64)
    j = torch.arange(hd // 2, dtype=torch.float64)
    ang = at[..., None] * torch.tensor(base, dtype=torch.float32).double() ** (-2 * j / hd)
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]
    eps = float(torch.tensor(eps, dtype=torch.float32))
    out, tols = [], []
    for t, gain in ((x[:, :Hq], gains[0]), (x[:, Hq:Hq + Hkv], gains[1])):
        t = t / (t.square().mean(-1, keepdim=True) + eps).sqrt()
        if gain is not None:
            t = t * gain.double()
        a, b = t[..., :hd // 2], t[..., hd // 2:]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        size = (a.abs() + b.abs()).repeat(1, 1, 1, 2)
        out.append(r)
        # a double's own rounding of the angle, here and in the table of turns: 2^-52 of it
        far = at.abs().max() * 2.0 ** -51
        tols.append(size * ((hd + 5 + 2 + 3 + 4) * U + far) + r.abs() * 2.0 ** -8)
    out.append(x[:, Hq + Hkv:])
    return out, tols
