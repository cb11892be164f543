"""The 8-bit prefix cache in 64 bits, on the CPU, straight from its definition."""
import torch

BLOCK, BIAS, E_MIN, E_MAX = 64, 127, -64, 118


def e4m3_table():
    """The 256 codes' values."""
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def round_e4m3(y):
    """Nearest E4M3 value of y (float64), ties to even, saturating at 448."""
    a = y.abs().clamp(max=448.0)
    power = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(power - 3)
    r = torch.round(a / step) * step
    return torch.where(torch.signbit(y), -r, r)


def exponent(top):
    """Smallest e in range with top <= 448 2^e."""
    e = E_MIN
    while e < E_MAX and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(codes, exps, x, lens, counts):
    """codes [B,H,cap,hd] uint8, exps [B,H,nblk] uint8, x [B,H,n,hd] bf16, all on the CPU: new codes and exponents."""
    codes, exps, table = codes.clone(), exps.clone(), e4m3_table()
    B, H, cap, hd = codes.shape
    for b in range(B):
        start, n = int(lens[b]), int(counts[b])
        if start < 0 or n < 0 or start + n > cap:
            continue
        for h in range(H):
            at = start
            while at < start + n:
                blk = at // BLOCK
                end = min(start + n, (blk + 1) * BLOCK)
                new = x[b, h, at - start:end - start].double()
                new = torch.where(torch.isnan(new), 0.0, new)
                fin = new[torch.isfinite(new)]
                e = exponent(float(fin.abs().max()) if fin.numel() else 0.0)
                base = blk * BLOCK
                if at > base:
                    was = int(exps[b, h, blk]) - BIAS
                    if e > was:
                        old = table[codes[b, h, base:at].long()]
                        codes[b, h, base:at] = to_codes(round_e4m3(old * 2.0 ** (was - e)))
                    else:
                        e = was
                codes[b, h, at:end] = to_codes(round_e4m3(new * 2.0 ** -e))
                exps[b, h, blk] = e + BIAS
                at = end
    return codes, exps


def to_codes(v):
    """Codes of values that E4M3 holds exactly."""
    return v.float().to(torch.float8_e4m3fn).view(torch.uint8)


def values(codes, exps):
    """[..., rows, hd] codes with exps [..., nblk] to float64."""
    scale = torch.exp2(exps.double() - BIAS).repeat_interleave(BLOCK, -1)[..., :codes.shape[-2]]
    return e4m3_table()[codes.long()] * scale[..., None]


def attention(K, V, Ke, Ve, lens, q, k, v, causal):
    """(o [B*C, Hq*hd] float64, tol): the output and how far a correct kernel may be from it.

    tol, element by element, with A = sum_i p_i |v_i| and N keys: the bf16 rounding of the output 2^-8 |o|; f16
    rounding of the probabilities 2^-11 A (the bf16 pair of the new tokens' is finer) and their floor, half a
    subnormal 2^-25 under a row maximum of 2^8, for N codes of at most 448 2^e; the base-2 exponential 2^-21 A; fp32
    accumulation of N products, and of their sum, 2 N 2^-24 A; fp32 accumulation of a score's hd products,
    hd 2^-23 of their absolute sum, which moves each probability and the sum by that much."""
    B, Hq, C, hd = q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    o = torch.zeros(B, C, Hq, hd, dtype=torch.float64)
    tol = torch.full_like(o, 1e-30)
    for b in range(B):
        n = int(lens[b])
        for g in range(Hkv):
            kk, vv = values(K[b, g, :n], Ke[b, g]), values(V[b, g, :n], Ve[b, g])
            if k is not None:
                kk, vv = torch.cat([kk, k[b, g].double()]), torch.cat([vv, v[b, g].double()])
            N = kk.shape[0]
            if N == 0:
                continue
            mask = torch.zeros(C, N, dtype=torch.bool)
            if k is not None and causal:
                mask[:, n:] = torch.ones(C, C, dtype=torch.bool).triu(1)
            floor = N * 2.0 ** -33 * float(vv.abs().max()) * 4
            for h in range(g * G, (g + 1) * G):
                qq = q[b, h].double()
                s = (qq @ kk.T) / hd ** 0.5
                s = s.masked_fill(mask, float("-inf"))
                p = torch.softmax(s, -1)
                ds = hd * 2.0 ** -23 * ((qq.abs() @ kk.abs().T) / hd ** 0.5).amax(-1, keepdim=True)
                A = p @ vv.abs()
                o[b, :, h] = p @ vv
                tol[b, :, h] = 2.0 ** -8 * o[b, :, h].abs() + A * (2.0 ** -11 + 2.0 ** -21 + 2 * N * 2.0 ** -24 + 2 * ds) \
                    + floor + 1e-30
    return o.reshape(B * C, Hq * hd), tol.reshape(B * C, Hq * hd)
