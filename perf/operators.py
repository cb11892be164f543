"""The operators of the 8-bit prefix cache: what is measured, in a plain form.

Three operators work on one cache of E4M3 codes with a power-of-two scale for
each block of 64 tokens and head:

* append     quantises new key and value rows into the cache as they are written
* read       reads a range of rows back as bf16
* attention  attends over the cached rows and, in bf16, the new tokens' own keys
             and values: a canvas of queries without a mask, a causal prompt
             piece, or a single token per sequence

Each sequence of a batch has its own length, held on the device.
"""
import random

import numpy as np
import torch

own = False

BLOCK = 64      # cached tokens per scale
BIAS = 127      # exponent byte x stands for the scale 2^(x - 127)
E_MIN, E_MAX = -64, 118
LOG2E = 1.4426950408889634


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one decoded token for each of 32 sequences, anywhere inside a block: what every token step pays
        dict(name="append_token_b32", op="append", B=32, Hkv=8, hd=128, n=1, lo=1, hi=4000, ragged=False),
        # the commit of finished 256-token blocks of 8 canvases, some of them shorter (padded rows stay out)
        dict(name="append_block_b8", op="append", B=8, Hkv=2, hd=128, n=256, lo=4096, hi=4864, ragged=True),
        # four long prompts written behind short odd heads
        dict(name="append_prompt_16k", op="append", B=4, Hkv=8, hd=128, n=16384, lo=0, hi=63, ragged=False),
        # a window read back for a second pass over it, from an odd row, some sequences ending inside it
        dict(name="read_window_hd64", op="read", B=8, Hkv=2, hd=64, n=1000, row0=37, lo=600, hi=2048),
        # the export of a whole long prefix to a bf16 cache
        dict(name="read_prefix_131k", op="read", B=1, Hkv=8, hd=128, n=131072, row0=0, lo=131072, hi=131072),
        # the tiny workload's canvas: the smallest call, all latency
        dict(name="canvas_tiny_hd32", op="attention", B=1, C=16, Hq=2, Hkv=1, hd=32, lo=32, hi=32, causal=False, tail=True),
        # one token of one sequence over a 2048-token prefix: latency again
        dict(name="token_b1_p2k", op="attention", B=1, C=1, Hq=8, Hkv=2, hd=128, lo=2048, hi=2048, causal=False, tail=True),
        # a batch of 32 sequences of all lengths, one token each
        dict(name="token_b32_ragged", op="attention", B=32, C=1, Hq=16, Hkv=8, hd=128, lo=0, hi=8192, causal=False, tail=True),
        # four very long sequences, one token each, already in the cache
        dict(name="token_b4_131k", op="attention", B=4, C=1, Hq=8, Hkv=8, hd=128, lo=131001, hi=131072, causal=False, tail=False),
        # the canvas of the annealed loop over its 8192-token prefix
        dict(name="canvas_p8k", op="attention", B=1, C=256, Hq=16, Hkv=8, hd=128, lo=8192, hi=8192, causal=False, tail=True),
        # the attention-heavy canvas over a 131072-token prefix
        dict(name="canvas_p131k", op="attention", B=1, C=256, Hq=8, Hkv=8, hd=128, lo=131072, hi=131072, causal=False, tail=True),
        # a causal prompt piece of 250 tokens for 8 sequences of odd lengths
        dict(name="piece_causal_b8", op="attention", B=8, C=250, Hq=8, Hkv=2, hd=128, lo=1, hi=5120, causal=True, tail=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    hd = rng.choice([32, 64, 128, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    op = rng.choice(["append", "read", "token", "token", "canvas", "canvas"])
    if op == "append":
        n = _log(rng, 1, 16384)
        B = _log(rng, 1, max(1, min(48, 65536 // n)))
        lo = rng.randrange(0, 200)
        return dict(op=op, B=B, Hkv=Hkv, hd=hd, n=n, lo=lo, hi=lo + _log(rng, 1, 4000), ragged=rng.random() < 0.5)
    if op == "read":
        n = _log(rng, 1, 131072)
        B = _log(rng, 1, max(1, min(32, 131072 // n)))
        row0 = rng.randrange(0, 300)
        hi = row0 + n + rng.randrange(0, 100)
        return dict(op=op, B=B, Hkv=Hkv, hd=hd, n=n, row0=row0, lo=max(0, hi - _log(rng, 1, 2000)), hi=hi)
    G = rng.choice([1, 2, 4, 8])
    if op == "token":
        hi = _log(rng, 16, 131072)
        B = _log(rng, 1, max(1, min(64, 524288 // hi)))
        return dict(op="attention", B=B, C=rng.choice([1, 1, 2, 3]), Hq=G * Hkv, Hkv=Hkv, hd=hd, lo=rng.randrange(0, hi + 1), hi=hi,
                    causal=rng.random() < 0.5, tail=rng.random() < 0.7)
    hd = rng.choice([64, 128, 128, 128])
    hi = _log(rng, 16, 65536)
    C = _log(rng, 4, 1024)
    B = _log(rng, 1, max(1, min(8, (1 << 27) // (C * G * Hkv * hi))))
    return dict(op="attention", B=B, C=C, Hq=G * Hkv, Hkv=Hkv, hd=hd, lo=rng.randrange(0, hi + 1), hi=hi, causal=rng.random() < 0.4, tail=True)


def _lengths(case):
    """The sequences' lengths: the first is the longest, the second the shortest, the others between."""
    r = random.Random("%d %d %d" % (case["B"], case["lo"], case["hi"]))
    more = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    return ([case["hi"], case["lo"]] + more)[:case["B"]]


def _counts(case):
    """New rows of each sequence: all n, or (ragged) any number up to n."""
    if not case["ragged"]:
        return [case["n"]] * case["B"]
    r = random.Random("%d %d rows" % (case["B"], case["n"]))
    return [case["n"] if b % 3 == 0 else r.randint(0, case["n"]) for b in range(case["B"])]


def _capacity(case):
    # room for the longest sequence, its new rows and the block they end in
    return max(_lengths(case)) + case.get("n", 0) * (case["op"] == "append") + 130


# ----------------------------------------------------------------- inputs ----
def _cache(case, g):
    """Codes and exponents as a cache of values of about unit size has them: a
    block's largest value lies in the top octave of E4M3; blocks differ by a
    few octaves; rows behind a sequence's end hold whatever was there before."""
    B, H, hd, cap = case["B"], case["Hkv"], case["hd"], _capacity(case)
    nb = -(-cap // BLOCK)
    codes, exps = [], []
    for _ in range(2):
        x = torch.randn(B, H, cap, hd, generator=g, device="cuda") * 100
        codes.append(x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        exps.append((BIAS - 7 + torch.randint(-1, 2, (B, H, nb), generator=g, device="cuda")).to(torch.uint8))
    return codes + exps


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    K, V, Ke, Ve = _cache(case, g)
    B, H, hd = case["B"], case["Hkv"], case["hd"]
    s = dict(case=case, K=K, V=V, Ke=Ke, Ve=Ve, len=torch.tensor(_lengths(case), dtype=torch.int32, device="cuda"))

    def rows(heads, n):
        # unit values with stronger and weaker channels
        x = torch.randn(B, heads, n, hd, generator=g, device="cuda")
        return (x * torch.exp(0.5 * torch.randn(heads, 1, hd, generator=g, device="cuda"))).to(torch.bfloat16)

    if case["op"] == "append":
        s["k"], s["v"] = rows(H, case["n"]), rows(H, case["n"])
        s["count"] = torch.tensor(_counts(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
    elif case["op"] == "read":
        s["k"] = torch.zeros(B, H, case["n"], hd, dtype=torch.bfloat16, device="cuda")
        s["v"] = torch.zeros_like(s["k"])
    else:
        s["q"] = rows(case["Hq"], case["C"])
        s["k"], s["v"] = (rows(H, case["C"]), rows(H, case["C"])) if case["tail"] else (None, None)
    if own:
        from block_diffusion_text_gb300 import dg
        s["cache"] = dg.Kv8Cache(K, V, Ke, Ve, s["len"])
    return s


# ------------------------------------------------------------- plain form ----
def _pow2(e):
    """2^e in float32, exactly, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_append(codes, exps, x, length, count):
    """The window of whole blocks that the new rows touch, rewritten: its old
    rows on the (grown) scale of their block, the new ones behind them."""
    B, H, n, hd = x.shape
    start = length.long() // BLOCK * BLOCK
    nb = -(-n // BLOCK) + 1
    row = start[:, None] + torch.arange(nb * BLOCK, device=x.device)          # [B, w]
    first = length.long()[:, None]
    isnew = (row >= first) & (row < first + count.long()[:, None])
    isold = row < first
    b = torch.arange(B, device=x.device)[:, None]
    blk = start[:, None] // BLOCK + torch.arange(nb, device=x.device)         # [B, nb]
    old = codes[b, :, row].permute(0, 2, 1, 3)                                # [B, H, w, hd]
    e_old = exps[b, :, blk].permute(0, 2, 1).to(torch.int32) - BIAS           # [B, H, nb]
    new = x[b, :, (row - first).clamp(0, n - 1)].permute(0, 2, 1, 3).float()
    new = torch.where(isnew[:, None, :, None], new, 0.0)
    top = new.abs().reshape(B, H, nb, BLOCK * hd).amax(-1)
    frac, power = torch.frexp(top)
    need = torch.where(frac <= 0.875, power - 9, power - 8)                   # smallest e with top <= 448 2^e
    need = torch.where(top > 0, need, E_MIN).clamp(E_MIN, E_MAX)
    touched = isnew.reshape(B, nb, BLOCK).any(-1)[:, None]
    holds = isold.reshape(B, nb, BLOCK).any(-1)[:, None]
    e = torch.where(touched, torch.where(holds, torch.maximum(e_old, need), need), e_old)
    per_row = lambda t: t.repeat_interleave(BLOCK, -1)[..., None]  # noqa: E731
    moved = old.view(torch.float8_e4m3fn).float() * _pow2(per_row((e_old - e).clamp(min=-126)))
    fresh = (new * _pow2(per_row(-e))).clamp(-448, 448)
    out = torch.where(isnew[:, None, :, None], fresh, moved).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = (isold & touched[:, 0].repeat_interleave(BLOCK, -1)) | isnew
    codes[b, :, row] = torch.where(keep[:, None, :, None], out, old).permute(0, 2, 1, 3)
    exps[b, :, blk] = (e + BIAS).to(torch.uint8).permute(0, 2, 1)


def _values(codes, exps):
    """The cached values in 32 bits."""
    scale = _pow2(exps.to(torch.int32) - BIAS).repeat_interleave(BLOCK, -1)[..., :codes.shape[2], None]
    return codes.view(torch.float8_e4m3fn).float() * scale


def _plain_read(codes, exps, row0, n, length, out):
    first, last = row0 // BLOCK, -(-(row0 + n) // BLOCK)
    x = _values(codes[:, :, first * BLOCK:last * BLOCK], exps[:, :, first:last])[:, :, row0 - first * BLOCK:][:, :, :n]
    there = (row0 + torch.arange(n, device=x.device)) < length[:, None]
    out.copy_(torch.where(there[:, None, :, None], x, out.float()))


def _plain_attention(s):
    case, q = s["case"], s["q"]
    B, H, C, hd, G = case["B"], case["Hkv"], case["C"], case["hd"], case["Hq"] // case["Hkv"]
    top = max(1, case["hi"])
    K, V = _values(s["K"][:, :, :top], s["Ke"]), _values(s["V"][:, :, :top], s["Ve"])
    seen = (torch.arange(top, device=q.device) < s["len"][:, None])[:, None, :].expand(B, C, top)
    if s["k"] is not None:
        i = torch.arange(C, device=q.device)
        new = (i[None, :] <= i[:, None]) if case["causal"] else torch.ones(C, C, dtype=torch.bool, device=q.device)
        K, V = torch.cat([K, s["k"].float()], 2), torch.cat([V, s["v"].float()], 2)
        seen = torch.cat([seen, new.expand(B, C, C)], 2)
    x = (q.float().reshape(B, H, G * C, hd) @ K.transpose(-1, -2)).mul_(hd ** -0.5).reshape(B, H, G, C, -1)
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.reshape(B, H, G * C, -1) @ V).reshape(B, H * G, C, hd) / total.reshape(B, H * G, C, 1).clamp(min=1e-30)
    return o.transpose(1, 2).reshape(B * C, H * G * hd).to(torch.bfloat16)


def run(s):
    case, c = s["case"], s.get("cache")
    if case["op"] == "append":
        if own:
            from block_diffusion_text_gb300 import dg
            dg.kv8_append(c, s["k"], s["v"], counts=s["count"])
        else:
            count = s["count"] if s["count"] is not None else torch.full_like(s["len"], case["n"])
            _plain_append(s["K"], s["Ke"], s["k"], s["len"], count)
            _plain_append(s["V"], s["Ve"], s["v"], s["len"], count)
        # the codes as the E4M3 values they stand for, and the exponents of the blocks' scales
        return dict(K=s["K"].view(torch.float8_e4m3fn), V=s["V"].view(torch.float8_e4m3fn), Ke=s["Ke"], Ve=s["Ve"])
    if case["op"] == "read":
        if own:
            from block_diffusion_text_gb300 import dg
            dg.kv8_read(c, case["row0"], case["n"], out=(s["k"], s["v"]))
        else:
            _plain_read(s["K"], s["Ke"], case["row0"], case["n"], s["len"], s["k"])
            _plain_read(s["V"], s["Ve"], case["row0"], case["n"], s["len"], s["v"])
        return dict(k=s["k"], v=s["v"])
    if own:
        from block_diffusion_text_gb300 import dg
        return dict(o=dg.kv8_attention(c, s["q"], s["k"], s["v"], causal=case["causal"]))
    return dict(o=_plain_attention(s))


# ------------------------------------------------------------------- work ----
def work(case):
    """Bytes: every input read once, every output written once.  Operations:
    the two products of attention, over the keys that the mask leaves."""
    B, H, hd = case["B"], case["Hkv"], case["hd"]
    lens = _lengths(case)
    blocks = lambda rows: sum(-(-r // BLOCK) for r in rows)  # noqa: E731
    if case["op"] == "append":
        rows = _counts(case)
        return dict(bytes=2 * H * (sum(rows) * hd * 3 + blocks(rows)) + 4 * B, flops=2 * 2 * H * sum(rows) * hd)
    if case["op"] == "read":
        rows = [max(0, min(case["n"], n - case["row0"])) for n in lens]
        return dict(bytes=2 * H * (sum(rows) * hd * 3 + blocks(rows)) + 4 * B, flops=2 * H * sum(rows) * hd)
    C, Hq = case["C"], case["Hq"]
    new = (C * C if not case["causal"] else C * (C + 1) // 2) if case["tail"] else 0
    pairs = sum(n * C for n in lens) + B * new
    moved = 2 * H * (sum(lens) * hd + blocks(lens)) + 4 * B + 2 * (2 * B * Hq * C * hd + (2 * B * H * C * hd if case["tail"] else 0))
    return dict(bytes=moved, flops=4 * Hq * hd * pairs)


# ---------------------------------------------------------- exact, 64 bits ----
def _round_e4m3(y):
    """y (64 bits) to the nearest E4M3 value, ties to even, largest 448."""
    a = y.abs().clamp(max=448.0)
    power = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(power - 3)
    return torch.sign(y) * torch.round(a / step) * step


def _exact_append(codes, exps, x, lens, counts):
    value = codes.view(torch.float8_e4m3fn).double()
    exps = exps.clone()
    for b, (start, n) in enumerate(zip(lens, counts)):
        at = start
        while at < start + n:
            blk = at // BLOCK
            # the whole blocks of a long run share one pass, the first partial one goes alone
            end = min(start + n, (blk + 1) * BLOCK) if at % BLOCK or start + n - at < BLOCK else at + (start + n - at) // BLOCK * BLOCK
            k = max(1, (end - at) // BLOCK) if at % BLOCK == 0 and (end - at) % BLOCK == 0 else 1
            new = x[b, :, at - start:end - start].double()
            top = new.abs().reshape(new.shape[0], k, -1).amax(-1)
            e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)).clamp(E_MIN, E_MAX)
            e = torch.where(top > 448.0 * torch.exp2(e), e + 1, torch.where((top <= 224.0 * torch.exp2(e)) & (e > E_MIN), e - 1, e))
            if at % BLOCK:
                was = exps[b, :, blk:blk + 1].double() - BIAS
                e = torch.maximum(e, was)
                back = blk * BLOCK
                value[b, :, back:at] = _round_e4m3(value[b, :, back:at] * torch.exp2(was - e)[..., None])
            rows = e.repeat_interleave((end - at) // k, -1)[..., None]
            value[b, :, at:end] = _round_e4m3(new * torch.exp2(-rows))
            exps[b, :, blk:blk + k] = (e + BIAS).to(torch.uint8)
            at = end
    return value, exps


def _exact_value(codes, exps, first, last):
    """Rows first..last-1 of one sequence, in 64 bits."""
    row = torch.arange(first, last, device=codes.device)
    scale = torch.exp2(exps[:, row // BLOCK].double() - BIAS)
    return codes[:, first:last].view(torch.float8_e4m3fn).double() * scale[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    lens = _lengths(case)
    if case["op"] == "append":
        K, Ke = _exact_append(s["K"], s["Ke"], s["k"], lens, _counts(case))
        V, Ve = _exact_append(s["V"], s["Ve"], s["v"], lens, _counts(case))
        return dict(K=K, V=V, Ke=Ke, Ve=Ve)
    if case["op"] == "read":
        out = {}
        for name, codes, exps in (("k", s["K"], s["Ke"]), ("v", s["V"], s["Ve"])):
            out[name] = torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda")
            for b, n in enumerate(lens):
                last = min(n, case["row0"] + case["n"])
                if last > case["row0"]:
                    out[name][b, :, :last - case["row0"]] = _exact_value(codes[b], exps[b], case["row0"], last)
        return out
    B, H, C, hd, Hq = case["B"], case["Hkv"], case["C"], case["hd"], case["Hq"]
    o = torch.zeros(B, C, Hq, hd, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        K, V = _exact_value(s["K"][b], s["Ke"][b], 0, n), _exact_value(s["V"][b], s["Ve"][b], 0, n)
        if case["tail"]:
            K, V = torch.cat([K, s["k"][b].double()], 1), torch.cat([V, s["v"][b].double()], 1)
        if K.shape[1] == 0:
            continue  # nothing to attend to: zero
        for h in range(Hq):
            x = s["q"][b, h].double() @ K[h // (Hq // H)].T / np.sqrt(hd)
            if case["tail"] and case["causal"]:
                i = torch.arange(C, device="cuda")
                x[:, n:] = x[:, n:].masked_fill(i[None, :] > i[:, None], float("-inf"))
            if x.shape[1]:
                o[b, :, h] = torch.softmax(x, -1) @ V[h // (Hq // H)]
    return dict(o=o.reshape(B * C, Hq * hd))
