"""The operators of a decoded token: what is measured, in a plain form.

Next to the 8-bit cache's append and attention, a step of one or a few tokens
needs four more operators:

* w4     a few rows times a matrix of 4-bit weights with a scale per group
* qk     norms of the query and key heads with the position rotation, split
         from the packed projection into the layouts that attention takes
* moe    a whole mixture-of-experts block for a few tokens
* sample a token from logits with temperature, top-k, top-p and min-p, by
         given random numbers
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one new token's heads: the smallest call, all latency
        dict(name="qk_token_b1", op="qk", B=1, C=1, Hq=8, Hkv=2, hd=128, gain=True, top=8192),
        # four prompts' pieces of 4096 tokens, far into a long prefix
        dict(name="qk_prompt_16k", op="qk", B=4, C=4096, Hq=16, Hkv=8, hd=128, gain=True, top=131072),
        # the packed q, k, v projection of one token
        dict(name="w4_qkv_m1", op="w4", M=1, N=4096, K=2816, group=64, out="bf16", resid=False),
        # the output projection with its residual, seven sequences, finer groups
        dict(name="w4_out_m7_g32", op="w4", M=7, N=2816, K=2048, group=32, out="bf16", resid=True),
        # the full-vocabulary LM head of one token
        dict(name="w4_head_m1", op="w4", M=1, N=262144, K=2816, group=64, out="f32", resid=False),
        # .. and of a batch of 32 sequences
        dict(name="w4_head_m32", op="w4", M=32, N=262144, K=2816, group=128, out="f32", resid=False),
        # a small expert layer, three tokens: latency
        dict(name="moe_small_m3", op="moe", M=3, d=1024, n_exp=16, top_k=2, Fe=512),
        # the 128-expert layer for one token
        dict(name="moe_m1", op="moe", M=1, d=2816, n_exp=128, top_k=8, Fe=768),
        # .. and for a batch of 16 sequences, most experts busy
        dict(name="moe_m16", op="moe", M=16, d=2816, n_exp=128, top_k=8, Fe=768),
        # one sequence's token from the full vocabulary
        dict(name="sample_r1_v262k", op="sample", R=1, V=262144, logits="f32"),
        # 32 sequences, each with settings of its own, bf16 logits (many ties), an odd vocabulary
        dict(name="sample_r32_bf16", op="sample", R=32, V=50257, logits="bf16"),
        # every position of a 256-token canvas
        dict(name="sample_r256_v262k", op="sample", R=256, V=262144, logits="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["qk", "w4", "w4", "moe", "moe", "sample", "sample"])
    if op == "qk":
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4])
        C = _log(rng, 1, 4096)
        return dict(op=op, B=_log(rng, 1, max(1, min(48, 16384 // C))), C=C, Hq=Hkv * min(G, 16 // Hkv), Hkv=Hkv,
                    hd=rng.choice([32, 64, 128]), gain=rng.random() < 0.8, top=_log(rng, 4096, 1 << 20))
    if op == "w4":
        group = rng.choice([32, 64, 64, 128])
        K = max(64, group) * _log(rng, 1, 8192 // max(64, group))
        return dict(op=op, M=_log(rng, 1, 32), N=_log(rng, 1, min(262144, (1 << 29) // K)), K=K, group=group,
                    out=rng.choice(["bf16", "f32"]), resid=rng.random() < 0.4)
    if op == "moe":
        d, Fe = 128 * _log(rng, 1, 22), 128 * _log(rng, 1, 8)
        n = _log(rng, 2, max(2, min(256, 270_000_000 // (d * Fe))))
        return dict(op=op, M=_log(rng, 1, min(32, max(1, (1 << 30) // (d * Fe * 8)))), d=d, n_exp=n,
                    top_k=rng.randint(1, min(8, n)), Fe=Fe)
    V = _log(rng, 2, 262144)
    return dict(op=op, R=_log(rng, 1, min(256, (1 << 25) // V)), V=V, logits=rng.choice(["f32", "bf16"]))


# ----------------------------------------------------------------- inputs ----
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    bf = torch.bfloat16

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = dict(case=case)
    if case["op"] == "qk":
        B, C, hd = case["B"], case["C"], case["hd"]
        heads = case["Hq"] + 2 * case["Hkv"]
        # projections of unit size with stronger and weaker heads
        x = randn(B, C, heads, hd) * torch.exp(0.7 * randn(heads, 1))
        s["qkv"] = x.reshape(B, C, heads * hd).to(bf)
        s["pos"] = torch.randint(0, case["top"] - C + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["q_gain"] = (1 + 0.2 * randn(hd)).to(bf) if case["gain"] else None
        s["k_gain"] = (1 + 0.2 * randn(hd)).to(bf) if case["gain"] else None
    elif case["op"] == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        # codes as rounding normal weights on a group's largest leaves them: few at the ends
        s["codes"] = torch.empty(N, K, dtype=torch.uint8, device="cuda")
        for n0 in range(0, N, 65536):
            c = s["codes"][n0:n0 + 65536]
            c.copy_(randn(*c.shape).mul_(2.6).round_().clamp_(-7, 7).add_(8))
        s["scales"] = (torch.exp(0.2 * randn(N, K // case["group"])) / (2.6 * math.sqrt(K))).to(bf)
        s["x"] = (randn(M, K) * torch.exp(0.5 * randn(K))).to(bf)
        s["alpha"] = torch.exp(rand(M) * 2) if case["out"] == "f32" else None
        s["resid"] = randn(M, N).to(bf) if case["resid"] else None
        if own:
            from block_diffusion_text_gb300 import dg
            s["W"] = dg.W4Matrix.from_codes(s["codes"], s["scales"])
    elif case["op"] == "moe":
        M, d, n, Fe = case["M"], case["d"], case["n_exp"], case["Fe"]
        s["h"] = randn(M, d).to(bf)
        s["Wr"] = (randn(n, d) / math.sqrt(d)).to(bf)
        s["We1"] = torch.empty(n + 1, Fe, d, dtype=bf, device="cuda").normal_(0, 1 / math.sqrt(d), generator=g)
        s["We2"] = torch.empty(n + 1, d, Fe, dtype=bf, device="cuda").normal_(0, 1 / math.sqrt(Fe), generator=g)
        if own:
            from block_diffusion_text_gb300 import dg
            s["ffn"] = dg.MoeFfn(s["Wr"], s["We1"], s["We2"], top_k=case["top_k"], rms_eps=EPS)
    else:
        R, V = case["R"], case["V"]
        # rows from nearly flat to sharp, with a few tokens banned
        x = randn(R, V) * torch.exp(math.log(0.7) + math.log(8) * rand(R, 1))
        ban = torch.randint(0, V, (R, 16), generator=g, device="cuda")
        x.scatter_(1, ban, float("-inf"))
        x[:, 0] = 0.0  # every row keeps a token
        s["logits"] = x if case["logits"] == "f32" else x.to(bf)
        s["u"] = rand(R)
        s["temperature"] = 0.4 + rand(R)
        pick = torch.randint(0, 4, (R,), generator=g, device="cuda")
        s["top_k"] = torch.where(pick % 2 == 0, (2 ** (1 + 9 * rand(R))).to(torch.int32), 0).to(torch.int32)
        s["top_p"] = torch.where(pick >= 1, 0.5 + 0.49 * rand(R), 1.0)
        s["min_p"] = torch.where(pick == 3, 0.1 * rand(R), 0.0)
    return s


# ------------------------------------------------------------- plain forms ----
def _plain_w4(s):
    case = s["case"]
    N, K, group = case["N"], case["K"], case["group"]
    w = s["codes"].to(torch.float32).sub_(8).reshape(N, K // group, group)
    w.mul_(s["scales"].float()[..., None])
    y = s["x"].float() @ w.reshape(N, K).T
    if s["alpha"] is not None:
        y = y * (s["alpha"] / math.sqrt(K))[:, None]
    if s["resid"] is not None:
        y = y + s["resid"].float()
    return dict(y=y if case["out"] == "f32" else y.to(torch.bfloat16))


def _plain_qk(s):
    case, x = s["case"], s["qkv"].float()
    B, C, Hq, Hkv, hd = case["B"], case["C"], case["Hq"], case["Hkv"], case["hd"]
    x = x.reshape(B, C, Hq + 2 * Hkv, hd).transpose(1, 2)
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    # angles in 64 bits: far positions lose them in 32
    j = torch.arange(hd // 2, device=x.device, dtype=torch.float64)
    at = s["pos"].double()[:, None] + torch.arange(C, device=x.device, dtype=torch.float64)
    a = at[..., None] * BASE ** (-2 * j / hd)
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]

    def turned(t, gain):
        t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS)
        if gain is not None:
            t = t * gain.float()
        lo, hi = t[..., :hd // 2], t[..., hd // 2:]
        return torch.cat([lo * cos - hi * sin, lo * sin + hi * cos], -1).to(torch.bfloat16)

    return dict(q=turned(q, s["q_gain"]), k=turned(k, s["k_gain"]), v=v.to(torch.bfloat16))


def _gelu(x):
    return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))


def _plain_moe(s):
    case, h = s["case"], s["h"].float()
    x = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    # value descending, the lower index first where two are equal
    value, order = (x @ s["Wr"].float().T).sort(dim=-1, descending=True, stable=True)
    idx = order[:, :case["top_k"]]
    gate = torch.softmax(value[:, :case["top_k"]], -1)
    # every token's own experts' matrices, the shared one (index n_exp) behind them
    idx = torch.cat([idx, torch.full_like(idx[:, :1], case["n_exp"])], 1)
    gate = torch.cat([gate, torch.ones_like(gate[:, :1])], 1)
    a = _gelu((s["We1"][idx].float() @ x[:, None, :, None]).squeeze(-1))            # [M][k + 1][Fe]
    y = (s["We2"][idx].float() @ a[..., None]).squeeze(-1)                          # [M][k + 1][d]
    return dict(h=(h + (gate[..., None] * y).sum(1)).to(torch.bfloat16))


def _plain_sample(s):
    # in 64 bits: sums over the vocabulary are compared with a border
    x = s["logits"].float()
    R, V = x.shape
    value, order = x.sort(dim=-1, descending=True, stable=True)
    w = torch.exp((value.double() - value[:, :1].double()) / s["temperature"].double()[:, None])
    rank = torch.arange(V, device=x.device)
    k = s["top_k"].long()[:, None]
    w = torch.where((k == 0) | (rank < k), w, 0.0)
    run = w.cumsum(-1)
    p = s["top_p"].double()[:, None]
    # the smallest leading run that reaches p: what starts below it
    w = torch.where((p >= 1) | (run - w < p * run[:, -1:]), w, 0.0)
    w = torch.where(w >= s["min_p"].double()[:, None], w, 0.0)
    by_token = torch.zeros_like(w).scatter_(1, order, w)
    run = by_token.cumsum(-1)
    total = run[:, -1:]
    token = (run > s["u"].double()[:, None] * total).to(torch.int8).argmax(-1)
    prob = by_token.gather(1, token[:, None]) / total
    return dict(token=token.to(torch.int32), logprob=prob.log().squeeze(1).float(), kept=(w > 0).sum(-1).to(torch.int32))


def run(s):
    case = s["case"]
    if own:
        from block_diffusion_text_gb300 import dg
        if case["op"] == "w4":
            return dict(y=dg.w4_matvec(s["W"], s["x"], alpha=s["alpha"],
                                       coef=1 / math.sqrt(case["K"]) if s["alpha"] is not None else 1.0, resid=s["resid"],
                                       dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16))
        if case["op"] == "qk":
            q, k, v = dg.qk_norm_rope(s["qkv"], s["pos"], case["Hq"], case["Hkv"], s["q_gain"], s["k_gain"], rms_eps=EPS,
                                      rope_base=BASE)
            return dict(q=q, k=k, v=v)
        if case["op"] == "moe":
            return dict(h=dg.moe_tokens(s["ffn"], s["h"]))
        token, logprob, kept = dg.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                         min_p=s["min_p"])
        return dict(token=token, logprob=logprob, kept=kept)
    return dict(w4=_plain_w4, qk=_plain_qk, moe=_plain_moe, sample=_plain_sample)[case["op"]](s)


# ------------------------------------------------------------------- work ----
def work(case):
    """Bytes: every input read once, every output written once; of the experts those that this many tokens choose."""
    if case["op"] == "qk":
        n = case["B"] * case["C"] * (case["Hq"] + 2 * case["Hkv"]) * case["hd"]
        return dict(bytes=4 * n + 4 * case["B"], flops=8 * n)
    if case["op"] == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        out = 4 if case["out"] == "f32" else 2
        return dict(bytes=N * K // 2 + 2 * N * K // case["group"] + 2 * M * K + M * N * (out + 2 * case["resid"]), flops=2 * M * N * K)
    if case["op"] == "moe":
        M, d, n, k, Fe = case["M"], case["d"], case["n_exp"], case["top_k"], case["Fe"]
        busy = n * (1 - (1 - k / n) ** M) + 1
        return dict(bytes=4 * busy * d * Fe + 2 * n * d + 4 * M * d, flops=4 * M * (k + 1) * d * Fe + 2 * M * n * d)
    n = case["R"] * case["V"]
    return dict(bytes=n * (4 if case["logits"] == "f32" else 2) + 32 * case["R"], flops=4 * n)


# ---------------------------------------------------------- exact, 64 bits ----
def _exact_sample(s):
    token, logprob = [], []
    for r in range(s["logits"].shape[0]):
        x = s["logits"][r].double()
        y = x / s["temperature"][r].double()
        k, p, least = int(s["top_k"][r]), float(s["top_p"][r]), float(s["min_p"][r])
        w = torch.exp(y - y.max())
        keep = torch.ones_like(w, dtype=torch.bool)
        order = torch.argsort(x, dim=-1, descending=True, stable=True)
        if k > 0:
            keep[order[k:]] = False
        if p < 1:
            mass = torch.where(keep, w, 0.0)[order].cumsum(0)
            n = int((mass < p * mass[-1]).sum()) + 1
            keep[order[n:]] = False
        keep &= w >= least
        mass = torch.where(keep, w, 0.0).cumsum(0)
        i = int((mass <= s["u"][r].double() * mass[-1]).sum())
        token.append(i)
        logprob.append(float(torch.log(w[i] / mass[-1])))
    return dict(token=None, logprob=torch.tensor(logprob, dtype=torch.float64, device="cuda"), kept=None)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    if case["op"] == "w4":
        M, N, K, group = case["M"], case["N"], case["K"], case["group"]
        y = torch.empty(M, N, dtype=torch.float64, device="cuda")
        x = s["x"].double()
        for n0 in range(0, N, 16384):
            w = (s["codes"][n0:n0 + 16384].double() - 8) * s["scales"][n0:n0 + 16384].double().repeat_interleave(group, 1)
            y[:, n0:n0 + 16384] = x @ w.T
        if s["alpha"] is not None:
            y *= s["alpha"].double()[:, None] / math.sqrt(K)
        if s["resid"] is not None:
            y += s["resid"].double()
        return dict(y=y)
    if case["op"] == "qk":
        B, C, Hq, Hkv, hd = case["B"], case["C"], case["Hq"], case["Hkv"], case["hd"]
        x = s["qkv"].double().reshape(B, C, Hq + 2 * Hkv, hd)
        out = dict(q=torch.empty(B, Hq, C, hd, dtype=torch.float64, device="cuda"),
                   k=torch.empty(B, Hkv, C, hd, dtype=torch.float64, device="cuda"),
                   v=x[:, :, Hq + Hkv:].transpose(1, 2).contiguous())
        i = torch.arange(C, device="cuda", dtype=torch.float64)
        theta = torch.exp(-math.log(BASE) / hd * torch.arange(0, hd, 2, device="cuda", dtype=torch.float64))
        for b in range(B):
            z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), (i + float(s["pos"][b]))[:, None] * theta)
            for name, first, heads in (("q", 0, Hq), ("k", Hq, Hkv)):
                t = x[b, :, first:first + heads]
                t = t / torch.sqrt((t * t).sum(-1, keepdim=True) / hd + EPS)
                if s[name + "_gain"] is not None:
                    t = t * s[name + "_gain"].double()
                c = torch.complex(t[..., :hd // 2], t[..., hd // 2:]) * z[:, None]
                out[name][b] = torch.cat([c.real, c.imag], -1).transpose(0, 1)
        return out
    h = s["h"].double()
    x = h / torch.sqrt((h * h).sum(-1, keepdim=True) / case["d"] + EPS)
    for m in range(case["M"]):
        logit = s["Wr"].double() @ x[m]
        best = torch.argsort(logit, dim=-1, descending=True, stable=True)[:case["top_k"]]
        gate = torch.exp(logit[best] - logit[best].max())
        gate = (gate / gate.sum()).tolist()
        for e, w in zip(best.tolist() + [case["n_exp"]], gate + [1.0]):
            a = s["We1"][e].double() @ x[m]
            h[m] += w * (s["We2"][e].double() @ (0.5 * a * torch.special.erfc(-a / math.sqrt(2))))
    return dict(h=h)
