"""Sampling with temperature, top-k, top-p and min-p, restated in 64 bits, and whether a drawn token is right.

The kernel's weights are whole numbers.  x = l log2(e) / T keeps 2^-46 of itself; of the remainder r <= 1 / 128 and
2^r - 1 = q <= 0.0055, r is rounded to 2^-32, q to three steps of 2^-24 of itself (2^-30), the table and the sum to
half a unit of 2^-29 each, and the series ends at 2^-34: less than 2^-28 of the weight altogether.  Rounding down to the
row's unit, the largest being 2^41 at least, takes 2^-41 of the largest.  So a sum over n weights is off by
2^-28 of itself and n 2^-41 of the largest, and a border is undecided within twice that."""
import torch

FMAX = torch.finfo(torch.float32).max


def order_of(x):
    return torch.argsort(x, dim=-1, descending=True, stable=True)


def check_row(x, u, T, top_k, top_p, min_p, token, logprob, kept):
    """None, or what is wrong with a row's outputs."""
    x = x.double()
    V = x.numel()
    fine = x > -float("inf")
    ok = bool((x == x).all()) and not bool((x == float("inf")).any()) and bool(fine.any())
    ok = ok and T >= 0 and T <= FMAX and top_p >= 0 and 0 <= min_p <= 1 and top_k >= 0 and 0 <= u < 1
    if not ok:
        return None if token == -1 and logprob != logprob and kept == 0 else "a row that cannot be drawn from"
    m = x.max()
    if T < 2.0 ** -64 or top_k == 1:
        first = int((x == m).nonzero()[0])
        return None if (token, logprob, kept) == (first, 0.0, 1) else f"greedy: {first}, 0, 1"
    w = torch.where(fine, torch.exp((x - m) / T), 0.0)
    order = order_of(x)
    n = int(fine.sum())
    n = min(n, top_k) if top_k else n
    lo = hi = n
    off = 2 * (2.0 ** -28 + V * 2.0 ** -41)     # of the total, which is 1 at least
    if top_p < 1:
        run = w[order[:n]].cumsum(0)
        need = top_p * run[-1]
        lo = int((run < need - off * run[-1]).sum()) + 1
        hi = min(n, int((run < need + off * run[-1]).sum()) + 1)
    if min_p > 0:
        edge = 2.0 ** -50
        a = int((w[order] >= min_p * (1 + edge)).sum())
        b = int((w[order] >= min_p * (1 - edge)).sum())
        lo, hi = min(lo, a), min(hi, b)
    if not lo <= kept <= hi:
        return f"kept {kept}, not {lo} to {hi}"
    keep = torch.zeros(V, dtype=torch.bool)
    keep[order[:kept]] = True
    if not 0 <= token < V or not keep[token]:
        return f"token {token} is not kept"
    run = torch.where(keep, w, 0.0).cumsum(0)
    total = run[-1]
    if not run[token] - w[token] - off * total <= u * total <= run[token] + off * total:
        return f"token {token}: its share ends at {float(run[token] / total)}, u is {u}"
    if w[token] <= 0 and u > off:
        return "a token without weight"
    want = (x[token] - m) / T - torch.log(total)
    if abs(float(want) - logprob) > 2.0 ** -23 * abs(float(want)) + off + 2.0 ** -40:
        return f"logprob {logprob}, not {float(want)}"
    return None
