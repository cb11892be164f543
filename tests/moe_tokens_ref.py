"""The mixture-of-experts block restated in 64 bits."""
import math

import torch


def gelu(x):
    return 0.5 * x * torch.special.erfc(-x / math.sqrt(2))


def block(h, Wr, We1, We2, top_k, eps=1e-6, idx=None):
    """(out, tolerance, idx, gates, fair) in 64 bits.  idx: the experts to take, by default the top_k; fair says
    whether none of them lies below one left out by more than the logits' errors.

    u = 2^-24.  Logits and first products: K = d products, each and their sums good to 2^-23 of S = sum |x w| per 16
    added on the tensor cores, d 2^-23 S in all (w4_ref.product); the rms and its product (d + 6) u relative.  A
    hidden value's error grows by GELU's slope (at most 1.13) and erff's own 4 u; the gate's error is twice its logits'
    (absolute, in the exponent), and 8 u; the pair of bf16 leaves 2^-17 of the value.  The second product carries the
    hidden errors by |We2|, and Fe 2^-23 of its own sum for each expert; all sums together run over at most
    (n_exp + 1) Fe products.  Then half a step of bf16 of h + y."""
    u = 2.0 ** -24
    M, d = h.shape
    n, Fe = Wr.shape[0], We1.shape[1]
    x = h.double()
    inv = 1 / (x.square().mean(-1, keepdim=True) + float(torch.tensor(eps, dtype=torch.float32))).sqrt()
    x = x * inv
    rel = (d + 6) * u
    logits = x @ Wr.double().T
    lerr = (x.abs() @ Wr.double().abs().T) * (d * 2 * u + rel)
    if idx is None:
        idx = logits.argsort(dim=-1, descending=True, stable=True)[:, :top_k]
    top = logits.gather(1, idx)
    gate = torch.softmax(top, -1)
    gerr = gate * (4 * lerr.amax(-1, keepdim=True) + 8 * u)
    left = logits.scatter(1, idx, -math.inf).amax(-1)
    fair = bool((top.amin(-1) >= left - 2 * lerr.amax(-1)).all()) and all(len(set(r)) == top_k for r in idx.tolist())
    out, tol = h.double().clone(), torch.zeros(M, d, dtype=torch.float64)
    adds = (n + 1) * Fe * 4 * u    # both terms of the pair
    for m in range(M):
        for e, g, ge in zip(idx[m].tolist() + [n], gate[m].tolist() + [1.0], gerr[m].tolist() + [0.0]):
            w1, w2 = We1[e].double(), We2[e].double()
            a = w1 @ x[m]
            aerr = (w1.abs() @ x[m].abs()) * (d * 2 * u + rel)
            v = gelu(a)
            verr = g * (1.13 * aerr + 8 * u * a.abs()) + ge * v.abs() + 2.0 ** -17 * g * v.abs()
            out[m] += g * (w2 @ v)
            tol[m] += w2.abs() @ (verr + adds * g * v.abs())
    return out, tol + (out.abs() + tol) * 2.0 ** -8 + 2 * u * h.double().abs(), idx, gate, fair
