"""The 4-bit matrices restated: quantisation in IEEE float32 as the header defines it, weights and products in 64 bits."""
import torch


def quantize(W, group):
    """(codes uint8 [N, K], scales bf16 [N, K / group]) of a bf16 matrix."""
    N, K = W.shape
    w = W.float().reshape(N, K // group, group)
    top = torch.where(w.isfinite(), w.abs(), 0.0).amax(-1)
    s = (top / 7).to(torch.bfloat16)
    sf = s.float()[..., None]
    q = torch.where(sf > 0, (w / sf).round(), torch.zeros(())).clamp(-7, 7)   # round: ties to even
    q = torch.where(w.isnan(), 0.0, q)
    return (q + 8).to(torch.uint8).reshape(N, K), s


def weights(codes, scales):
    """The weights in 64 bits."""
    N, K = codes.shape
    return (codes.double() - 8) * scales.double().repeat_interleave(K // scales.shape[1], 1)


def product(codes, scales, x, alpha=None, coef=1.0, resid=None, dtype=torch.float32):
    """(y, tolerance) in 64 bits.

    The products x w / s are exact in fp32; a group's are added on the tensor cores, 16 and the running sum to an
    instruction, each addend good to 2^-24 of the largest, then scaled and added: with S = sum |x w| every one of
    the K products and K / 32 scaled sums adds at most 2^-24 S (1.1 K 2^-24 S in all, 2^-23 K S has room).  coef
    alpha, its product with the sum and the residual's addition are one fp32 rounding each, the output is rounded by
    half a step."""
    w = weights(codes, scales)
    f = float(torch.tensor(coef, dtype=torch.float32)) * (torch.ones(x.shape[0]) if alpha is None else alpha).double()[:, None]
    y, S = f * (x.double() @ w.T), f.abs() * (x.double().abs() @ w.T.abs())
    tol = S * (x.shape[1] * 2.0 ** -23 + 2.0 ** -22)
    if resid is not None:
        y = y + resid.double()
        tol = tol + 2.0 ** -23 * (S + resid.double().abs())
    return y, tol + y.abs() * torch.finfo(dtype).eps / 2
