"""Attention over the 8-bit cache with elements, tokens and scales far from the others: what a row cannot see, and what
its keys do not use, costs it no bits, in whichever kernel the sizes select."""
import pytest
import torch

import kv8_ref
from block_diffusion_text_gb300 import dg
from test_gpu_kv8 import filled, rows, state

pytestmark = pytest.mark.gpu


def tight(K, V, Ke, Ve, lens, q, k, v, causal):
    """(o, tol) as kv8_ref.attention's, with a tolerance from the visible keys alone.

    Queries, new keys and new values are bf16 and a cached value is one, so the products are exact and a score is off
    by its fp32 accumulation only: ds_j = hd 2^-23 sum |q||k_j| (and 2^-21 of itself for the softmax factor and the
    argument's rounding).  It moves the output by sum_j p_j ds_j (|v_j| + A), A = sum_j p_j |v_j|.  Cached rows'
    probabilities are f16, 2^-11 of them, and have a floor of half a subnormal, 2^-25 under a row maximum of 2^8, for
    codes of at most 448 on the largest visible scale; those of new tokens are pairs of bf16, 2^-17.  The exponential
    is off by 2^-21, the sums over N keys by 2 N 2^-24, and the output is rounded to bf16, 2^-8."""
    B, Hq, C, hd = q.shape
    Hkv = K.shape[1]
    o = torch.zeros(B, C, Hq, hd, dtype=torch.float64)
    tol = torch.full_like(o, 1e-30)
    for b in range(B):
        n = int(lens[b])
        for h in range(Hq):
            g = h // (Hq // Hkv)
            kk, vv = kv8_ref.values(K[b, g, :n], Ke[b, g]), kv8_ref.values(V[b, g, :n], Ve[b, g])
            if k is not None:
                kk, vv = torch.cat([kk, k[b, g].double()]), torch.cat([vv, v[b, g].double()])
            N = kk.shape[0]
            if N == 0:
                continue
            seen = torch.ones(C, N, dtype=torch.bool)
            if k is not None and causal:
                seen[:, n:] = torch.ones(C, C, dtype=torch.bool).tril()
            qq = q[b, h].double()
            s = (qq @ kk.T) / hd ** 0.5
            p = torch.softmax(s.masked_fill(~seen, float("-inf")), -1)
            ds = torch.where(seen, hd * 2.0 ** -23 * (qq.abs() @ kk.abs().T) / hd ** 0.5 + 2.0 ** -21 * s.abs(), 0.0)
            o[b, :, h] = p @ vv
            A, cached = p @ vv.abs(), p[:, :n] @ vv[:n].abs()
            top = 448 * 2.0 ** (float(Ve[b, g, :-(-n // 64)].double().max()) - 127) if n else 0.0
            # the row sum is taken over the probabilities before their rounding
            tol[b, :, h] = 2.0 ** -8 * o[b, :, h].abs() + 2.0 ** -11 * cached + n * 2.0 ** -33 * top + 1e-30 \
                + (2.0 ** -17 + 2.0 ** -20 + 4 * N * 2.0 ** -24) * A + (p * ds) @ vv.abs() + (p * ds).sum(-1, keepdim=True) * A
    return o.reshape(B * C, Hq * hd), tol.reshape(B * C, Hq * hd)


def check(c, q, k, v, causal):
    K, V, Ke, Ve, ln = state(c)
    want, tol = tight(K, V, Ke, Ve, ln, q, k, v, causal)
    got = dg.kv8_attention(c, *[None if t is None else t.cuda() for t in (q, k, v)], causal=causal)
    torch.cuda.synchronize()
    assert torch.isfinite(got).all()
    off = (got.cpu().double() - want).abs()
    assert (off <= tol).all(), f"largest error over tolerance {float((off / tol).max()):.3f}"
    assert c.status() == 0


# C, hd, cap: single tokens, short and long caches, pieces of few and of many rows, both head dims of the tensor cores
SIZES = [(1, 128, 400), (3, 32, 400), (40, 128, 400), (40, 128, 3000), (256, 128, 400), (256, 128, 3000), (40, 64, 5000),
         (256, 64, 5000), (130, 128, 3000), (40, 128, 20000), (60, 64, 20000)]
ids = [f"c{c}h{h}cap{n}" for c, h, n in SIZES]


@pytest.mark.parametrize("C,hd,cap", SIZES, ids=ids)
def test_ordinary_rows(C, hd, cap):
    g = torch.Generator().manual_seed(50)
    for causal in (False, True):
        c = filled(g, 2, 2, cap, hd, [390, 65])
        check(c, rows(g, 2, 4, C, hd), rows(g, 2, 2, C, hd), rows(g, 2, 2, C, hd), causal)


@pytest.mark.parametrize("power", [8, 12, 16])
@pytest.mark.parametrize("C,hd,cap", SIZES, ids=ids)
def test_query_elements_that_no_key_uses(C, hd, cap, power):
    """One channel of the queries 2^power times the others, zero in every key: it takes no part in any score."""
    g = torch.Generator().manual_seed(51)
    c = filled(g, 1, 2, cap, hd, [390])
    c.K[:, :, :, 5] = 0
    q, k, v = rows(g, 1, 4, C, hd), rows(g, 1, 2, C, hd), rows(g, 1, 2, C, hd)
    q[..., 5] = 2.0 ** power * torch.randn(1, 4, C, generator=g).sign().to(torch.bfloat16)
    k[..., 5] = 0
    check(c, q, k, v, False)


@pytest.mark.parametrize("power", [8, 12, 16, 20])
@pytest.mark.parametrize("C,hd,cap", SIZES[1:], ids=ids[1:])
def test_tokens_behind_the_causal_mask(C, hd, cap, power):
    """The last new tokens, seen by themselves alone (in a ragged piece: padding), with keys and values 2^power
    times the others'."""
    g = torch.Generator().manual_seed(52)
    c = filled(g, 2, 2, cap, hd, [390, 0])
    q, k, v = rows(g, 2, 4, C, hd), rows(g, 2, 2, C, hd), rows(g, 2, 2, C, hd)
    k[:, :, C - 1] *= 2.0 ** power
    v[:, :, C - 1] *= 2.0 ** power
    k[1, 1, C - 2] *= -2.0 ** power
    check(c, q, k, v, True)


@pytest.mark.parametrize("power", [8, 12, 16])
@pytest.mark.parametrize("C,hd,cap", SIZES, ids=ids)
def test_tokens_that_get_no_weight(C, hd, cap, power):
    """A new token that all rows see, whose key is 2^power times the others' and points away from every query."""
    g = torch.Generator().manual_seed(53)
    c = filled(g, 1, 2, cap, hd, [390])
    q, k, v = rows(g, 1, 4, C, hd), rows(g, 1, 2, C, hd), rows(g, 1, 2, C, hd)
    q[..., 7] = 1
    k[:, :, C // 2] = 0
    k[:, :, C // 2, 7] = -2.0 ** power
    check(c, q, k, v, False)


@pytest.mark.parametrize("power", [-40, -90, -100, -120, 50])
@pytest.mark.parametrize("C,hd,cap", SIZES, ids=ids)
def test_small_queries_over_large_keys(C, hd, cap, power):
    """Queries of 2^power over keys 2^-power times larger: ordinary scores."""
    g = torch.Generator().manual_seed(54)
    c = filled(g, 1, 2, cap, hd, [390])
    c.K_exp -= power
    q, k, v = rows(g, 1, 4, C, hd) * 2.0 ** power, rows(g, 1, 2, C, hd) * 2.0 ** -power, rows(g, 1, 2, C, hd)
    check(c, q, k, v, False)


@pytest.mark.parametrize("C,hd,cap", SIZES, ids=ids)
def test_a_sequence_without_numbers_stays_alone(C, hd, cap):
    """NaN and infinities in one sequence's queries, keys and values (which the call does not take: its own rows are
    not to be used) leave the other sequences' rows as they are."""
    g = torch.Generator().manual_seed(55)
    c = filled(g, 3, 2, cap, hd, [390, 65, 200])
    q, k, v = rows(g, 3, 4, C, hd), rows(g, 3, 2, C, hd), rows(g, 3, 2, C, hd)
    want = dg.kv8_attention(c, q.cuda(), k.cuda(), v.cuda())
    q[1], k[1], v[1, 0], v[1, 1] = float("nan"), float("nan"), float("inf"), float("nan")
    got = dg.kv8_attention(c, q.cuda(), k.cuda(), v.cuda())
    assert torch.equal(got[:C], want[:C]) and torch.equal(got[2 * C:], want[2 * C:])
