"""The 8-bit prefix cache through its public entry points: append and read bit for bit, attention within
tolerances derived in kv8_ref.attention, against its definition in 64 bits."""
import pytest
import torch

import kv8_ref
from block_diffusion_text_gb300 import dg, synth

pytestmark = pytest.mark.gpu


def rows(g, *shape, spread=0.5):
    """bf16 rows of unit size with stronger and weaker channels and tokens."""
    x = torch.randn(*shape, generator=g)
    x = x * torch.exp(spread * torch.randn(shape[0], shape[1], 1, shape[3], generator=g))
    return (x * torch.exp(spread * torch.randn(shape[0], shape[1], shape[2], 1, generator=g))).to(torch.bfloat16)


def filled(g, B, H, cap, hd, lens, behind=0x7f):
    """A cache on the GPU holding `lens` rows of random codes; every byte behind them is `behind` (NaN codes), and
    the exponents of blocks without rows are 255."""
    t = []
    for _ in range(2):
        c = (torch.randn(B, H, cap, hd, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        e = (120 + torch.randint(-2, 3, (B, H, -(-cap // 64)), generator=g)).to(torch.uint8)
        for b, n in enumerate(lens):
            c[b, :, n:] = behind
            e[b, :, -(-n // 64):] = 255
        t += [c, e]
    ln = torch.tensor(lens, dtype=torch.int32)
    return dg.Kv8Cache(*[x.cuda() for x in (t[0], t[2], t[1], t[3], ln)])


def state(c):
    return [t.cpu() for t in (c.K, c.V, c.K_exp, c.V_exp, c.len)]


def check_append(c, k, v, counts=None, status=0, **kw):
    K, V, Ke, Ve, ln = state(c)
    n = [k.shape[2]] * c.B if counts is None else counts
    wK, wKe = kv8_ref.append(K, Ke, k, ln, n)
    wV, wVe = kv8_ref.append(V, Ve, v, ln, n)
    ct = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    dg.kv8_append(c, k.cuda(), v.cuda(), counts=ct, **kw)
    torch.cuda.synchronize()
    gK, gV, gKe, gVe, gl = state(c)
    assert torch.equal(gl, ln)
    assert torch.equal(gKe, wKe) and torch.equal(gVe, wVe)
    assert torch.equal(gK, wK) and torch.equal(gV, wV)
    assert c.status() == status


# ------------------------------------------------------------------ append ----
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("n,lens,cap", [(1, [0, 1, 63, 64, 65, 127], 200), (64, [0, 64, 1, 63, 100, 5], 190),
                                        (63, [1, 0, 2, 64, 65, 30], 150), (200, [0, 7, 64, 120, 200, 33], 401),
                                        (257, [3, 0, 63, 64, 143, 10], 400)])
def test_append_is_exact(hd, n, lens, cap):
    g = torch.Generator().manual_seed(n + hd)
    c = filled(g, len(lens), 2, cap, hd, lens)
    check_append(c, rows(g, len(lens), 2, n, hd), rows(g, len(lens), 2, n, hd, spread=2.0))


@pytest.mark.parametrize("hd", [32, 128])
def test_append_counts_leave_padding_out(hd):
    """Counts from 0 to n; the padding rows hold NaN, which must not reach a scale or the status word."""
    g = torch.Generator().manual_seed(5)
    counts, lens = [0, 1, 70, 130, 5, 129], [10, 0, 60, 64, 63, 1]
    c = filled(g, 6, 3, 300, hd, lens)
    k, v = rows(g, 6, 3, 130, hd), rows(g, 6, 3, 130, hd)
    for b, m in enumerate(counts):
        k[b, :, m:] = float("nan")
        v[b, :, m:] = float("inf")
    check_append(c, k, v, counts)


def test_append_token_by_token_grows_scales():
    """150 tokens one by one, magnitudes rising and falling over many octaves: scales grow within a block and the
    earlier codes move with them."""
    g = torch.Generator().manual_seed(6)
    c = filled(g, 2, 2, 256, 64, [0, 37])
    for i in range(150):
        x = rows(g, 2, 2, 1, 64) * float(torch.exp2(torch.randint(-14, 14, (1,), generator=g).float()))
        check_append(c, x, x.flip(3))
        c.len += 1


def test_append_extremes():
    """Zeros of both signs, subnormals, the largest values, ties between codes, and a block of zeros."""
    g = torch.Generator().manual_seed(7)
    tiny, big = 2.0 ** -133, 3.3895e38
    pats = [torch.zeros(64), torch.full((64,), -0.0), torch.full((64,), tiny), torch.full((64,), big),
            torch.full((64,), -big), torch.cat([torch.full((32,), big), torch.full((32,), 1.0)]),
            torch.cat([torch.full((1,), 448.0), torch.arange(63) / 16.0]),        # ties at the codes' midpoints
            torch.cat([torch.full((1,), 450.0), torch.arange(63) / 512.0]),       # one past 448: next scale
            torch.full((64,), 2.0 ** -74), torch.full((64,), 448 * 2.0 ** -64), torch.full((64,), 449 * 2.0 ** -64)]
    for start in (0, 13):
        for x in pats:
            c = filled(g, 1, 1, 128, 64, [start])
            x = x.to(torch.bfloat16).reshape(1, 1, 1, 64)
            check_append(c, x, -x)


def test_append_non_finite_values():
    """NaN is stored as 0, infinities saturate on the scale of the finite values, the status word says so."""
    g = torch.Generator().manual_seed(8)
    for start in (0, 20):
        c = filled(g, 2, 2, 256, 128, [start, start])
        k, v = rows(g, 2, 2, 100, 128), rows(g, 2, 2, 100, 128)
        k[0, 1, 3, 7] = float("nan")
        k[1, 0, 99, 127] = float("-inf")
        v[1, 1, 50] = float("inf")
        v[0, 0, 64:] = float("nan")
        check_append(c, k, v, status=dg.DG_ERR_VALUE)


def test_append_past_the_capacity_leaves_the_sequence():
    g = torch.Generator().manual_seed(9)
    c = filled(g, 3, 2, 100, 64, [90, 91, 0])
    check_append(c, rows(g, 3, 2, 10, 64), rows(g, 3, 2, 10, 64), status=dg.DG_ERR_CAPACITY)
    c = filled(g, 3, 2, 100, 64, [0, 0, 0])
    c.len[1] = -5
    check_append(c, rows(g, 3, 2, 10, 64), rows(g, 3, 2, 10, 64), status=dg.DG_ERR_CAPACITY)
    c = filled(g, 2, 2, 100, 64, [0, 0])
    K, V, Ke, Ve, ln = state(c)
    k = rows(g, 2, 2, 10, 64).cuda()
    dg.kv8_append(c, k, k, counts=torch.tensor([11, -1], dtype=torch.int32).cuda())
    assert c.status() == dg.DG_ERR_ARG and torch.equal(c.K.cpu(), K) and torch.equal(c.V_exp.cpu(), Ve)
    with pytest.raises(dg.DgError):
        k = rows(g, 2, 2, 101, 64).cuda()
        dg.kv8_append(c, k, k)


# -------------------------------------------------------------------- read ----
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("row0,n,pitch", [(0, 1, 1), (0, 200, 200), (37, 100, 130), (64, 64, 64), (199, 30, 31),
                                          (250, 5, 5)])
def test_read_is_exact_and_keeps_other_rows(hd, row0, n, pitch):
    g = torch.Generator().manual_seed(row0 + n)
    lens = [200, 0, 1, 64, 137]
    c = filled(g, 5, 2, 200, hd, lens)
    K, V, Ke, Ve, _ = state(c)
    out = [torch.full((5, 2, pitch, hd), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    got = dg.kv8_read(c, row0, n, out=out)
    for o, t, codes, exps in zip(got, out, (K, V), (Ke, Ve)):
        assert o is t
        want = torch.full((5, 2, pitch, hd), 7.0, dtype=torch.float64)
        val = kv8_ref.values(codes, exps)
        for b, m in enumerate(lens):
            last = min(m, row0 + n)
            if last > row0:
                want[b, :, :last - row0] = val[b, :, row0:last]
        assert torch.equal(o.cpu().double(), want)
    assert c.status() == 0


@pytest.mark.parametrize("hd", [32, 128])
def test_outputs_aligned_to_16_bytes_only(hd):
    """Outputs, queries and new rows that begin 16 bytes into an allocation."""
    g = torch.Generator().manual_seed(12)
    c = filled(g, 2, 1, 100, hd, [100, 50])

    def shifted(t):
        flat = torch.zeros(t.numel() + 8, dtype=t.dtype, device="cuda")
        flat[8:] = t.flatten().cuda()
        return flat[8:].view(t.shape)
    out = [shifted(torch.full((2, 1, 90, hd), 7.0).to(torch.bfloat16)) for _ in range(2)]
    assert out[0].data_ptr() % 32 == 16
    for a, b in zip(dg.kv8_read(c, 10, 90, out=out), dg.kv8_read(c, 10, 90)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1, :, :40], b[1, :, :40]) and (a[1, :, 40:] == 7).all()
    q, k, v = rows(g, 2, 2, 3, hd), rows(g, 2, 1, 3, hd), rows(g, 2, 1, 3, hd)
    o = shifted(torch.zeros(6, 2 * hd, dtype=torch.bfloat16))
    assert torch.equal(dg.kv8_attention(c, shifted(q), shifted(k), shifted(v), out=o),
                       dg.kv8_attention(c, q.cuda(), k.cuda(), v.cuda()))
    c.len -= 10
    one, two = [dg.Kv8Cache(*[t.clone() for t in (c.K, c.V, c.K_exp, c.V_exp, c.len)]) for _ in range(2)]
    dg.kv8_append(one, shifted(k), shifted(v))
    dg.kv8_append(two, k.cuda(), v.cuda())
    assert torch.equal(one.K, two.K) and torch.equal(one.V, two.V)


def test_read_covers_every_code_and_extreme_scales():
    for e in (63, 64, 120, 127, 200, 245):
        codes = torch.arange(256, dtype=torch.uint8).reshape(1, 1, 4, 64)
        codes[(codes & 0x7f) == 0x7f] = 0
        c = dg.Kv8Cache(codes.cuda(), codes.flip(2).contiguous().cuda(),
                        *[torch.full((1, 1, 1), e, dtype=torch.uint8).cuda() for _ in range(2)],
                        torch.tensor([4], dtype=torch.int32).cuda())
        K, V = dg.kv8_read(c, 0, 4)
        assert torch.equal(K.cpu().double(), kv8_ref.values(codes, torch.full((1, 1, 1), e)))
        assert torch.equal(V.cpu().double(), kv8_ref.values(codes.flip(2), torch.full((1, 1, 1), e)))


def test_append_then_read_is_within_half_a_step():
    """E4M3 keeps 2^-4 of a value in its normal range, and 2^-10 of the block's scale below it."""
    g = torch.Generator().manual_seed(11)
    c = dg.Kv8Cache.empty(2, 2, 300, 128)
    k, v = rows(g, 2, 2, 300, 128), rows(g, 2, 2, 300, 128)
    dg.kv8_append(c, k.cuda(), v.cuda())
    c.len += 300
    for got, x, e in zip(dg.kv8_read(c, 0, 300), (k, v), (c.K_exp, c.V_exp)):
        scale = torch.exp2(e.cpu().double() - 127).repeat_interleave(64, -1)[..., :300, None]
        bound = torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * scale)
        assert ((got.cpu().double() - x.double()).abs() <= bound).all()


# --------------------------------------------------------------- attention ----
def check_attention(c, q, k, v, causal, **kw):
    K, V, Ke, Ve, ln = state(c)
    want, tol = kv8_ref.attention(K, V, Ke, Ve, ln, q, k, v, causal)
    dev = [None if t is None else t.cuda() for t in (q, k, v)]
    got = dg.kv8_attention(c, *dev, causal=causal, **kw)
    torch.cuda.synchronize()
    off = (got.cpu().double() - want).abs()
    assert torch.isfinite(got).all()
    assert (off <= tol).all(), f"largest error over tolerance {float((off / tol).max()):.3f}"
    assert c.status() == 0
    return got


CASES = [
    # B, C, Hq, Hkv, hd, lens, causal, new tokens
    (1, 1, 1, 1, 128, [1], False, False),
    (1, 1, 1, 1, 32, [0], False, True),
    (3, 1, 4, 2, 128, [0, 1, 63], False, False),
    (6, 1, 8, 2, 128, [0, 64, 65, 127, 128, 2000], False, True),
    (2, 1, 16, 1, 128, [700, 31], True, True),
    (2, 1, 32, 1, 64, [129, 640], False, True),
    (4, 1, 8, 8, 64, [5, 64, 0, 333], False, False),
    (2, 1, 6, 2, 32, [1000, 33], False, True),
    (2, 3, 8, 4, 128, [100, 4097], True, True),
    (2, 5, 8, 2, 64, [50, 0], True, True),
    (2, 17, 2, 1, 32, [32, 95], False, True),
    (1, 16, 2, 1, 32, [32], False, True),
    (3, 40, 4, 2, 64, [0, 63, 300], True, True),
    (3, 33, 4, 2, 128, [0, 63, 300], False, True),
    (2, 64, 8, 2, 128, [1, 1025], True, True),
    (2, 100, 4, 4, 128, [128, 200], False, True),
    (1, 128, 2, 1, 128, [0], True, True),
    (2, 129, 2, 2, 128, [500, 0], True, True),
    (2, 250, 8, 2, 128, [385, 77], True, True),
    (1, 256, 16, 8, 128, [1024], False, True),
    (2, 256, 2, 2, 128, [640, 1], False, False),
    (1, 1000, 2, 2, 128, [130], True, True),
    (1, 200, 3, 1, 64, [777], True, True),
    # caches long enough that a sequence's keys are shared out over many warps
    (3, 1, 8, 2, 64, [5000, 0, 4200], True, True),
    (2, 17, 2, 1, 32, [4500, 100], False, True),
    (4, 1, 4, 4, 128, [6000, 1, 0, 3333], False, False),
    (2, 9, 2, 2, 64, [4097, 4096], True, True),
    # up to 128 rows on the tensor cores: the row tiles share the rows, each every other key tile
    (1, 17, 1, 1, 128, [0], False, True),
    (3, 20, 4, 2, 128, [0, 129, 1], True, True),
    (2, 32, 4, 1, 128, [3000, 255], False, True),
    (2, 128, 1, 1, 128, [256, 0], False, False),
    (5, 25, 10, 2, 128, [64, 640, 0, 127, 1111], True, True),
    # more sequences than lanes, most of them empty or short
    (70, 1, 4, 2, 128, [0, 5, 0, 64, 65] * 14, False, False),
    (40, 3, 2, 1, 32, [1, 0, 0, 0, 99, 4200, 7, 31] * 5, True, True),
    (36, 40, 2, 2, 128, [0, 200, 1] * 12, False, True),
    # several row tiles to a kv head
    (2, 300, 8, 2, 128, [100, 700], True, True),
    (1, 1024, 2, 1, 64, [70], True, True),
]


@pytest.mark.parametrize("case", CASES, ids=[f"b{c[0]}c{c[1]}q{c[2]}k{c[3]}h{c[4]}l{max(c[5])}{'c' * c[6]}{'n' * c[7]}"
                                             for c in CASES])
@pytest.mark.parametrize("room", [3, 1600])
def test_attention(case, room):
    """Each case in a cache with hardly any room left and in one with more, which takes other kernels."""
    B, C, Hq, Hkv, hd, lens, causal, new = case
    g = torch.Generator().manual_seed(sum(lens) + C)
    c = filled(g, B, Hkv, max(lens) + room, hd, lens)
    q = rows(g, B, Hq, C, hd)
    k, v = (rows(g, B, Hkv, C, hd), rows(g, B, Hkv, C, hd)) if new else (None, None)
    check_attention(c, q, k, v, causal)


EDGES = [
    # B, C, Hq, Hkv, hd, lens, cap, causal: the smallest call, many sequences, many heads to one kv head, the longest
    # pieces, and caches filled to the last row
    (1, 1, 1, 1, 32, [1], 1, True),
    (2500, 1, 1, 1, 32, [0, 1] * 1250, 1, False),
    (200, 2, 2, 1, 32, [0, 4200, 1, 64, 100] * 40, 4200, True),
    (1, 1, 2048, 1, 128, [300], 300, False),
    (1, 1, 2048, 1, 64, [300], 5000, False),
    (1, 1024, 1, 1, 32, [0], 5000, True),
    (2, 1024, 2, 1, 128, [64, 65], 65, True),
    (1, 1, 65535, 1, 32, [3], 3, False),
]


@pytest.mark.parametrize("case", EDGES, ids=[f"b{c[0]}c{c[1]}q{c[2]}h{c[4]}cap{c[6]}" for c in EDGES])
def test_attention_at_the_ends_of_its_range(case):
    B, C, Hq, Hkv, hd, lens, cap, causal = case
    g = torch.Generator().manual_seed(cap + C)
    c = filled(g, B, Hkv, cap, hd, lens)
    check_attention(c, rows(g, B, Hq, C, hd), rows(g, B, Hkv, C, hd), rows(g, B, Hkv, C, hd), causal)


LONG = [
    # B, C, Hq, Hkv, hd, lens, cap, causal: caches too long for a cluster of CTAs to a unit, sequences of any length
    (1, 1, 8, 2, 128, [69999], 70000, True),
    (2, 3, 4, 1, 128, [40000, 5], 70000, True),
    (1, 2, 2, 1, 64, [70000], 70000, False),
    (3, 5, 2, 1, 32, [0, 33000, 64], 70000, True),
    (1, 9, 2, 1, 128, [66000], 66003, True),
    # and caches that clusters of two to eight finish, several tiles to a warp
    (1, 1, 8, 2, 128, [32000], 32000, True),
    (2, 1, 8, 8, 128, [23000, 1], 23000, True),
    (5, 1, 4, 4, 64, [0, 9000, 65, 12000, 1], 12000, True),
    (9, 2, 8, 4, 32, [9000, 0, 1, 4000, 64, 63, 5, 8999, 700], 9000, True),
    (15, 1, 8, 4, 128, [5000, 0, 1, 4000, 64] * 3, 5000, True),
    (2, 40, 4, 2, 128, [6000, 129], 6000, True),
    # head dim 64 on the tensor cores
    (2, 40, 4, 2, 64, [20000, 129], 20000, True),
    (1, 256, 8, 2, 64, [5000], 9000, True),
    (2, 256, 2, 2, 64, [640, 1], 4000, False),
    (3, 64, 2, 1, 64, [0, 33000, 64], 40000, False),
    (2, 300, 8, 2, 64, [100, 700], 1000, True),
    (40, 70, 2, 1, 64, [1, 0, 64, 2000, 129] * 8, 2003, True),
    # more units than SMs: CTAs shared by groups of warps, down to one warp a unit, the last CTA not full
    (25, 1, 16, 8, 128, [0, 1, 64, 129, 700] * 5, 1000, True),
    (61, 1, 8, 8, 32, [5, 0, 64, 260] * 15 + [300], 300, False),
    (101, 16, 4, 4, 128, [0, 65, 200, 31, 1] * 20 + [199], 200, True),
    (201, 1, 4, 4, 128, [130, 0, 64, 1, 65, 7] * 33 + [2, 3, 4], 130, True),
    (301, 2, 8, 8, 64, [100, 0, 64] * 100 + [1], 127, True),
    # several whole units to a CTA
    (33, 4, 64, 8, 64, [128, 0, 170, 192, 5, 288, 271, 62, 204, 149, 190] * 3, 305, True),
    (33, 4, 64, 8, 64, [128, 0, 170, 192, 5, 288, 271, 62, 204, 149, 190] * 3, 2305, True),
    (33, 6, 6, 2, 128, [0, 2791, 64, 1088, 1408, 1, 200, 130, 129, 128, 384] * 3, 2821, True),
    (40, 20, 8, 4, 128, [0, 1, 127, 128, 129, 300, 5, 0] * 5, 700, False),
    (64, 64, 8, 4, 64, [5, 0, 128, 127] * 16, 2000, False),
    (30, 100, 12, 4, 128, [0, 1, 255, 256, 257, 600] * 5, 2000, True),
]


@pytest.mark.parametrize("case", LONG, ids=[f"b{c[0]}c{c[1]}q{c[2]}h{c[4]}cap{c[6]}" for c in LONG])
def test_attention_over_long_caches(case):
    B, C, Hq, Hkv, hd, lens, cap, causal = case
    g = torch.Generator().manual_seed(cap + C)
    c = filled(g, B, Hkv, cap, hd, lens)
    check_attention(c, rows(g, B, Hq, C, hd), rows(g, B, Hkv, C, hd), rows(g, B, Hkv, C, hd), causal)


@pytest.mark.parametrize("C,hd,cap", [(1, 128, 640), (8, 64, 640), (256, 128, 640), (256, 128, 5000), (30, 128, 5000), (256, 64, 5000),
                                      (1, 128, 5000)])
def test_attention_follows_scales_of_many_octaves(C, hd, cap):
    """Key and value scales that differ by many octaves from block to block, with small queries: the value scale is
    part of the running maximum, the key scale of each block's softmax factor."""
    g = torch.Generator().manual_seed(21)
    lens = [640, 333]
    c = filled(g, 2, 2, cap, hd, lens)
    c.V_exp[:] = torch.randint(100, 150, tuple(c.V_exp.shape), generator=g).to(torch.uint8).cuda()
    c.K_exp[:] = torch.randint(105, 121, tuple(c.K_exp.shape), generator=g).to(torch.uint8).cuda()
    q = rows(g, 2, 4, C, hd)
    check_attention(c, q, rows(g, 2, 2, C, hd) , rows(g, 2, 2, C, hd), False)


@pytest.mark.parametrize("C,hd,cap", [(1, 128, 500), (1, 32, 500), (256, 128, 500), (256, 128, 3000), (40, 128, 3000),
                                      (256, 64, 3000)])
def test_attention_of_peaked_rows(C, hd, cap):
    """Scores of some hundreds: almost all weight on one key, first in one row and last in another."""
    g = torch.Generator().manual_seed(22)
    c = filled(g, 1, 1, cap, hd, [451])
    q = rows(g, 1, 2, C, hd) * 20
    check_attention(c, q.to(torch.bfloat16), rows(g, 1, 1, C, hd), rows(g, 1, 1, C, hd), False)


@pytest.mark.parametrize("C,hd,cap", [(2, 128, 200), (2, 64, 200), (200, 128, 200), (200, 128, 3000), (30, 128, 3000),
                                      (200, 64, 3000)])
def test_attention_scales_queries_exactly(C, hd, cap):
    """Queries of 2^-40 and 2^30, zero rows among them, and one element 2^12 times the others: the power-of-two
    scaling of a row keeps what its scores need."""
    g = torch.Generator().manual_seed(23)
    c = filled(g, 1, 2, cap, hd, [190])
    for f in (2.0 ** -40, 1.0):
        q = rows(g, 1, 4, C, hd) * f
        q[0, 1, 0] = 0
        q[0, 2, 1, 3] *= 2.0 ** 6
        check_attention(c, q, rows(g, 1, 2, C, hd), rows(g, 1, 2, C, hd), False)
    c.K_exp -= 30
    q = rows(g, 1, 4, C, hd) * 2.0 ** 30
    check_attention(c, q, None, None, False)


WIDE = [(1, 128, 400), (1, 128, 5000), (20, 32, 400), (9, 64, 5000), (40, 128, 5000), (256, 128, 5000), (256, 64, 5000)]


@pytest.mark.parametrize("C,hd,cap", WIDE)
def test_attention_over_blocks_of_zeros_and_large_values(C, hd, cap):
    """Values of 2^48 beside blocks of zeros, whose scale is the smallest: 2^104 between the scales, and equal
    weights.  The zeros' probabilities count in full in the row's sum."""
    g = torch.Generator().manual_seed(35)
    c = filled(g, 1, 2, cap, hd, [390])
    for blk in (0, 2, 3, 5):
        c.V[:, :, 64 * blk:min(64 * blk + 64, 390)] = 0
        c.V_exp[:, :, blk] = 63
    for blk in (1, 4):
        c.V_exp[:, :, blk] = 167
    c.V_exp[:, 1, 6] = 63
    q = rows(g, 1, 4, C, hd) * 0.1
    check_attention(c, q, rows(g, 1, 2, C, hd), rows(g, 1, 2, C, hd), False)


@pytest.mark.parametrize("C,hd,cap", WIDE)
def test_attention_reports_values_it_does_not_take(C, hd, cap):
    g = torch.Generator().manual_seed(36)
    q, k, v = rows(g, 1, 4, C, hd).cuda(), rows(g, 1, 2, C, hd).cuda(), rows(g, 1, 2, C, hd).cuda()
    c = filled(g, 1, 2, cap, hd, [390])
    c.V_exp[0, 1, 3] = 168
    dg.kv8_attention(c, q, k, v)
    assert c.status() == dg.DG_ERR_VALUE
    c = filled(g, 1, 2, cap, hd, [390])
    big = v.clone()
    big[0, 1, C - 1, 5] = 448 * 2.0 ** 40
    dg.kv8_attention(c, q, k, big)
    assert c.status() == dg.DG_OK
    big[0, 1, C - 1, 5] = 450 * 2.0 ** 40
    dg.kv8_attention(c, q, k, big)
    assert c.status() == dg.DG_ERR_VALUE


def test_attention_without_any_key_is_zero():
    g = torch.Generator().manual_seed(24)
    for C, hd, cap in ((1, 128, 64), (5, 32, 64), (200, 128, 64), (200, 128, 3000), (20, 128, 3000), (1, 64, 5000)):
        c = filled(g, 2, 1, cap, hd, [0, 0])
        out = torch.full((2 * C, 2 * hd), 9.0, dtype=torch.bfloat16, device="cuda")
        dg.kv8_attention(c, rows(g, 2, 2, C, hd).cuda(), out=out)
        assert torch.count_nonzero(out).item() == 0


def test_attention_writes_its_output_alone():
    """Bytes around the output and behind the workspace keep their values; the cache is read only."""
    g = torch.Generator().manual_seed(25)
    for C, cap in ((1, 400), (70, 400), (1, 5000), (70, 5000), (20, 5000), (1, 40000)):
        c = filled(g, 2, 2, cap, 128, [399, 17])
        before = state(c)
        q, k, v = rows(g, 2, 4, C, 128).cuda(), rows(g, 2, 2, C, 128).cuda(), rows(g, 2, 2, C, 128).cuda()
        need = c.workspace_bytes(C, 4)
        ws = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device="cuda")
        big = torch.full((2 * C + 2, 4 * 128), 3.0, dtype=torch.bfloat16, device="cuda")
        dg.kv8_attention(c, q, k, v, out=big[1:-1], ws=ws[:need])
        torch.cuda.synchronize()
        assert (big[0] == 3).all() and (big[-1] == 3).all() and (ws[need:] == 0x5a).all()
        assert all(torch.equal(x, y) for x, y in zip(before, state(c)))
        assert torch.equal(big[1:-1], dg.kv8_attention(c, q, k, v))


def test_results_repeat_bit_for_bit():
    g = torch.Generator().manual_seed(26)
    for C, cap in ((1, 3000), (256, 3000), (16, 3000), (1, 5000), (1, 40000)):
        c = filled(g, 5, 2, cap, 128, [3000, 1, 0, 1555, 64])
        q, k, v = rows(g, 5, 8, C, 128).cuda(), rows(g, 5, 2, C, 128).cuda(), rows(g, 5, 2, C, 128).cuda()
        first = dg.kv8_attention(c, q, k, v)
        for _ in range(5):
            assert torch.equal(first, dg.kv8_attention(c, q, k, v))


def test_lengths_outside_the_cache_are_reported():
    g = torch.Generator().manual_seed(27)
    c = filled(g, 2, 1, 100, 64, [100, 100])
    c.len[1] = 101
    dg.kv8_attention(c, rows(g, 2, 1, 1, 64).cuda())
    assert c.status() == dg.DG_ERR_CAPACITY
    c.status_word.zero_()
    dg.kv8_read(c, 0, 100)
    assert c.status() == dg.DG_ERR_CAPACITY


def test_calls_that_the_binding_refuses():
    """Wrong types, shapes, strides and workspaces raise before any launch, and write nothing."""
    g = torch.Generator().manual_seed(38)
    c = filled(g, 2, 2, 40000, 64, [100, 7])
    q, k, v = rows(g, 2, 4, 3, 64).cuda(), rows(g, 2, 2, 3, 64).cuda(), rows(g, 2, 2, 3, 64).cuda()
    before = state(c)
    out = torch.full((6, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    need = c.workspace_bytes(3, 4)
    assert need > 0
    ws = torch.zeros(need + 256, dtype=torch.uint8, device="cuda")
    wrong = [dict(q=q.half()), dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(q=q[:, :, :2]), dict(q=q[0]),
             dict(q=q[..., :32]), dict(q=q.cpu()), dict(k=None), dict(v=None), dict(k=k[:1], v=v[:1]),
             dict(k=k.transpose(2, 3).contiguous()), dict(v=v[:, :, :2].contiguous()), dict(out=out[:5]),
             dict(out=out.float()), dict(out=out.cpu()), dict(ws=ws.cpu()), dict(ws=ws[::2])]
    for kw in wrong:
        with pytest.raises(ValueError):
            dg.kv8_attention(c, **dict(dict(q=q, k=k, v=v, out=out), **kw))
    for kw in (dict(ws=ws[:need - 1]), dict(ws=ws[128:128 + need]), dict(q=q[:, :3].contiguous(), out=out[:, :192].contiguous()),
               dict(q=q[:, :, :0], k=k[:, :, :0], v=v[:, :, :0], out=out[:0])):
        with pytest.raises(dg.DgError):
            dg.kv8_attention(c, **dict(dict(q=q, k=k, v=v, out=out), **kw))
    for kw in (dict(k=k.half()), dict(v=v[:, :1]), dict(k=k[..., :32].contiguous()), dict(counts=torch.ones(2).cuda()),
               dict(counts=torch.ones(2, dtype=torch.int32)), dict(counts=torch.ones(3, dtype=torch.int32).cuda())):
        with pytest.raises(ValueError):
            dg.kv8_append(c, **dict(dict(k=k, v=v), **kw))
    big = torch.zeros(2, 2, 9, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(dg.DgError):
        dg.kv8_read(c, 0, 10, out=(big, big.clone()))
    with pytest.raises(dg.DgError):
        dg.kv8_read(c, -1, 5)
    with pytest.raises(ValueError):
        dg.kv8_read(c, 0, 5, out=(big, big.half()))
    dg.kv8_append(c, k[:, :, :0], v[:, :, :0])
    assert dg.kv8_read(c, 5, 0)[0].shape == (2, 2, 0, 64)
    torch.cuda.synchronize()
    assert (out == 5).all() and c.status() == 0 and all(torch.equal(x, y) for x, y in zip(before, state(c)))


def test_offsets_past_32_bits():
    """A cache of 4.7 GB of codes each for K and V, its last head past 2^32 bytes."""
    g = torch.Generator().manual_seed(28)
    B, H, hd, cap = 3, 8, 128, 1_530_000
    assert (B * H - 1) * cap * hd > 2 ** 32
    c = dg.Kv8Cache.empty(B, H, cap, hd)
    k, v = rows(g, B, H, 200, hd), rows(g, B, H, 200, hd)
    dg.kv8_append(c, k.cuda(), v.cuda())
    c.len += 200
    small = dg.Kv8Cache.empty(B, H, 200, hd)
    dg.kv8_append(small, k.cuda(), v.cuda())
    small.len += 200
    assert torch.equal(c.K[:, :, :200], small.K) and torch.equal(c.V[:, :, :200], small.V)
    for x, y in zip(dg.kv8_read(c, 0, 200), dg.kv8_read(small, 0, 200)):
        assert torch.equal(x, y)
    for C in (1, 64):
        q = rows(g, B, 2 * H, C, hd).cuda()
        assert torch.equal(dg.kv8_attention(c, q), dg.kv8_attention(small, q))


# ----------------------------------------------------- streams and graphs ----
def test_on_another_stream():
    g = torch.Generator().manual_seed(31)
    c = filled(g, 2, 2, 300, 128, [200, 77])
    q, k, v = rows(g, 2, 4, 9, 128).cuda(), rows(g, 2, 2, 9, 128).cuda(), rows(g, 2, 2, 9, 128).cuda()
    want = dg.kv8_attention(c, q, k, v)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = dg.kv8_attention(c, q, k, v, stream=st)
    dg.kv8_append(c, k, v, stream=st)
    K, V = dg.kv8_read(c, 0, 300, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    K2, V2 = dg.kv8_read(c, 0, 300)
    assert torch.equal(K, K2) and torch.equal(V, V2)


def test_calls_on_two_streams_at_once():
    """The workspaces that the cache keeps by itself are a stream's own: calls of one cache that overlap on the GPU,
    of sizes that grow the workspace in between, give what they give alone."""
    g = torch.Generator().manual_seed(37)
    c = filled(g, 4, 2, 40000, 128, [9000, 1, 4000, 8111])
    sizes = (1, 40, 3, 256)
    x = {C: [rows(g, 4, h, C, 128).cuda() for h in (8, 2, 2)] for C in sizes}
    want = {C: dg.kv8_attention(c, *x[C]) for C in sizes}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(10):
        for j, st in enumerate(streams):
            C = sizes[(i + 2 * j) % 4]
            got.append((C, dg.kv8_attention(c, *x[C], stream=st)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[C]) for C, o in got)
    # two graphs, each with a workspace from its own pool, replayed side by side
    graphs = []
    for C in (40, 1):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = dg.kv8_attention(c, *x[C])
        graphs.append((C, gr, o))
    for _ in range(5):
        for _, _, o in graphs:
            o.zero_()
        torch.cuda.synchronize()
        for st, (_, gr, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[C]) for C, _, o in graphs)


def test_captured_decoding_follows_the_growing_cache():
    """One token of two layers captured once and replayed 80 times: append and attention read the lengths on the
    device, so the replays cross block borders and grow scales as eager calls do."""
    g = torch.Generator().manual_seed(32)
    B, Hq, Hkv, hd, steps, cap = 3, 4, 2, 128, 80, 200
    start = [0, 60, 101]
    eager = [filled(g, B, Hkv, cap, hd, start) for _ in range(2)]
    ln = eager[0].len
    eager = [dg.Kv8Cache(c.K, c.V, c.K_exp, c.V_exp, ln) for c in eager]
    ln2 = ln.clone()
    graph_c = [dg.Kv8Cache(c.K.clone(), c.V.clone(), c.K_exp.clone(), c.V_exp.clone(), ln2) for c in eager]
    data = [[rows(g, B, h, steps, hd).cuda() for h in (Hq, Hkv, Hkv)] for _ in range(2)]

    def token(caches, x):
        out = []
        for c, (q, k, v) in zip(caches, x):
            out.append(dg.kv8_attention(c, q, k, v))
            dg.kv8_append(c, k, v)
        caches[0].len.add_(1)
        return out

    def at(i):
        return [[t[:, :, i:i + 1].contiguous() for t in layer] for layer in data]

    static = at(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = [[t.clone() for t in (c.K, c.V, c.K_exp, c.V_exp)] for c in graph_c]
    with torch.cuda.stream(side):
        token(graph_c, static)
    torch.cuda.current_stream().wait_stream(side)
    ln2.copy_(ln)
    for c, saved in zip(graph_c, keep):
        for t, s in zip((c.K, c.V, c.K_exp, c.V_exp), saved):
            t.copy_(s)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        outs = token(graph_c, static)
    for i in range(steps):
        x = at(i)
        want = token(eager, x)
        for s, t in zip(static, x):
            for a, b in zip(s, t):
                a.copy_(b)
        gr.replay()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), i
    for a, b in zip(graph_c, eager):
        assert all(torch.equal(x, y) for x, y in zip(state(a), state(b)))
        assert a.status() == b.status() == 0


def test_assigned_lengths_reach_the_calls():
    """cache.len = .. writes into the tensor whose address the calls hold."""
    g = torch.Generator().manual_seed(34)
    c = filled(g, 2, 1, 200, 64, [150, 70])
    q = rows(g, 2, 1, 1, 64)
    c.len = c.len - 50
    assert c.len.tolist() == [100, 20]
    check_attention(c, q, None, None, False)
    c.len = torch.tensor([3, 150], dtype=torch.int32)
    assert c.s.len == c.len.data_ptr()
    K, V = dg.kv8_read(c, 0, 200)
    assert torch.count_nonzero(K[0, :, 3:]).item() == 0


def test_two_graphs_in_a_row_share_a_workspace():
    g = torch.Generator().manual_seed(33)
    c1, c2 = filled(g, 2, 2, 40000, 128, [900, 3]), filled(g, 2, 2, 9000, 128, [0, 499])
    assert c1.workspace_bytes(1, 8) > 0 and c2.workspace_bytes(64, 8) > 0
    q = [rows(g, 2, 8, C, 128).cuda() for C in (1, 64)]
    ws = torch.empty(max(c1.workspace_bytes(1, 8), c2.workspace_bytes(64, 8)), dtype=torch.uint8, device="cuda")
    want = [dg.kv8_attention(c1, q[0]), dg.kv8_attention(c2, q[1])]
    graphs, outs = [], []
    for c, x in ((c1, q[0]), (c2, q[1])):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(dg.kv8_attention(c, x, ws=ws))
        graphs.append(gr)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for gr in graphs:
            gr.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


# ---------------------------------------------------------------- together ----
def test_prompt_blocks_and_tokens_together():
    """A prompt in causal pieces, a canvas over it, its commit, then single tokens, ragged throughout: each call's
    output is the attention over the rows read back so far and the new tokens' own keys and values."""
    g = torch.Generator().manual_seed(41)
    B, Hq, Hkv, hd = 3, 8, 2, 128
    c = dg.Kv8Cache.empty(B, Hkv, 700, hd)
    for C, causal, counts in ((130, True, [130, 7, 64]), (64, False, None), (130, True, [1, 130, 0]), (1, True, None),
                              (1, True, None), (16, False, [16, 0, 3])):
        q, k, v = rows(g, B, Hq, C, hd), rows(g, B, Hkv, C, hd), rows(g, B, Hkv, C, hd)
        check_attention(c, q, k, v, causal)
        check_append(c, k, v, counts)
        c.len += C if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    assert c.len.tolist() == [130 + 64 + 1 + 2 + 16, 7 + 64 + 130 + 2, 64 + 64 + 2 + 3]


def test_step_queries_over_the_model_cache_in_8_bits():
    """The denoising step's own q, k, v over its prefix cache quantised: equal to the step's attention
    (attention_noalloc) over the values read back into the model's bf16 cache."""
    dims, seed = synth.workload("step_v32k_c256_p2k")
    w = synth.make_weights(dims, seed, device="cuda")
    model = dg.Model(dims, w)
    canvas = dg.Canvas(*synth.make_canvas(dims, seed, device="cuda"))
    d = dg.denoise_step(model, canvas, tau=0.8, b=0.1, seed=seed, step=0, debug=True)["debug"]
    c = dg.Kv8Cache.empty(dims.B, dims.Hkv, model.cap, dims.hd)
    dg.kv8_append(c, model.K, model.V)
    c.len += dims.P
    dg.kv8_read(c, 0, dims.P, out=(model.K, model.V))
    want = dg.attention_noalloc(d["q"], model.K, model.V, dims.P, d["k"], d["v"])
    check_attention(c, d["q"].cpu(), d["k"].cpu(), d["v"].cpu(), False)
    got = dg.kv8_attention(c, d["q"], d["k"], d["v"])
    # both are within 2^-8 of the output (bf16) and 2^-11 of sum p |v| of the same real values
    A = (want.float().abs() * 2.0 ** -7 + 2.0 ** -10 * 4.0).double()
    assert ((got.double() - want.double()).abs() <= A).all()
