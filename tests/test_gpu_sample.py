"""Sampling through the public entry point against its definition in 64 bits (sample_ref: what is undecided at a
border is derived there)."""
import itertools

import pytest
import torch

import sample_ref
from block_diffusion_text_gb300 import dg

pytestmark = pytest.mark.gpu
INF = float("inf")


def check(x, u, T=1.0, k=0, p=1.0, mp=0.0, **kw):
    """x [R, V] on the CPU; settings numbers or tensors [R]."""
    dev = lambda v: v.cuda() if isinstance(v, torch.Tensor) else v  # noqa: E731
    tok, lp, kept = (t.cpu() for t in dg.sample(x.cuda(), u.cuda(), temperature=dev(T), top_k=dev(k), top_p=dev(p),
                                                min_p=dev(mp), **kw))
    f32 = lambda v, r: float(v[r]) if isinstance(v, torch.Tensor) else float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    for r in range(x.shape[0]):
        kr = int(k[r]) if isinstance(k, torch.Tensor) else k
        why = sample_ref.check_row(x[r].float(), float(u[r]), f32(T, r), kr, f32(p, r), f32(mp, r), int(tok[r]), float(lp[r]),
                                   int(kept[r]))
        assert why is None, (r, why, f32(T, r), kr, f32(p, r), f32(mp, r))
    return tok, lp, kept


def settings(g, R):
    """Every combination of cuts, in turn."""
    on = torch.tensor(list(itertools.islice(itertools.cycle(itertools.product([0, 1], repeat=3)), R)), dtype=torch.bool)
    k = torch.where(on[:, 0], (2 ** (10 * torch.rand(R, generator=g))).int(), 0).int()
    p = torch.where(on[:, 1], torch.rand(R, generator=g), 1.0)
    mp = torch.where(on[:, 2], torch.rand(R, generator=g) ** 3, 0.0)
    return 0.3 + torch.rand(R, generator=g), k, p, mp


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 3, 31, 512, 4096, 4097, 16385, 32769, 50257, 262144])
def test_all_cuts(V, dtype):
    g = torch.Generator().manual_seed(V)
    R = 24 if V < 100000 else 16
    x = torch.randn(R, V, generator=g) * torch.exp(2 * torch.rand(R, 1, generator=g) - 0.7)
    T, k, p, mp = settings(g, R)
    check(x.to(dtype), torch.rand(R, generator=g), T, k, p, mp)


@pytest.mark.parametrize("V", [7, 1000, 40000])
def test_ties_go_to_the_lowest_index(V):
    """Logits of a few values: cuts inside runs of equal ones."""
    g = torch.Generator().manual_seed(V)
    R = 32
    x = torch.randint(-2, 3, (R, V), generator=g).float() * 0.5
    T, k, p, mp = settings(g, R)
    check(x, torch.rand(R, generator=g), T, k, p, mp)
    # all equal: top_k = n keeps the first n, top_p = q the first ceil(q V)
    u = torch.rand(4, generator=g)
    for k in (1, 2, V // 2 + 1, V, V + 5):
        tok, _, kept = check(torch.full((4, V), -3.25), u, k=k)
        assert kept.tolist() == [min(k, V)] * 4 and bool((tok < k).all())
    for q in (0.0, 0.25, 0.5, 0.75):
        tok, _, kept = check(torch.full((4, V), 2.0), u, p=q)
        assert kept.tolist() == [max(1, -(-int(4 * q * V) // 4) if (4 * q * V) % 4 == 0 else int(q * V) + 1)] * 4


def test_ends_of_u():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 3001, generator=g)
    x[:, 0] = x[:, -1] = -INF
    u = torch.tensor([0.0, 1 - 2.0 ** -24] * 3)
    tok, *_ = check(x, u)
    assert tok[:2].tolist() == [1, 2999]
    check(x, u, k=5)
    check(x, u, p=0.9)


def test_banned_tokens_and_lowest_values():
    """-inf is never kept; the type's lowest value is a value: alone it is drawn."""
    g = torch.Generator().manual_seed(2)
    V = 5000
    x = torch.full((8, V), -INF)
    x[0, 77] = -5.0
    x[1, [3, 4000]] = torch.tensor([1.0, 2.0])
    x[2] = -sample_ref.FMAX
    x[3, 5:9] = -sample_ref.FMAX
    x[4] = -sample_ref.FMAX
    x[4, 100] = 0.0
    x[5, ::2] = torch.randn(V // 2, generator=g)
    x[6] = sample_ref.FMAX
    x[7, 9], x[7, 10] = sample_ref.FMAX, -sample_ref.FMAX
    u = torch.rand(8, generator=g)
    tok, _, kept = check(x, u)
    assert int(tok[0]) == 77 and kept.tolist() == [1, 2, V, 4, V, V // 2, V, 2]
    check(x, u, k=3)
    check(x, u, p=0.7)
    check(x, u, T=0.01, mp=0.5)
    check(x.to(torch.bfloat16).masked_fill(x < -1e38, -3.3895e38), u, k=3, p=0.5)


def test_large_logits_and_extreme_temperatures():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(10, 2000, generator=g)
    x[1] += 1e4
    x[2] *= 1e6
    x[3] -= 3e5
    x[4] = x[4] * 1e30
    x[5] = x[5] * 1e-30
    x[6] = x[6] * 1e-42
    x[7] = torch.linspace(0, 300, 2000)
    u = torch.rand(10, generator=g)
    for T in (1.0, 1e-3, 1e-12, 2.0 ** -64, 1e-25, 0.0, 50.0, 1e20, 3e38):
        check(x, u, T=T)
        check(x, u, T=T, p=0.8, mp=1e-4)
        check(x, u, T=T, k=40, p=0.9)


def test_negative_zero_is_zero():
    x = torch.tensor([[-0.0, 0.0, -0.0, 0.0], [-0.0, -0.0, -0.0, -0.0], [-1.0, -0.0, 0.0, -2.0], [-0.0, -1.0, -1.0, -1.0]])
    u = torch.tensor([0.99, 0.6, 0.5, 0.1])
    for kw in (dict(T=0.0), dict(k=1), dict(k=2), dict(p=0.5), dict(mp=1.0), dict(k=3, p=0.6), dict(mp=0.5)):
        check(x, u, **kw)


def test_rows_that_cannot_be_drawn_from():
    x = torch.zeros(12, 600)
    x[0, 5] = float("nan")
    x[1, 599] = INF
    x[2] = -INF
    T, p, mp, u = torch.ones(12), torch.ones(12), torch.zeros(12), torch.full((12,), 0.5)
    k = torch.zeros(12, dtype=torch.int32)
    T[3], T[4], p[5], mp[6], mp[7], u[8], u[9], k[10] = -1.0, float("nan"), -0.1, -1.0, 1.5, 1.0, float("nan"), -2
    tok, lp, kept = check(x, u, T, k, p, mp)
    assert tok.tolist()[:11] == [-1] * 11 and int(tok[11]) == 300


def test_pitch_out_and_optional_outputs():
    g = torch.Generator().manual_seed(4)
    for dt in (torch.float32, torch.bfloat16):
        wide = torch.full((5, 1100), float("nan"), dtype=dt)
        wide[:, 3:1004] = torch.randn(5, 1001, generator=g).to(dt)
        u = torch.rand(5, generator=g)
        want = check(wide[:, 3:1004].clone(), u, k=9, p=0.8)
        out = tuple(torch.zeros(5, dtype=t, device="cuda") for t in (torch.int32, torch.float32, torch.int32))
        w = wide.cuda()
        got = dg.sample(w[:, 3:1004], u.cuda(), top_k=9, top_p=0.8, out=out)
        assert got is out and all(torch.equal(a.cpu(), b) for a, b in zip(out, want))
    how = dg.dg_sampling(temperature_all=1.0, top_p_all=0.8, top_k_all=9)
    tok, uc = torch.zeros(5, dtype=torch.int32, device="cuda"), u.cuda()
    rc = dg.load().dg_sample(w[:, 3:].data_ptr(), 1, 1100, 5, 1001, dg.ct.byref(how), uc.data_ptr(), tok.data_ptr(), None, None,
                             torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(tok.cpu(), want[0])


@pytest.mark.parametrize("R,period", [(1, 4), (3, 4), (40, 8)])
@pytest.mark.parametrize("high", [0, 1])
def test_logits_whose_sample_misleads(R, period, high):
    """Every period-th 128 values are higher: the ones that a sample of every period-th sees, or ones that it does not.
    The cuts lie among either, above and below min_p's floor."""
    g = torch.Generator().manual_seed(10 * R + high)
    V = 262144
    x = 0.3 * torch.randn(R, V, generator=g) + 4.0 * (torch.arange(V) // 128 % period == high)
    u = torch.rand(R, generator=g)
    p = 0.3 + 0.69 * torch.arange(R).float() / R if R > 3 else torch.tensor([0.95, 0.6, 0.3])[:R]
    floors = torch.tensor([0.0, 2.0 ** -9, 0.01, 0.1, 0.5])
    for n in range(5 if R <= 3 else 2):
        mp = floors[(torch.arange(R) + n) % 5]
        check(x, u, p=p, mp=mp)
    check(x.to(torch.bfloat16), u, p=p, mp=2.0 ** -9)


def test_many_long_rows():
    """More rows than run at once, from flat to sharp, cut by top_p and min_p."""
    g = torch.Generator().manual_seed(5)
    R, V = 80, 262144
    x = torch.randn(R, V, generator=g) * torch.exp(2.4 * torch.rand(R, 1, generator=g) - 0.7)
    check(x, torch.rand(R, generator=g), p=0.5 + 0.499 * torch.rand(R, generator=g),
          mp=torch.where(torch.arange(R) % 2 == 0, 0.0, 0.05 * torch.rand(R, generator=g) ** 2))


def test_longest_vocabulary():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(3, 1 << 20, generator=g)
    u = torch.rand(3, generator=g)
    check(x, u)
    check(x, u, p=0.9)
    check(x, u, k=100000, mp=1e-3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_past_32_bits_apart(dtype):
    g = torch.Generator().manual_seed(12)
    R, V, ld = 3, 9001, 2 ** 31 + 8
    x = (torch.randn(R, V, generator=g) * 2).to(dtype)
    u = torch.rand(R, generator=g)
    wide = torch.empty((R - 1) * ld + V, dtype=dtype, device="cuda").as_strided((R, V), (ld, 1))
    wide.copy_(x)
    for kw in (dict(top_p=0.9), dict(top_k=30), dict(min_p=0.01)):
        got, want = dg.sample(wide, u.cuda(), **kw), dg.sample(x.cuda(), u.cuda(), **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_top_k_of_any_size_as_a_number():
    g = torch.Generator().manual_seed(13)
    x, u = torch.randn(4, 300, generator=g).cuda(), torch.rand(4, generator=g).cuda()
    want = dg.sample(x, u)
    for k in (300, 301, 2 ** 31, 2 ** 32 + 1, 10 ** 30):
        assert all(torch.equal(a, b) for a, b in zip(dg.sample(x, u, top_k=k), want))
    for k in (-1, -2 ** 32 + 1):
        assert dg.sample(x, u, top_k=k)[0].tolist() == [-1] * 4


def test_shares_follow_the_weights():
    """The whole range of u in equal steps draws each token as often as its weight says, to a step at either end."""
    x = torch.tensor([0.3, -1.0, 2.0, -INF, 0.9, 2.0])
    n = 4096
    u = (torch.arange(n) + 0.5) / n
    tok, *_ = dg.sample(x.expand(n, 6).contiguous().cuda(), u.cuda(), temperature=0.7)
    share = torch.bincount(tok.cpu(), minlength=6) / n
    assert bool(((share - torch.softmax(x / 0.7, 0)).abs() <= 2 / n).all())
    assert bool((tok[1:] >= tok[:-1]).all())


@pytest.mark.parametrize("T", [1.0, 0.37])
def test_logprob_of_nearly_certain_tokens(T):
    """Relative to itself: the others' weights are off by 2^-28 and a unit, 2^-41 of the largest at most, each; the result
    by 2^-24."""
    d = torch.tensor([0.0, 1.0, 3.0, 6.0, 9.0, 12.0, 40.0])
    x = torch.full((len(d), 7), -1e4)
    x[:, 3], x[:, 5], x[:, 6] = 20.0, 20.0 - d, 19.5 - d
    tok, lp, kept = (t.cpu() for t in dg.sample(x.cuda(), torch.full((len(d),), 1e-6, device="cuda"), temperature=T))
    tk = float(torch.tensor(T, dtype=torch.float32))
    rest = torch.exp((x[:, 5:].double() - 20.0) / tk).sum(1)
    want = -torch.log1p(rest)
    assert tok.tolist() == [3] * len(d)
    assert bool(((lp.double() - want).abs() <= -want * (2.0 ** -24 + 2.0 ** -27) + 2 * 2.0 ** -41).all()), (lp, want)
    tok, lp, kept = (t.cpu() for t in dg.sample(x.cuda(), torch.full((len(d),), 0.3, device="cuda"), temperature=T, top_p=1e-3))
    assert kept.tolist() == [1] * len(d) and tok.tolist() == [3] * len(d) and bool((lp == 0).all())


def test_streams_graphs_and_the_same_bits():
    g = torch.Generator().manual_seed(6)
    x = torch.randn(40, 70000, generator=g).cuda()
    u = torch.rand(40, generator=g).cuda()
    kw = dict(temperature=0.8, top_k=0, top_p=0.95, min_p=1e-4)
    want = dg.sample(x, u, **kw)
    torch.cuda.synchronize()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(dg.sample(x, u, **kw), want))
    st = torch.cuda.Stream()
    got = dg.sample(x, u, stream=st, **kw)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = dg.sample(x, u, **kw)
    u2 = torch.rand(40, generator=g).cuda()
    want2 = dg.sample(x, u2, **kw)
    for src, ref in ((u2, want2), (u.clone(), want)):
        u.copy_(src)
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_binding_refusals():
    x, u = torch.zeros(3, 50, device="cuda"), torch.zeros(3, device="cuda")
    i32 = torch.zeros(3, dtype=torch.int32, device="cuda")
    for kw in (dict(logits=x.half()), dict(logits=x[0]), dict(logits=x.T.contiguous().T), dict(u=u[:2]), dict(u=u.double()),
               dict(u=u.cpu()), dict(top_k=u), dict(temperature=i32), dict(top_p=u[:1]), dict(min_p=u.cpu()),
               dict(out=(i32, i32, i32)), dict(out=(i32[:2], u, i32))):
        with pytest.raises(ValueError):
            dg.sample(**dict(dict(logits=x, u=u), **kw))
    assert [t.shape[0] for t in dg.sample(x[:0], u[:0])] == [0, 0, 0]
    with pytest.raises(dg.DgError):
        dg.sample(x[:, :0], u)
