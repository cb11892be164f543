"""4-bit matrices through the public entry points: quantisation and read-back bit for bit, products against their
definition in 64 bits with the tolerance derived in w4_ref.product."""
import pytest
import torch

import w4_ref
from block_diffusion_text_gb300 import dg

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def drawn(g, N, K, group, codes=(0, 16)):
    c = torch.randint(codes[0], codes[1], (N, K), generator=g, dtype=torch.uint8)
    s = (torch.randn(N, K // group, generator=g) * 0.05).to(BF)
    return c, s


def check(w, c, s, x, out=None, dtype=BF, alpha=None, resid=None, **kw):
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    y = dg.w4_matvec(w, x if x.is_cuda else x.cuda(), alpha=cu(alpha), resid=cu(resid), dtype=dtype, out=out, **kw)
    want, tol = w4_ref.product(c, s, x.cpu(), alpha, kw.get("coef", 1.0), resid, y.dtype)
    err = (y.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    return y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 128), (16, 256), (17, 128), (100, 640), (33, 2816)])
def test_quantise_and_read_are_exact(N, K, group):
    g = torch.Generator().manual_seed(N + group)
    W = (torch.randn(N, K, generator=g) * torch.exp2(torch.randint(-30, 30, (N, 1), generator=g).float())).to(BF)
    W[0, :group] = 0
    W[-1, -1] = 3e38
    c, s = w4_ref.quantize(W, group)
    assert torch.equal(dg.w4_quantize(W.cuda(), group).read().cpu().double(), w4_ref.weights(c, s))
    # a matrix inside a wider one
    wide = torch.full((N, K + 24), float("nan"), dtype=BF)
    wide[:, :K] = W
    assert torch.equal(dg.w4_quantize(wide.cuda()[:, :K], group).read().cpu().double(), w4_ref.weights(c, s))
    c, s = drawn(g, N, K, group)
    assert torch.equal(dg.W4Matrix.from_codes(c.cuda(), s.cuda()).read().cpu().double(), w4_ref.weights(c, s))


def test_quantise_tiny_and_non_finite():
    W = torch.zeros(4, 64, dtype=BF)
    W[0, 3], W[0, 5] = 1e-39, -1e-39            # subnormal, with a subnormal scale
    W[1, 7], W[1, 8], W[1, 9], W[1, 10] = float("inf"), float("-inf"), float("nan"), 1.0
    W[2, :] = float("nan")
    c, s = w4_ref.quantize(W, 64)
    with pytest.raises(dg.DgError) as e:
        dg.w4_quantize(W.cuda())
    assert e.value.code == dg.DG_ERR_VALUE
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = dg.w4_quantize(W.cuda(), status=word)
    assert int(word) == dg.DG_ERR_VALUE
    assert torch.equal(w.read().cpu().double(), w4_ref.weights(c, s))
    assert c[1, 7] == 15 and c[1, 8] == 1 and c[1, 9] == 8 and c[1, 10] == 15


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 24, 25, 32])
@pytest.mark.parametrize("N,K,group", [(1, 64, 64), (15, 64, 32), (257, 128, 128), (100, 192, 64), (1000, 1088, 32),
                                       (6000, 2816, 64), (40000, 256, 128)])
def test_products(M, N, K, group):
    g = torch.Generator().manual_seed(M * 7 + N)
    c, s = drawn(g, N, K, group)
    w = dg.W4Matrix.from_codes(c.cuda(), s.cuda())
    x = (torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(BF)
    check(w, c, s, x)
    check(w, c, s, x, dtype=torch.float32, alpha=torch.rand(M, generator=g) * 9 - 3, coef=0.37)
    check(w, c, s, x, resid=torch.randn(M, N, generator=g).to(BF))


@pytest.mark.parametrize("M", [3, 32])
def test_pitches_and_what_lies_between(M):
    """Rows of x, the residual and y inside wider tensors whose other elements are NaN, or stay as they were."""
    g = torch.Generator().manual_seed(M)
    N, K = 77, 320
    c, s = drawn(g, N, K, 32)
    w = dg.W4Matrix.from_codes(c.cuda(), s.cuda())
    x = torch.full((M, K + 40), float("nan"), dtype=BF, device="cuda")
    x[:, 8:8 + K] = torch.randn(M, K, generator=g).to(BF).cuda()
    r = torch.full((M, N + 5), float("nan"), dtype=BF)
    r[:, 3:3 + N] = torch.randn(M, N, generator=g).to(BF)
    for dt in (BF, torch.float32):
        y = torch.full((M + 2, N + 9), 5.0, dtype=dt, device="cuda")
        check(w, c, s, x[:, 8:8 + K], out=y[1:1 + M, 2:2 + N])
        check(w, c, s, x[:, 8:8 + K], out=y[1:1 + M, 2:2 + N], resid=r[:, 3:3 + N])
        y[1:1 + M, 2:2 + N] = 5.0
        assert bool((y == 5.0).all())


def test_residual_in_place():
    g = torch.Generator().manual_seed(1)
    c, s = drawn(g, 200, 128, 64)
    w = dg.W4Matrix.from_codes(c.cuda(), s.cuda())
    x, r = torch.randn(5, 128, generator=g).to(BF), torch.randn(5, 200, generator=g).to(BF)
    want, rc = dg.w4_matvec(w, x.cuda(), resid=r.cuda()), r.cuda()
    dg.w4_matvec(w, x.cuda(), resid=rc, out=rc)
    assert torch.equal(rc, want)


def test_rows_do_not_touch_each_other():
    """A row of infinities or NaN leaves the others' bits, and so does the number of rows."""
    g = torch.Generator().manual_seed(2)
    c, s = drawn(g, 333, 640, 64)
    w = dg.W4Matrix.from_codes(c.cuda(), s.cuda())
    x = torch.randn(8, 640, generator=g).to(BF).cuda()
    want = dg.w4_matvec(w, x)
    for bad in (float("nan"), float("inf")):
        z = x.clone()
        z[3] = bad
        y = dg.w4_matvec(w, z)
        keep = [0, 1, 2, 4, 5, 6, 7]
        assert torch.equal(y[keep], want[keep]) and not bool(y[3].isfinite().any())
    assert torch.equal(dg.w4_matvec(w, x[:3]), want[:3])


def test_large_and_small_values():
    """Sums near the ends of fp32 keep their relative error: the scales come last."""
    g = torch.Generator().manual_seed(3)
    c = torch.randint(0, 16, (64, 256), generator=g, dtype=torch.uint8)
    for e in (-100, 60):
        s = torch.full((64, 4), 2.0 ** e, dtype=BF)
        w = dg.W4Matrix.from_codes(c.cuda(), s.cuda())
        check(w, c, s, torch.randn(4, 256, generator=g).to(BF), dtype=torch.float32)


def test_streams_and_graphs():
    g = torch.Generator().manual_seed(4)
    c, s = drawn(g, 5000, 512, 64)
    w = dg.W4Matrix.from_codes(c.cuda(), s.cuda())
    x = torch.randn(2, 512, generator=g).to(BF).cuda()
    want = dg.w4_matvec(w, x)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y = dg.w4_matvec(w, x, stream=st)
    st.synchronize()
    assert torch.equal(y, want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y = dg.w4_matvec(w, x)
    x2 = torch.randn(2, 512, generator=g).to(BF).cuda()
    want2 = dg.w4_matvec(w, x2)
    for src, ref in ((x2.clone(), want2), (x.clone(), want)):
        x.copy_(src)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)


def test_binding_refusals():
    c, s = drawn(torch.Generator().manual_seed(5), 32, 128, 64)
    w = dg.W4Matrix.from_codes(c.cuda(), s.cuda())
    x = torch.zeros(2, 128, dtype=BF, device="cuda")
    bad = [dict(x=x.float()), dict(x=x.cpu()), dict(x=x[0]), dict(x=x[:, :64]), dict(x=x.T.contiguous().T),
           dict(alpha=torch.ones(3, device="cuda")), dict(alpha=torch.ones(2, dtype=BF, device="cuda")),
           dict(resid=torch.zeros(1, 32, dtype=BF, device="cuda")), dict(resid=torch.zeros(2, 32, device="cuda")),
           dict(out=torch.zeros(2, 31, device="cuda")), dict(out=torch.zeros(2, 32, dtype=torch.float16, device="cuda")),
           dict(dtype=torch.float16)]
    for kw in bad:
        with pytest.raises(ValueError):
            dg.w4_matvec(w, **dict(dict(x=x), **kw))
    with pytest.raises(dg.DgError):
        dg.w4_matvec(w, torch.zeros(33, 128, dtype=BF, device="cuda"))
    with pytest.raises(dg.DgError):   # a pitch that breaks the 16-byte rule
        dg.w4_matvec(w, torch.zeros(2, 132, dtype=BF, device="cuda")[:, :128])
    with pytest.raises(dg.DgError):
        dg.W4Matrix.from_codes(c.cuda(), s[:, :1].contiguous().cuda().repeat(1, 8))
    with pytest.raises(ValueError):
        dg.W4Matrix.from_codes(c.cuda()[:, ::2], s.cuda())


@pytest.mark.parametrize("M", [9, 16, 17, 32])
@pytest.mark.parametrize("N,K,group", [(38912, 64, 64), (40007, 192, 32), (45000, 640, 128), (60000, 320, 64), (39000, 1088, 32)])
def test_products_of_many_rows(M, N, K, group):
    """The kernel that keeps x in shared memory: row tiles that do not divide, columns that end inside a chunk."""
    g = torch.Generator().manual_seed(M + N)
    c, s = drawn(g, N, K, group)
    w = dg.W4Matrix.from_codes(c.cuda(), s.cuda())
    x = torch.randn(M, K, generator=g).to(BF)
    check(w, c, s, x, dtype=torch.float32, alpha=torch.rand(M, generator=g) + 0.5)
    check(w, c, s, x, resid=torch.randn(M, N, generator=g).to(BF))


@pytest.mark.parametrize("M", [1, 5, 8, 9, 32])
@pytest.mark.parametrize("N,K,group", [(9712, 320, 64), (9713, 128, 128), (9729, 192, 32), (14600, 64, 64), (29168, 128, 64), (29169, 192, 32),
                                       (29200, 384, 128)])
def test_products_where_the_kernels_change(M, N, K, group):
    g = torch.Generator().manual_seed(M + N)
    c, s = drawn(g, N, K, group)
    w = dg.W4Matrix.from_codes(c.cuda(), s.cuda())
    check(w, c, s, torch.randn(M, K, generator=g).to(BF), dtype=torch.float32)


@pytest.mark.parametrize("M,group", [(8, 64), (12, 64), (32, 128), (32, 32)])
def test_long_products_side_by_side(M, group):
    """Two streams and a captured product at once over the same long matrix: the same bits as alone."""
    g = torch.Generator().manual_seed(M + group)
    N, K = 39001, 384
    c, s = drawn(g, N, K, group)
    w = dg.W4Matrix.from_codes(c.cuda(), s.cuda())
    xs = [torch.randn(M, K, generator=g).to(BF).cuda() for _ in range(3)]
    want = [check(w, c, s, x, dtype=torch.float32) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    out = [torch.zeros(M, N, device="cuda") for _ in xs]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=streams[2]):
        dg.w4_matvec(w, xs[2], out=out[2], dtype=torch.float32)
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                dg.w4_matvec(w, xs[i], out=out[i], dtype=torch.float32)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert dg.w4_status() == 0


@pytest.mark.parametrize("M,group", [(3, 64), (20, 32), (32, 128)])
def test_codes_past_32_bits(M, group):
    """A matrix of more than 2^32 codes (2^31 bytes): its rows at both ends and about the border."""
    g = torch.Generator(device="cuda").manual_seed(M)
    N, K = 2 ** 19 + 40, 8320
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    codes = torch.stack((codes & 15, codes >> 4), dim=2).view(N, K)
    scales = (torch.randn(N, K // group, generator=g, device="cuda") * 0.05).to(BF)
    w = dg.W4Matrix.from_codes(codes, scales)
    assert w.codes.numel() > 2 ** 31
    x = torch.randn(M, K, generator=g, device="cuda").to(BF)
    y = dg.w4_matvec(w, x, dtype=torch.float32)
    border = 2 ** 32 // K
    rows = torch.cat([torch.arange(a, a + 40) for a in (0, border - 20, N - 40)])
    want, tol = w4_ref.product(codes[rows.cuda()].cpu(), scales[rows.cuda()].cpu(), x.cpu(), None, 1.0, None, torch.float32)
    err = (y[:, rows.cuda()].double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
