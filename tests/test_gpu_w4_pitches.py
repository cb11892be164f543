"""Rows of the 4-bit products' operands further apart than 32 bits count (elements)."""
import pytest
import torch

import w4_ref
from test_gpu_w4 import BF, check, drawn
from block_diffusion_text_gb300 import dg

pytestmark = pytest.mark.gpu


def apart(t, pitch):
    """The rows of t on the GPU, `pitch` elements from one to the next."""
    M, K = t.shape
    wide = torch.empty((M - 1) * pitch + K, dtype=t.dtype, device="cuda").as_strided((M, K), (pitch, 1))
    wide.copy_(t)
    return wide


# a pitch that is K or N modulo 2^32 would pass for the packed one; nine rows over a long matrix take the kernel with x
# in shared memory
@pytest.mark.parametrize("M,N,over", [(2, 77, 1 << 32), (2, 9729, 1 << 32), (9, 29185, 1 << 31), (3, 77, 1 << 31)])
def test_products_of_rows_far_apart(M, N, over):
    g = torch.Generator().manual_seed(M + N)
    K = 192
    c, s = drawn(g, N, K, 64)
    w = dg.W4Matrix.from_codes(c.cuda(), s.cuda())
    x, r = torch.randn(M, K, generator=g).to(BF), torch.randn(M, N, generator=g).to(BF)
    want = check(w, c, s, x, dtype=torch.float32)
    assert torch.equal(dg.w4_matvec(w, apart(x, over + K), dtype=torch.float32), want)
    want = check(w, c, s, x, resid=r)
    assert torch.equal(dg.w4_matvec(w, x.cuda(), resid=apart(r, over + N)), want)
    if M < 9:
        y = apart(torch.zeros(M, N, dtype=BF), over + N)
        assert dg.w4_matvec(w, x.cuda(), resid=r.cuda(), out=y) is y and torch.equal(y, want)
        y = apart(r, over + N)
        assert torch.equal(dg.w4_matvec(w, x.cuda(), resid=y, out=y), want)


@pytest.mark.parametrize("over", [1 << 31, 1 << 32])
def test_quantises_rows_far_apart(over):
    W = torch.randn(3, 256, generator=torch.Generator().manual_seed(1)).to(BF)
    far = apart(W, over + 256)
    assert torch.equal(dg.w4_quantize(far, 64).read().cpu().double(), w4_ref.weights(*w4_ref.quantize(W, 64)))


def test_reads_to_rows_far_apart():
    g = torch.Generator().manual_seed(2)
    c, s = drawn(g, 2, 128, 64)
    w = dg.W4Matrix.from_codes(c.cuda(), s.cuda())
    out = apart(torch.zeros(2, 128), (1 << 32) + 128)
    assert dg.load().dg_w4_read(dg.ct.byref(w.s), out.data_ptr(), out.stride(0), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out.cpu().double(), w4_ref.weights(c, s))
