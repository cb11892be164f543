"""The 4-bit matrices' entry points without a GPU: what they refuse before touching the device, and the restatement
that the GPU tests compare with.  Device pointers passed here are never dereferenced."""
import ctypes as ct
import os

import pytest
import torch

import w4_ref

FAKE = 1 << 20


@pytest.fixture(scope="module")
def dg():
    import __graft_entry__ as g
    from block_diffusion_text_gb300 import dg as _dg
    if not os.path.exists(_dg.LIB_PATH):
        g.build_cuda()
    _dg.load()
    return _dg


def _w4(dg, **kw):
    d = dict(codes=FAKE, scales=FAKE, N=100, K=256, group=64)
    d.update(kw)
    return ct.byref(dg.dg_w4(*[d[f] for f, _ in dg.dg_w4._fields_]))


BAD = [(dict(codes=0), "ARG"), (dict(scales=0), "ARG"), (dict(codes=FAKE + 8), "ARG"), (dict(scales=FAKE + 2), "ARG"),
       (dict(N=0), "ARG"), (dict(K=-64), "ARG"), (dict(group=0), "ARG"), (dict(group=16), "SHAPE"), (dict(K=96), "SHAPE"),
       (dict(K=192, group=128), "SHAPE"), (dict(K=65536 + 64), "SHAPE"), (dict(N=(1 << 24) + 1), "SHAPE")]


@pytest.mark.parametrize("kw,code", BAD, ids=[str(k) for k, _ in BAD])
def test_bad_matrices_are_refused(dg, kw, code):
    L, f, w = dg.load(), FAKE, _w4(dg, **kw)
    want = getattr(dg, "DG_ERR_" + code)
    assert L.dg_w4_quantize(w, f, 1 << 20, f, None) == want
    assert L.dg_w4_pack(w, f, f, None) == want
    assert L.dg_w4_read(w, f, 1 << 20, None) == want
    assert L.dg_w4_matvec(w, f, 1 << 20, 1, None, 1.0, None, 0, f, 1 << 26, 0, None) == want


def test_bytes(dg):
    L, a, b = dg.load(), ct.c_size_t(), ct.c_size_t()
    assert L.dg_w4_bytes(17, 128, 32, ct.byref(a), ct.byref(b)) == dg.DG_OK
    assert (a.value, b.value) == (64 * 64, 64 * 4 * 2)
    assert L.dg_w4_bytes(17, 128, 32, None, ct.byref(b)) == L.dg_w4_bytes(17, 128, 32, ct.byref(a), None) == dg.DG_ERR_ARG
    assert L.dg_w4_bytes(0, 128, 32, ct.byref(a), ct.byref(b)) == dg.DG_ERR_ARG
    assert L.dg_w4_bytes(17, 100, 32, ct.byref(a), ct.byref(b)) == dg.DG_ERR_SHAPE


def test_refusals(dg):
    L, f, w = dg.load(), FAKE, _w4(dg)
    assert L.dg_w4_quantize(None, f, 256, f, None) == L.dg_w4_quantize(w, None, 256, f, None) == dg.DG_ERR_ARG
    assert L.dg_w4_quantize(w, f, 255, f, None) == L.dg_w4_quantize(w, f, 256, None, None) == dg.DG_ERR_ARG
    assert L.dg_w4_quantize(w, f + 1, 256, f, None) == L.dg_w4_quantize(w, f, 256, f + 2, None) == dg.DG_ERR_ARG
    assert L.dg_w4_pack(w, None, f, None) == L.dg_w4_pack(w, f, None, None) == L.dg_w4_pack(w, f, f + 1, None) == dg.DG_ERR_ARG
    assert L.dg_w4_read(w, None, 256, None) == L.dg_w4_read(w, f, 255, None) == L.dg_w4_read(w, f + 2, 256, None) == dg.DG_ERR_ARG
    ok = dict(w=w, x=f, ldx=256, M=4, alpha=f, coef=1.0, resid=f, ldr=100, y=f, ldy=100, f32=1)

    def rc(**kw):
        return L.dg_w4_matvec(*dict(ok, **kw).values(), None)
    assert rc(w=None) == rc(x=None) == rc(y=None) == rc(M=0) == rc(M=-1) == dg.DG_ERR_ARG
    assert rc(ldx=248) == rc(ldx=260) == rc(ldy=99) == rc(ldr=99) == dg.DG_ERR_ARG
    assert rc(x=f + 8) == rc(y=f + 2) == rc(resid=f + 1) == rc(alpha=f + 2) == rc(y=f + 1, f32=0) == dg.DG_ERR_ARG
    assert rc(M=33) == dg.DG_ERR_SHAPE


def test_binding_refuses_cpu_tensors(dg):
    with pytest.raises(ValueError):
        dg.w4_quantize(torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        dg.W4Matrix.from_codes(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.bfloat16))


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantised_weights_are_within_half_a_step(group):
    g = torch.Generator().manual_seed(group)
    W = (torch.randn(50, 256, generator=g) * torch.exp2(torch.randint(-20, 20, (50, 1), generator=g).float())).to(torch.bfloat16)
    c, s = w4_ref.quantize(W, group)
    err = (w4_ref.weights(c, s) - W.double()).abs()
    step = s.double().repeat_interleave(group, 1)
    # the scale is rounded by 2^-9 at most: the largest weight, 7 steps before, is off by 7 * 2^-9 of a step more
    assert bool((err <= step * (0.5 + 7 * 2.0 ** -8)).all())
    assert c.min() >= 1 and c.max() <= 15


def test_status_refuses_null(dg):
    assert dg.load().dg_w4_status(None, None) == 1


def test_sizes_beyond_32_bits_are_not_cut(dg):
    for N, K, group in (((1 << 32) + 16, 64, 64), (16, (1 << 32) + 64, 64), (16, 64, (1 << 32) + 64), (-(1 << 32) + 16, 64, 64)):
        with pytest.raises(dg.DgError) as e:
            dg.W4Matrix(N, K, group)
        assert e.value.code == dg.DG_ERR_SHAPE
