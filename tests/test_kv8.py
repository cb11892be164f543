"""The 8-bit prefix cache's entry points without a GPU: what they refuse, before touching the device, and the
64-bit restatement that the GPU tests compare with.  Device pointers passed here are never dereferenced."""
import ctypes as ct
import os

import pytest
import torch

import kv8_ref

FAKE = 1 << 20


@pytest.fixture(scope="module")
def dg():
    import __graft_entry__ as g
    from block_diffusion_text_gb300 import dg as _dg
    if not os.path.exists(_dg.LIB_PATH):
        g.build_cuda()
    _dg.load()
    return _dg


def _cache(dg, **kw):
    d = dict(K=FAKE, V=FAKE, K_exp=FAKE, V_exp=FAKE, len=FAKE, status=FAKE, B=2, Hkv=2, cap=256, hd=128)
    d.update(kw)
    return dg.dg_kv8_cache(*[d[f] for f, _ in dg.dg_kv8_cache._fields_])


BAD_CACHES = [(dict(K=0), "ARG"), (dict(V=0), "ARG"), (dict(K_exp=0), "ARG"), (dict(V_exp=0), "ARG"),
              (dict(len=0), "ARG"), (dict(status=0), "ARG"), (dict(B=0), "ARG"), (dict(Hkv=-1), "ARG"),
              (dict(cap=0), "ARG"), (dict(K=FAKE + 8), "ARG"), (dict(V=FAKE + 1), "ARG"), (dict(hd=96), "SHAPE"),
              (dict(B=65536, Hkv=1), "SHAPE"), (dict(B=1024, Hkv=8, cap=1 << 20), "SHAPE")]


@pytest.mark.parametrize("kw,code", BAD_CACHES, ids=[str(k) for k, _ in BAD_CACHES])
def test_bad_caches_are_refused(dg, kw, code):
    L, f, z = dg.load(), FAKE, ct.c_size_t()
    c = ct.byref(_cache(dg, **kw))
    want = getattr(dg, "DG_ERR_" + code)
    assert L.dg_kv8_append(c, f, f, 4, None, None) == want
    assert L.dg_kv8_read(c, 0, 4, f, f, 4, None) == want
    assert L.dg_kv8_attention_workspace(c, 4, 8, ct.byref(z)) == want
    assert L.dg_kv8_attention(c, f, f, f, f, 4, 8, 0, f, 1 << 40, None) == want


def test_append_refusals(dg):
    L, f = dg.load(), FAKE
    c = ct.byref(_cache(dg))
    assert L.dg_kv8_append(None, f, f, 4, None, None) == dg.DG_ERR_ARG
    assert L.dg_kv8_append(c, None, f, 4, None, None) == dg.DG_ERR_ARG
    assert L.dg_kv8_append(c, f, None, 4, None, None) == dg.DG_ERR_ARG
    assert L.dg_kv8_append(c, f, f, 0, None, None) == dg.DG_ERR_ARG
    assert L.dg_kv8_append(c, f + 8, f, 4, None, None) == dg.DG_ERR_ARG
    assert L.dg_kv8_append(c, f, f + 2, 4, None, None) == dg.DG_ERR_ARG
    assert L.dg_kv8_append(c, f, f, 257, None, None) == dg.DG_ERR_CAPACITY


def test_read_refusals(dg):
    L, f = dg.load(), FAKE
    c = ct.byref(_cache(dg))
    assert L.dg_kv8_read(None, 0, 4, f, f, 4, None) == dg.DG_ERR_ARG
    assert L.dg_kv8_read(c, -1, 4, f, f, 4, None) == dg.DG_ERR_ARG
    assert L.dg_kv8_read(c, 0, 0, f, f, 4, None) == dg.DG_ERR_ARG
    assert L.dg_kv8_read(c, 0, 4, f, f, 3, None) == dg.DG_ERR_ARG
    assert L.dg_kv8_read(c, 0, 4, None, f, 4, None) == dg.DG_ERR_ARG
    assert L.dg_kv8_read(c, 0, 4, f, f + 4, 4, None) == dg.DG_ERR_ARG


def test_attention_refusals(dg):
    L, f, z = dg.load(), FAKE, ct.c_size_t()
    # a short cache is finished in one launch, without a workspace; a long one needs one
    assert L.dg_kv8_attention_workspace(ct.byref(_cache(dg)), 16, 8, ct.byref(z)) == dg.DG_OK and z.value == 0
    c = ct.byref(_cache(dg, cap=65536))
    assert L.dg_kv8_attention_workspace(c, 16, 8, ct.byref(z)) == dg.DG_OK and z.value > 0
    assert L.dg_kv8_attention_workspace(c, 16, 8, None) == dg.DG_ERR_ARG
    ok = dict(c=c, q=f, k=f, v=f, o=f, C=16, Hq=8, causal=0, ws=f, n=z.value)

    def rc(**kw):
        a = dict(ok, **kw)
        return L.dg_kv8_attention(a["c"], a["q"], a["k"], a["v"], a["o"], a["C"], a["Hq"], a["causal"], a["ws"],
                                  a["n"], None)
    assert rc(c=None) == rc(q=None) == rc(o=None) == rc(ws=None) == dg.DG_ERR_ARG
    assert rc(k=None) == rc(v=None) == dg.DG_ERR_ARG          # one without the other
    assert rc(C=0) == rc(Hq=0) == rc(Hq=7) == dg.DG_ERR_ARG
    assert rc(q=f + 8) == rc(k=f + 8) == rc(v=f + 8) == rc(o=f + 8) == dg.DG_ERR_ARG
    assert rc(C=1025) == rc(Hq=65536) == dg.DG_ERR_SHAPE
    big = ct.byref(_cache(dg, B=2048, Hkv=1, cap=64))
    assert rc(c=big, C=1024) == dg.DG_ERR_SHAPE               # B * C > 2^20
    assert rc(ws=f + 128) == rc(n=z.value - 1) == dg.DG_ERR_WORKSPACE


def test_binding_refuses_wrong_tensors(dg):
    u8 = dict(dtype=torch.uint8)
    t = dict(K=torch.zeros(2, 2, 100, 64, **u8), V=torch.zeros(2, 2, 100, 64, **u8), K_exp=torch.zeros(2, 2, 2, **u8),
             V_exp=torch.zeros(2, 2, 2, **u8), len=torch.zeros(2, dtype=torch.int32))
    bad = [dict(K=torch.zeros(2, 2, 100, 64)), dict(V=torch.zeros(2, 2, 99, 64, **u8)),
           dict(K_exp=torch.zeros(2, 2, 1, **u8)), dict(len=torch.zeros(2, dtype=torch.int64)),
           dict(len=torch.zeros(3, dtype=torch.int32)), dict()]   # the last: right shapes, but on the CPU
    for kw in bad:
        with pytest.raises(ValueError):
            dg.Kv8Cache(**dict(t, **kw))


def test_reference_rounding_is_torchs():
    """round_e4m3 and exponent against torch's own conversion and frexp."""
    g = torch.Generator().manual_seed(3)
    y = torch.cat([torch.randn(20000, generator=g) * torch.exp2(torch.randint(-12, 9, (20000,), generator=g).float()),
                   kv8_ref.e4m3_table()[:126].float() * 1.0,
                   (kv8_ref.e4m3_table()[1:126] + kv8_ref.e4m3_table()[:125]).float() / 2]).clamp(-448, 448)
    assert torch.equal(kv8_ref.round_e4m3(y.double()).float(), y.to(torch.float8_e4m3fn).float())
    for top in (448.0, 448.0 * 2 ** -3, 449.0, 1e-30, 0.0, 3e38, 1.0, 1.75, 1.7578125):
        e = kv8_ref.exponent(top)
        assert e == kv8_ref.E_MAX or top <= 448.0 * 2.0 ** e
        assert e == kv8_ref.E_MIN or top > 448.0 * 2.0 ** (e - 1)
