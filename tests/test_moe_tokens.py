"""dg_moe_tokens without a GPU: what it refuses.  Device pointers passed here are never dereferenced."""
import ctypes as ct
import os

import pytest
import torch

FAKE = 1 << 20


@pytest.fixture(scope="module")
def dg():
    import __graft_entry__ as g
    from block_diffusion_text_gb300 import dg as _dg
    if not os.path.exists(_dg.LIB_PATH):
        g.build_cuda()
    _dg.load()
    return _dg


def _model(dg, Wr=FAKE, We1=FAKE, We2=FAKE, **kw):
    m = dg.dg_model()
    m.dims = dg.dg_dims(**dict(dict(d=256, n_exp=8, top_k=2, Fe=128, rms_eps=1e-6, L=2), **kw))
    m.Wr, m.We1, m.We2 = Wr, We1, We2
    return ct.byref(m)


BAD = [(dict(d=0), "ARG"), (dict(n_exp=0), "ARG"), (dict(top_k=0), "ARG"), (dict(top_k=9), "ARG"), (dict(Fe=-128), "ARG"),
       (dict(L=0), "ARG"), (dict(rms_eps=-1.0), "ARG"), (dict(rms_eps=float("nan")), "ARG"), (dict(d=192), "SHAPE"),
       (dict(d=16512), "SHAPE"), (dict(Fe=64), "SHAPE"), (dict(Fe=16512), "SHAPE"), (dict(n_exp=257), "SHAPE"),
       (dict(n_exp=32, top_k=17), "SHAPE"), (dict(L=65), "SHAPE")]


@pytest.mark.parametrize("kw,code", BAD, ids=[str(k) for k, _ in BAD])
def test_bad_sizes_are_refused(dg, kw, code):
    L, f, z, want = dg.load(), FAKE, ct.c_size_t(), getattr(dg, "DG_ERR_" + code)
    assert L.dg_moe_tokens_workspace(_model(dg, **kw), 4, ct.byref(z)) == want
    assert L.dg_moe_tokens(_model(dg, **kw), 0, f, f, 4, f, f, f, 1 << 30, None) == want


def test_refusals(dg):
    L, f, z = dg.load(), FAKE, ct.c_size_t()
    assert L.dg_moe_tokens_workspace(None, 4, ct.byref(z)) == L.dg_moe_tokens_workspace(_model(dg), 4, None) == dg.DG_ERR_ARG
    assert L.dg_moe_tokens_workspace(_model(dg), 0, ct.byref(z)) == dg.DG_ERR_ARG
    assert L.dg_moe_tokens_workspace(_model(dg), 33, ct.byref(z)) == dg.DG_ERR_SHAPE
    assert L.dg_moe_tokens_workspace(_model(dg), 32, ct.byref(z)) == dg.DG_OK and z.value > 0
    ok = dict(model=_model(dg), layer=1, h=f, out=f, M=32, idx=f, gate=f, ws=f, n=z.value)

    def rc(**kw):
        return L.dg_moe_tokens(*dict(ok, **kw).values(), None)
    for kw in (dict(model=None), dict(layer=-1), dict(layer=2), dict(h=None), dict(out=None), dict(M=0), dict(ws=None),
               dict(h=f + 8), dict(out=f + 2), dict(idx=f + 2), dict(gate=f + 1), dict(model=_model(dg, Wr=0)),
               dict(model=_model(dg, We1=0)), dict(model=_model(dg, We2=0)), dict(model=_model(dg, Wr=f + 8)),
               dict(model=_model(dg, We1=f + 8)), dict(model=_model(dg, We2=f + 2))):
        assert rc(**kw) == dg.DG_ERR_ARG, kw
    assert rc(M=33) == dg.DG_ERR_SHAPE
    assert rc(ws=f + 64) == rc(n=z.value - 1) == dg.DG_ERR_WORKSPACE


def test_binding_refuses_cpu_tensors(dg):
    bf = torch.bfloat16
    with pytest.raises(ValueError):
        dg.MoeFfn(torch.zeros(8, 256, dtype=bf), torch.zeros(9, 128, 256, dtype=bf), torch.zeros(9, 256, 128, dtype=bf), 2)
