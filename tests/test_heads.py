"""dg_qk_norm_rope without a GPU: what it refuses.  Device pointers passed here are never dereferenced."""
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


def test_refusals(dg):
    ok = dict(qkv=FAKE, sb=1024, st=512, pos=FAKE, qg=FAKE, kg=None, q=FAKE, k=FAKE, v=FAKE, B=2, C=2, Hq=2, Hkv=1, hd=128,
              base=10000.0, eps=1e-6)

    def rc(**kw):
        return dg.load().dg_qk_norm_rope(*dict(ok, **kw).values(), None)
    for kw in (dict(qkv=None), dict(pos=None), dict(q=None), dict(k=None), dict(v=None), dict(B=0), dict(C=-1), dict(Hq=0),
               dict(Hkv=0), dict(st=511), dict(st=516), dict(st=256), dict(sb=1028), dict(sb=8), dict(qkv=FAKE + 8),
               dict(q=FAKE + 2), dict(k=FAKE + 8), dict(v=FAKE + 4), dict(pos=FAKE + 2), dict(qg=FAKE + 1), dict(kg=FAKE + 1),
               dict(base=0.5), dict(base=float("nan")), dict(base=float("inf")), dict(eps=-1.0), dict(eps=float("nan"))):
        assert rc(**kw) == dg.DG_ERR_ARG, kw
    for kw in (dict(hd=96), dict(hd=256), dict(Hq=1025, st=1 << 20, sb=1 << 21), dict(B=1 << 20, C=65)):
        assert rc(**kw) == dg.DG_ERR_SHAPE, kw


def test_binding_refuses_cpu_tensors(dg):
    with pytest.raises(ValueError):
        dg.qk_norm_rope(torch.zeros(1, 1, 128, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32), 2, 1)
