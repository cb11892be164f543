"""dg_sample without a GPU: what it refuses, and the restatement that the GPU tests go by.  Device pointers passed here
are never dereferenced."""
import ctypes as ct
import os

import pytest
import torch

import sample_ref

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
    def how(**kw):
        return ct.byref(dg.dg_sampling(**dict(dict(temperature_all=1.0, top_p_all=1.0), **kw)))
    f = FAKE
    ok = dict(logits=f, bf16=0, ld=100, R=2, V=100, how=how(), u=f, token=f, logprob=f, kept=f)

    def rc(**kw):
        return dg.load().dg_sample(*dict(ok, **kw).values(), None)
    for kw in (dict(logits=None), dict(how=None), dict(u=None), dict(token=None), dict(R=0), dict(V=0), dict(V=-5), dict(ld=99),
               dict(logits=f + 2), dict(logits=f + 1, bf16=1), dict(u=f + 2), dict(token=f + 1), dict(logprob=f + 2),
               dict(kept=f + 2), dict(how=how(temperature=f + 2)), dict(how=how(top_p=f + 1)), dict(how=how(min_p=f + 2)),
               dict(how=how(top_k=f + 3))):
        assert rc(**kw) == dg.DG_ERR_ARG, kw
    assert rc(V=(1 << 20) + 1, ld=1 << 21) == dg.DG_ERR_SHAPE


def test_binding_refuses_cpu_tensors(dg):
    with pytest.raises(ValueError):
        dg.sample(torch.zeros(2, 8), torch.zeros(2))


def test_restatement_knows_wrong_answers():
    x = torch.tensor([0.0, 1.0, 1.0, -1.0])
    w = torch.exp(x.double() - 1)
    lp = float((w[1] / w[[1, 2]].sum()).log())
    good = dict(token=1, logprob=lp, kept=2)

    def bad(**kw):
        return sample_ref.check_row(x, 0.2, 1.0, 2, 1.0, 0.0, **dict(good, **kw))
    assert bad() is None
    assert bad(token=2) and bad(token=0) and bad(kept=3) and bad(logprob=lp + 1e-3) and bad(token=-1)
