"""The workspaces that attention over the 8-bit cache keeps by itself: one for a stream, whatever the number of caches
and of host threads."""
import threading

import pytest
import torch

from block_diffusion_text_gb300 import dg
from test_gpu_kv8 import filled, rows

pytestmark = pytest.mark.gpu


def test_a_stack_of_caches_shares_one_workspace():
    g = torch.Generator().manual_seed(70)
    first = filled(g, 1, 2, 20000, 128, [19000])
    stack = [first] + [dg.Kv8Cache(first.K, first.V, first.K_exp, first.V_exp, first.len, first.status_word)
                       for _ in range(7)]
    q = rows(g, 1, 8, 256, 128).cuda()
    out = torch.empty(256, 8 * 128, dtype=torch.bfloat16, device="cuda")
    need = first.workspace_bytes(256, 8)
    assert need > 2 ** 22
    dg.kv8_release_workspaces()
    before = torch.cuda.memory_allocated()
    for c in stack:
        dg.kv8_attention(c, q, out=out)
    assert torch.cuda.memory_allocated() - before < 2 * need
    torch.cuda.synchronize()
    dg.kv8_release_workspaces("cuda")
    assert torch.cuda.memory_allocated() == before


def test_a_released_workspace_is_taken_anew():
    g = torch.Generator().manual_seed(71)
    c = filled(g, 2, 2, 20000, 128, [19000, 3])
    q = rows(g, 2, 8, 64, 128).cuda()
    want = dg.kv8_attention(c, q)
    dg.kv8_release_workspaces()
    filler = torch.full((c.workspace_bytes(64, 8),), 0xff, dtype=torch.uint8, device="cuda")
    assert torch.equal(dg.kv8_attention(c, q), want) and (filler == 0xff).all()


@pytest.mark.parametrize("one_cache", [True, False])
def test_host_threads_on_one_stream(one_cache):
    """Calls of four threads on one stream, of sizes that grow the workspace and take different kernels: a call's
    launches follow one another, so each gives what it gives alone."""
    g = torch.Generator().manual_seed(72)
    c = filled(g, 2, 2, 20000, 128, [19000, 777])
    caches = [c if one_cache else dg.Kv8Cache(c.K, c.V, c.K_exp, c.V_exp, c.len) for _ in range(4)]
    sizes = (1, 40, 3, 256)
    x = [[rows(g, 2, h, C, 128).cuda() for h in (8, 2, 2)] for C in sizes]
    want = [dg.kv8_attention(c, *t) for t in x]
    torch.cuda.synchronize()
    dg.kv8_release_workspaces()
    st = torch.cuda.Stream()
    got, errors = [[] for _ in sizes], []
    start = threading.Barrier(len(sizes))

    def work(i):
        try:
            start.wait()
            for _ in range(40):
                got[i].append(dg.kv8_attention(caches[i], *x[i], stream=st))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for outs, w in zip(got, want):
        assert len(outs) == 40 and all(torch.equal(o, w) for o in outs)
