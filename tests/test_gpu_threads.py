"""Host threads: a call may be a thread's first use of the GPU."""
import threading

import pytest
import torch

from block_diffusion_text_gb300 import dg, synth
from test_gpu_kv8 import filled, rows

pytestmark = pytest.mark.gpu


def in_thread(fn):
    """fn() in a new thread; its result or its exception."""
    box = []

    def run():
        try:
            box.append(fn())
        except Exception as e:  # noqa: BLE001
            box.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if isinstance(box[0], Exception):
        raise box[0]
    return box[0]


@pytest.mark.parametrize("C,cap", [(1, 400), (256, 5000)])
def test_attention_over_8_bits_is_a_threads_first_call(C, cap):
    g = torch.Generator().manual_seed(80)
    c = filled(g, 1, 2, cap, 128, [390])
    x = [rows(g, 1, h, C, 128).cuda() for h in (4, 2, 2)]
    want = dg.kv8_attention(c, *x)
    out = torch.zeros_like(want)
    ws = torch.empty(max(c.workspace_bytes(C, 4), 256), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    in_thread(lambda: dg.kv8_attention(c, *x, out=out, ws=ws))
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_step_is_a_threads_first_call():
    dims, seed = synth.workload("tiny_v512_c16")
    model = dg.Model(dims, synth.make_weights(dims, seed, device="cuda"))
    state = [t.cuda() for t in synth.make_canvas(dims, seed, device="cpu")]

    def step():
        return dg.denoise_step(model, dg.Canvas(*[t.clone() for t in state]), tau=0.8, b=0.1, seed=seed, step=0)

    want = step()
    torch.cuda.synchronize()
    got = in_thread(step)
    torch.cuda.synchronize()
    assert torch.equal(got["entropy"], want["entropy"])
