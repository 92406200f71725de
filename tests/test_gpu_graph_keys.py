"""Calls replay captured graphs; a graph is of the models it was captured with and of their settings."""
import pytest
import torch

import synthetic as syn
from oracle import af_oracle as O
from tests.gpu_util import to_dev

pytestmark = pytest.mark.gpu

SHAPE = syn.ModelShape(C=64, d=128, heads=2, layers=1, mlp_ratio=2, frame_len=130, max_frames=1, dtype="bf16")


@pytest.fixture(scope="module")
def flow():
    from video_generation_b200 import build
    build.build()
    from video_generation_b200 import flow as F
    assert torch.cuda.is_available()
    return F


def _model(flow, block):
    return flow.AFModel(SHAPE, syn.make_weights(SHAPE, block=block, head_std=5e-2))


def test_a_model_made_after_another_was_destroyed(flow):
    """The second block of a stack destroyed and made anew, again and again in the same buffers: allocators give the new
    one the old one's addresses now and then."""
    first, x = _model(flow, 0), to_dev(syn.make_latents(2, 130, 64, 3))
    ws, z, ld = first.workspace(2, 130), torch.empty_like(x), torch.empty(2, device="cuda")
    handles = []
    for block in range(1, 9):
        second = _model(flow, block)
        handles.append(second.handle if isinstance(second.handle, int) else second.handle.value)
        flow.flow_stack_forward([first, second], [O.L2R, O.R2L], x, ws=ws, z=z, logdet=ld)
        mid, ld0 = flow.af_forward(first, x, O.L2R)
        want, ld1 = flow.af_forward(second, mid, O.R2L)
        assert torch.equal(z, want) and torch.allclose(ld, ld0 + ld1, rtol=1e-6, atol=1e-3)
        second.close()
    print("addresses used again:", len(handles) - len(set(handles)))


def test_the_wait_limit_of_every_block_of_a_stack(flow):
    """A limit set on the second block after the stack's graph was captured."""
    first, second = _model(flow, 0), _model(flow, 1)
    x = to_dev(syn.make_latents(2, 130, 64, 3))
    ws, z, ld = first.workspace(2, 130), torch.empty_like(x), torch.empty(2, device="cuda")

    def run():
        flow.flow_stack_forward([first, second], [O.L2R, O.R2L], x, ws=ws, z=z, logdet=ld)
        return first.device_error(), second.device_error()

    assert run() == (0, 0)
    want = z.clone()
    second.set_wait_limit(1e-9)
    codes = [run() for _ in range(3)]
    assert all(a == 0 for a, _ in codes) and any(b for _, b in codes) and not any(b & 2 for _, b in codes)
    second.set_wait_limit(2.0)
    assert run() == (0, 0) and torch.equal(z, want)
