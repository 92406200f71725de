"""Calls that run smaller calls of several sizes in one workspace (flow_pipeline_inverse with a shorter last group,
af_inverse_jacobi_stream with a shorter last window): the documented size serves every one of them, and the results are
those of the smaller calls by themselves."""
import itertools

import pytest
import torch

import synthetic as syn
from oracle import af_oracle as O
from tests.gpu_util import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def flow():
    from video_generation_b200 import build
    build.build()
    from video_generation_b200 import flow as F
    assert torch.cuda.is_available()
    return F


def _up(n):
    return -(-n // 256) * 256


WIDTHS = [(128, 2), (256, 4), (256, 2), (768, 12), (1024, 8)]


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("d,heads", WIDTHS)
def test_the_size_serves_every_group_and_window(flow, d, heads, bits):
    """By arithmetic only: what a group or window of n frames needs, against the part of the documented size that is
    not staging."""
    for F in (26, 130, 195, 390):
        shape = syn.ModelShape(C=64, d=d, heads=heads, layers=1, mlp_ratio=1, frame_len=F, max_frames=8, dtype="bf16")
        m = flow.AFModel(shape, syn.make_weights(shape))
        m.set_cache_bits(bits)
        for batch, n in itertools.product((1, 2, 3, 5), range(1, 9)):
            staged = 2 * _up(batch * n * F * 64 * 4)
            pipeline = flow.lib().flow_pipeline_workspace_bytes(m.handle, 3, batch, F, n) - staged - _up(3 * batch * n * 4)
            stream = flow.lib().af_stream_workspace_bytes(m.handle, batch, n) - staged - _up(batch * n * 4)
            assert pipeline >= max(m.workspace_bytes(batch * g, F) for g in range(1, n + 1)), (F, batch, n)
            assert stream >= max(m.workspace_bytes(batch, g * F, F) for g in range(1, n + 1)), (F, batch, n)
    assert flow.lib().flow_pipeline_workspace_bytes(m.handle, 3, 2 ** 20, 390, 2 ** 20) == 0
    assert flow.lib().flow_pipeline_workspace_bytes(m.handle, 3, 1, 0, 2) == 0
    assert flow.lib().af_stream_workspace_bytes(m.handle, 1, 9) == 0


def _model(flow, shape, block, bits):
    m = flow.AFModel(shape, syn.make_weights(shape, block=block, head_std=1e-2))
    m.set_cache_bits(bits)
    return m


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("batch,frames,group", [(2, 3, 2), (1, 6, 4), (1, 7, 4)])
def test_a_pipeline_whose_last_group_is_shorter(flow, batch, frames, group, bits):
    """Frames of 390 tokens through a stack of width 768 with 12 heads."""
    F = 390
    deep = _model(flow, syn.ModelShape(C=64, d=128, heads=2, layers=1, mlp_ratio=2, frame_len=F, max_frames=8,
                                       dtype="bf16"), 0, bits)
    narrow = syn.ModelShape(C=64, d=768, heads=12, layers=4, mlp_ratio=4, frame_len=F, max_frames=1, dtype="bf16")
    models, dirs = [_model(flow, narrow, 1 + t, bits) for t in range(2)], (O.L2R, O.R2L)
    z = to_dev(syn.make_latents(batch, frames * F, 64, 5))
    x, itd, its = flow.flow_pipeline_inverse(deep, models, dirs, z, F, 1e-3, 8, 8, True, group=group,
                                             stream_shallow=torch.cuda.Stream())
    u, itu = flow.af_inverse_jacobi(deep, z, O.L2R, F, 1e-3, 8, True)
    assert torch.equal(itd, itu)
    for f0 in range(0, frames, group):
        n = min(group, frames - f0)
        fr = u[:, f0 * F:(f0 + n) * F].reshape(batch * n, F, 64).contiguous()
        xf, itf = flow.flow_stack_inverse(models, dirs, fr, F, 1e-3, 8, False)
        assert torch.equal(x[:, f0 * F:(f0 + n) * F], xf.reshape(batch, n * F, 64))
        assert torch.equal(its[:, :, f0:f0 + n], itf.reshape(2, batch, n))
    assert deep.device_error() == 0 and all(m.device_error() == 0 for m in models)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("d,heads,layers,F,window,overlap,frames", [
    (256, 4, 2, 130, 5, 1, 8),      # windows of 5 and 4 frames
    (768, 12, 2, 195, 6, 2, 9),     # 6 and 5
    (768, 12, 1, 195, 6, 1, 13),    # 6, 6, 3
    (128, 2, 1, 390, 4, 0, 3),      # one window, shorter than `window`
])
def test_a_stream_whose_last_window_is_shorter(flow, d, heads, layers, F, window, overlap, frames, bits):
    """Every window is the encoding of its observed frames and the inverse of the others."""
    shape = syn.ModelShape(C=64, d=d, heads=heads, layers=layers, mlp_ratio=2, frame_len=F, max_frames=window, dtype="bf16")
    m = _model(flow, shape, 0, bits)
    z = to_dev(syn.make_latents(2, frames * F, 64, 9))
    x, iters = flow.af_inverse_jacobi_stream(m, z, window, overlap, 1e-3, 8, True)
    s0 = 0
    while True:
        n, seen = min(window, frames - s0), overlap if s0 else 0
        zw, ws = z[:, s0 * F:(s0 + n) * F].contiguous(), m.workspace(2, n * F, F)
        xw = torch.zeros_like(zw)
        if seen:
            xw[:, :seen * F] = x[:, s0 * F:(s0 + seen) * F]
            flow.af_prefix_encode(m, xw, O.L2R, F, seen * F, ws)
        _, it = flow.af_inverse_jacobi_schedule(m, zw, O.L2R, [F] * n, 1e-3, 8, True, b_begin=seen, b_end=n, ws=ws, x=xw)
        assert torch.equal(x[:, s0 * F:(s0 + n) * F], xw)
        assert torch.equal(iters[:, s0 + seen:s0 + n], it[:, seen:n])
        if s0 + window >= frames:
            break
        s0 += window - overlap
    assert m.device_error() == 0
