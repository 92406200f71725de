"""What the operators' binding does to the tensors it is given."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def flow():
    from video_generation_b200 import build
    build.build()
    from video_generation_b200 import flow as F
    assert torch.cuda.is_available()
    return F


def test_what_a_call_writes_moves_its_version(flow):
    """A graph that saved a tensor must not use it after a call wrote over it."""
    B, n, H, D = 2, 3, 2, 64
    cache = flow.KVCache(B, H, D, 8)
    x = torch.randn(B, n, H, D, device="cuda").bfloat16()
    pos, length = torch.zeros(B * n, 3, dtype=torch.int32, device="cuda"), torch.tensor([n, n], dtype=torch.int32, device="cuda")
    bufs = {name: torch.ones(B, n, H, D, dtype=torch.bfloat16, device="cuda") for name in ("q", "k", "v", "out")}
    w = {name: torch.ones((), device="cuda", requires_grad=True) for name in bufs}
    y = {name: (t * w[name]).sum() for name, t in bufs.items()}      # each saves its buffer
    before = cache.storage._version
    flow.af_cache_write(cache, x, x)
    assert cache.storage._version == before + 1
    rope = flow.Rope(D, (8, 8, 8))
    q, none = flow.af_qk_norm_rope(rope, x.flatten(0, 1), None, pos, q_out=bufs["q"].flatten(0, 1))
    assert none is None and q.data_ptr() == bufs["q"].data_ptr()
    k, v = flow.af_cache_read(cache, n, k=bufs["k"], v=bufs["v"])
    assert k is bufs["k"] and v is bufs["v"]
    assert flow.af_cache_attention(cache, x, length, out=bufs["out"]) is bufs["out"]
    for name, t in y.items():
        with pytest.raises(RuntimeError, match="inplace"):
            t.backward()
    # what is only read does not move
    assert x._version == 0 and pos._version == 0 and length._version == 0


def test_calls_in_inference_mode_and_without_gradients(flow):
    cache = flow.KVCache(1, 2, 64, 8)
    x = torch.randn(1, 3, 2, 64, device="cuda").bfloat16()
    length = torch.tensor([3], dtype=torch.int32, device="cuda")
    flow.af_cache_write(cache, x, x)
    want = flow.af_cache_attention(cache, x, length)
    with torch.no_grad():
        assert torch.equal(flow.af_cache_attention(cache, x.clone().requires_grad_(), length), want)
    with torch.inference_mode():
        c = flow.KVCache(1, 2, 64, 8)
        y = x.clone()
        flow.af_cache_write(c, y, y)
        out = torch.empty_like(y)
        assert torch.equal(flow.af_cache_attention(c, y, length, out=out), want)
    flow.af_cache_write(c, x, x)                             # an inference tensor, written outside
    assert torch.equal(flow.af_cache_attention(c, x, length), want)


def test_outputs_whose_strides_differ_where_they_say_nothing(flow):
    """One sequence and one row: rows of unlike buffers have one layout."""
    cache = flow.KVCache(1, 2, 64, 8)
    x = torch.randn(1, 4, 2, 64, device="cuda").bfloat16()
    flow.af_cache_write(cache, x, x)
    start = torch.tensor([2], dtype=torch.int32, device="cuda")
    want, _ = flow.af_cache_read(cache, 1, start=start)
    wide = torch.zeros(5, 7, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    k, v = wide[1:2, 3:4, 1], torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert k.stride() != v.stride()
    flow.af_cache_read(cache, 1, start=start, k=k, v=v)
    assert torch.equal(k, want) and torch.equal(v, want) and int((wide != 0).sum()) == int((want != 0).sum())
    # rows that do differ stay refused
    for k, v in ((wide[:1, :4, 0], torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device="cuda")),
                 (wide[:1, :4, 0], wide[:1, 3:6, 0].flatten(2).unflatten(2, (2, 64)).contiguous())):
        with pytest.raises(ValueError):
            flow.af_cache_read(cache, 4, k=k, v=v)
