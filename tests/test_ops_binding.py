"""What the operators' compiled binding refuses before it asks for a device (host tensors stand in; nothing is launched)."""
import pytest
import torch


@pytest.fixture(scope="module")
def flow():
    from video_generation_b200 import build
    build.build()
    from video_generation_b200 import flow as F
    return F


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


def rows(*shape, grad=False):
    return torch.zeros(*shape, dtype=torch.bfloat16).requires_grad_(grad)


@pytest.fixture
def cache(flow):
    return flow.KVCache(2, 2, 64, 10, device="cpu")


def calls(flow, cache, grad):
    """Each call with one tensor that requires grad."""
    rope, pos, x = flow.Rope(64, (8, 8, 8)), torch.zeros(3, 3, dtype=torch.int32), rows(2, 3, 2, 64)
    yield lambda: flow.af_qk_norm_rope(rope, rows(3, 2, 64, grad=grad), None, pos)
    yield lambda: flow.af_qk_norm_rope(rope, None, rows(3, 2, 64, grad=grad), pos)
    yield lambda: flow.af_qk_norm_rope(rope, rows(3, 2, 64), None, pos, torch.ones(64, requires_grad=grad))
    yield lambda: flow.af_qk_norm_rope(rope, rows(3, 2, 64), None, pos, q_out=rows(3, 2, 64, grad=grad))
    yield lambda: flow.af_cache_write(cache, x, rows(2, 3, 2, 64, grad=grad))
    yield lambda: flow.af_cache_read(cache, 3, k=rows(2, 3, 2, 64, grad=grad), v=x)
    yield lambda: flow.af_cache_attention(cache, rows(2, 3, 2, 64, grad=grad), ints(3, 3))
    yield lambda: flow.af_cache_attention(cache, x, ints(3, 3), out=rows(2, 3, 2, 64, grad=grad))


def test_a_tensor_that_requires_grad_is_refused(flow, cache):
    for i, call in enumerate(calls(flow, cache, True)):
        with pytest.raises(ValueError, match="requires grad"):
            call()
            pytest.fail(f"call {i} was taken")


def test_it_is_taken_where_gradients_are_off(flow, cache):
    """Then the next complaint is another one: the tensors are not on a device, or there is none."""
    for grad in (True, False):
        with torch.no_grad():
            for call in calls(flow, cache, grad):
                with pytest.raises((ValueError, RuntimeError)) as e:
                    call()
                assert "requires grad" not in str(e.value)


def test_a_workspace_that_is_not_dense_is_refused(flow, cache):
    """A broadcast byte says that it has as many as it is asked for."""
    x = rows(2, 3, 2, 64)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(1 << 16, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="contiguous"):
            flow.af_cache_attention(cache, x, ints(3, 3), ws=ws)


@pytest.mark.parametrize("bad", [lambda n: torch.zeros(n - 1, dtype=torch.uint8),
                                 lambda n: torch.zeros(1, dtype=torch.uint8).expand(n),
                                 lambda n: torch.zeros(n, 2, dtype=torch.uint8)[:, 1]])
def test_a_storage_that_changed_after_the_handle_was_made_is_refused(flow, cache, bad):
    x = rows(2, 3, 2, 64)
    cache.storage = bad(cache.bytes)
    for call in (lambda: flow.af_cache_write(cache, x, x), lambda: flow.af_cache_read(cache, 3),
                 lambda: flow.af_cache_read(cache, 3, k=x, v=x.clone()), lambda: flow.af_cache_attention(cache, x, ints(3, 3))):
        with pytest.raises(ValueError, match="contiguous|needs"):
            call()
    cache.storage = torch.zeros(cache.bytes, dtype=torch.uint8)
    cache.storage.resize_(cache.bytes // 2)
    with pytest.raises(ValueError, match="needs"):
        flow.af_cache_write(cache, x, x)
