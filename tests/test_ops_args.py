"""Refusals of the attention-layer operators that need no device: every call below has one bad argument and returns
AF_ERR_ARG (or AF_ERR_WORKSPACE) with a message before anything is enqueued; the pointers are never read."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def flow():
    from video_generation_b200 import build
    build.build()
    from video_generation_b200 import flow as F
    return F


def _rejected(flow, status, expect=1):
    assert status == expect, flow.lib().af_status_string(status)
    assert flow.lib().af_last_error_string()


def _rope(flow, dim=64, pairs=(8, 12, 12), theta=1e4, layout=0, eps=1e-6):
    return ctypes.byref(flow.RopeC(theta, dim, (ctypes.c_int * 3)(*pairs), layout, eps))


P = 1 << 20                                        # an aligned address that no refused call reads


@pytest.mark.parametrize("bad", [
    dict(rope=dict(dim=48)), dict(rope=dict(dim=0)), dict(rope=dict(dim=512)), dict(rope=dict(pairs=(8, 12, 13))),
    dict(rope=dict(pairs=(-1, 12, 12))), dict(rope=dict(pairs=(2 ** 31 - 1, 2 ** 31 - 1, 12))),
    dict(rope=dict(theta=0.5)), dict(rope=dict(theta=float("nan"))), dict(rope=dict(theta=float("inf"))),
    dict(rope=dict(eps=0.0)), dict(rope=dict(eps=float("nan"))), dict(rope=dict(layout=2)), dict(rope=None),
    dict(dtype=2), dict(rows=-1), dict(rows=2 ** 30 + 1), dict(heads=-1), dict(kv_heads=65537),
    dict(q=0), dict(q=P + 2), dict(qs=60), dict(qs=-128), dict(qos=64), dict(qo=0), dict(qo=P + 8), dict(k=0),
    dict(ks=124), dict(kos=0), dict(ko=0), dict(pos=0), dict(qo=P, qos=256)])
def test_qk_norm_rope_refuses(flow, bad):
    a = dict(rope={}, dtype=1, rows=3, q=P, qs=128, heads=2, k=P + 1024, ks=128, kv_heads=2, pos=P, qo=P + 4096,
             qos=128, ko=P + 8192, kos=128)
    a.update(bad)
    rope = None if a["rope"] is None else _rope(flow, **a["rope"])
    _rejected(flow, flow.lib().af_qk_norm_rope(rope, a["dtype"], a["rows"], a["q"], a["qs"], a["heads"], a["k"],
                                               a["ks"], a["kv_heads"], None, None, a["pos"], a["qo"], a["qos"],
                                               a["ko"], a["kos"], None))


BAD_CONFIGS = [(-1, 2, 64, 100), (2, 0, 64, 100), (2, 2, 96, 100), (2, 2, 64, 0), (1 << 20, 1 << 10, 64, 100)]


@pytest.mark.parametrize("c", BAD_CONFIGS)
def test_cache_config_refused(flow, c):
    L, cfg = flow.lib(), ctypes.byref(flow.CacheConfigC(*c))
    assert L.af_cache_bytes(cfg) == 0
    assert L.af_cache_attention_workspace_bytes(cfg, 2, 1) == 0
    _rejected(flow, L.af_cache_write(cfg, P, 1, P, 256, 128, P, 256, 128, None, None, None))
    _rejected(flow, L.af_cache_read(cfg, P, 1, None, None, 1, P, 2 * P, 256, 128, None))
    _rejected(flow, L.af_cache_attention(cfg, P, 1, 2, P, 256, 128, P, None, 1, 0.1, 2 * P, 256, 128, P, 1 << 20, None))
    with pytest.raises(flow.AFError):
        flow.KVCache(*c, device="cpu")


def test_cache_bytes(flow):
    # five bits a value, each part on a 256-byte boundary
    assert flow.KVCache.needed(2, 3, 64, 100) == 2 * (19200 + 4864)
    assert flow.KVCache.needed(1, 16, 128, 46800) == 46800 * 16 * 2 * 80
    assert flow.KVCache.needed(0, 4, 64, 8) == 0
    import torch
    with pytest.raises(ValueError):
        flow.KVCache(1, 1, 64, 10, storage=torch.zeros(100, dtype=torch.uint8))
    with pytest.raises(ValueError):
        flow.KVCache(1, 1, 64, 10, storage=torch.zeros(10000, dtype=torch.int8))


def _cfg(flow):
    return ctypes.byref(flow.CacheConfigC(2, 2, 64, 100))


@pytest.mark.parametrize("bad", [
    dict(cache=0), dict(cache=P + 16), dict(rows=-1), dict(rows=2 ** 30 + 1), dict(k=0), dict(k=P + 2), dict(v=0),
    dict(v=P + 8), dict(krs=124), dict(krs=-128), dict(kbs=4), dict(vrs=1), dict(vbs=-8)])
def test_cache_write_refuses(flow, bad):
    a = dict(cache=P, rows=3, k=P, kbs=384, krs=128, v=P, vbs=384, vrs=128)
    a.update(bad)
    _rejected(flow, flow.lib().af_cache_write(_cfg(flow), a["cache"], a["rows"], a["k"], a["kbs"], a["krs"], a["v"],
                                              a["vbs"], a["vrs"], None, None, None))


@pytest.mark.parametrize("bad", [
    dict(cache=0), dict(cache=P + 128), dict(rows=-1), dict(dtype=2), dict(k=0), dict(k=P + 8), dict(v=0),
    dict(v=P + 4), dict(rs=64), dict(rs=130), dict(bs=120), dict(v=P)])
def test_cache_read_refuses(flow, bad):
    a = dict(cache=P, rows=3, dtype=1, k=P, v=2 * P, bs=384, rs=128)
    a.update(bad)
    _rejected(flow, flow.lib().af_cache_read(_cfg(flow), a["cache"], a["rows"], None, None, a["dtype"], a["k"], a["v"],
                                             a["bs"], a["rs"], None))


@pytest.mark.parametrize("bad,status", [
    (dict(cache=0), 1), (dict(cache=P + 32), 1), (dict(rows=-1), 1), (dict(heads=3), 1), (dict(heads=0), 1),
    (dict(rows=2 ** 20), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(q=0), 1), (dict(q=P + 8), 1), (dict(qrs=-256), 1), (dict(qbs=4), 1),
    (dict(out=0), 1), (dict(out=P), 1), (dict(out=2 * P + 8), 1), (dict(ors=128), 1), (dict(ors=260), 1),
    (dict(obs=128), 1), (dict(length=0), 1), (dict(ws=0), 3), (dict(ws=P + 128), 3)])
def test_cache_attention_refuses(flow, bad, status):
    a = dict(cache=P, rows=3, heads=4, q=P, qbs=768, qrs=256, length=P, scale=0.125, out=2 * P, obs=768, ors=256,
             ws=P, nb=1 << 20)
    a.update(bad)
    _rejected(flow, flow.lib().af_cache_attention(_cfg(flow), a["cache"], a["rows"], a["heads"], a["q"], a["qbs"],
                                                  a["qrs"], a["length"], None, 1, a["scale"], a["out"], a["obs"],
                                                  a["ors"], a["ws"], a["nb"], None), status)


def test_nothing_to_do_needs_no_device(flow):
    L = flow.lib()
    assert L.af_qk_norm_rope(_rope(flow), 1, 0, None, 0, 2, None, 0, 2, None, None, None, None, 0, None, 0, None) == 0
    assert L.af_qk_norm_rope(_rope(flow), 1, 5, None, 0, 0, None, 0, 0, None, None, None, None, 0, None, 0, None) == 0
    empty = ctypes.byref(flow.CacheConfigC(0, 2, 64, 100))
    for cfg, rows in ((_cfg(flow), 0), (empty, 5)):
        assert L.af_cache_write(cfg, P, rows, None, 0, 0, None, 0, 0, None, None, None) == 0
        assert L.af_cache_read(cfg, P, rows, None, None, 1, None, None, 0, 0, None) == 0
        assert L.af_cache_attention(cfg, P, rows, 2, None, 0, 0, None, None, 1, 0.1, None, 0, 0, None, 0, None) == 0


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_a_scale_whose_log2_units_are_not_finite_is_refused(flow, scale):
    """scale * log2(e) is what multiplies the scores: infinite, it would make NaN of a score of 0."""
    _rejected(flow, flow.lib().af_cache_attention(_cfg(flow), P, 3, 4, P, 768, 256, P, None, 1, scale, 2 * P, 768, 256, P,
                                                  1 << 20, None))
