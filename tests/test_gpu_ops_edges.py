"""Attention over the 4-bit cache at the edges of its arithmetic, whichever kernel a call goes to."""
import math

import numpy as np
import pytest
import torch

from tests import ops_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def flow():
    from video_generation_b200 import build
    build.build()
    from video_generation_b200 import flow as F
    assert torch.cuda.is_available()
    return F


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def exact_rows(cache, q, length, causal):
    """ops_util.attention64 on the device, all rows of a sequence and head at once: (out, tolerance)."""
    B, R, H, D = q.shape
    k, v = (torch.from_numpy(x).cuda() for x in U.cache_values(cache.storage, B, cache.kv_heads, D, cache.capacity))
    out, tol = torch.zeros(B, R, H, D, dtype=torch.float64, device="cuda"), torch.zeros(B, R, H, D, dtype=torch.float64, device="cuda")
    scale = D ** -0.5
    for b, L in enumerate(length):
        for h in range(H):
            x, K, V = q[b, :, h].double(), k[b, h // (H // cache.kv_heads), :L], v[b, h // (H // cache.kv_heads), :L]
            s = x @ K.T * scale
            if causal:
                s.masked_fill_(torch.arange(L, device="cuda") > torch.arange(L - R, L, device="cuda")[:, None], -math.inf)
            w = torch.softmax(s, 1)
            d = scale * (U.HALF_BF16 * (x.abs() @ K.abs().T) +
                         64 * U.HALF_FP32 * (x.abs() @ (K.abs() + 5 * K.abs().amax(1, keepdim=True)).T))
            e = 2 * torch.expm1(2 * d) + 2 * U.HALF_BF16
            out[b, :, h] = w @ V
            tol[b, :, h] = (U.HALF_BF16 + (w * e).sum(1, keepdim=True)) * out[b, :, h].abs() + (w * e) @ V.abs() + 1e-30
    return out, tol


# ------------------------------------------------------------------ rows without a finite score

def _signed_keys(B, cap, H, D, sign, seed):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(B, cap, H, D, generator=g)
    k[..., 5] = sign * (1 + k[..., 5].abs())
    return k.bfloat16().cuda(), torch.randn(B, cap, H, D, generator=g).bfloat16().cuda()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,cap", [(1, 60), (1, 3000), (9, 3000), (40, 9000), (100, 9000), (300, 700), (300, 9000)])
@pytest.mark.parametrize("causal", [True, False])
def test_a_row_whose_scores_are_all_minus_infinity_is_nan(flow, D, rows, cap, causal):
    """softmax of scores that are all -inf is NaN, not the zeros of a row that attends nothing: an infinite query
    channel against keys of one sign, in the first row (few keys) and the last.  The other rows are what they are
    without it, within their roundings (not bit for bit: next to a row with a NaN the tensor core's sums are rounded a
    little differently)."""
    B, H = 2, 2
    for sign in (1.0, -1.0):
        cache = flow.KVCache(B, H, D, cap)
        flow.af_cache_write(cache, *_signed_keys(B, cap, H, D, sign, rows))
        q = torch.randn(B, rows, H, D, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
        want, tol = exact_rows(cache, q, [cap, rows], causal)
        hit = torch.zeros(B, rows, H, dtype=torch.bool, device="cuda")
        for r, value in ((0, math.inf), (0, -math.inf), (rows - 1, math.inf), (rows - 1, -math.inf)):
            x = q.clone()
            x[:, r, 1, 5] = value
            got = flow.af_cache_attention(cache, x, ints([cap, rows]), causal=causal)
            hit.zero_()
            hit[:, r, 1] = True
            assert torch.isnan(got[hit]).all()
            assert ((got.double() - want).abs() <= tol)[~hit].all()
        # with no key to attend it stays zero, whatever the row holds
        x = q.clone()
        x[:, :, :, 5] = -math.inf
        assert (flow.af_cache_attention(cache, x, ints([0, 0]), causal=causal) == 0).all()


# ------------------------------------------------------------------ queries with channels far above the others

def _grid_rows(n, D, seed, silent):
    """Key rows [n, D] that the cache holds exactly: multiples of 1/4 in -2 .. 7/4, both ends in every group of 32, and
    0 (a code in the middle of the grid) in the `silent` channels."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(0, 16, (n, D // 32, 32), generator=g)
    ends = torch.stack([torch.randperm(31, generator=g)[:2] + 1 for _ in range(n * D // 32)]).view(n, D // 32, 2)
    x.scatter_(2, ends, torch.tensor([0, 15]).expand(n, D // 32, 2))
    x = (x.flatten(1) - 8) / 4
    x[:, silent] = 0
    return x


# (the silent channels are the first of their groups, which never hold a group's ends)
@pytest.mark.parametrize("size", [1.0, 100.0, 1000.0, 30000.0])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,cap", [(1, 2000), (5, 700), (8, 333), (13, 2000), (16, 130), (40, 700), (200, 1300)])
def test_a_channel_far_above_the_others(flow, D, rows, cap, size):
    """The keys say nothing in the channel, so what it costs is what the others lose beside it.  Keys are exact here; the
    output, the weights and the values are rounded to bf16, independently, each with an rms of 2^-8 / sqrt(3) at most:
    0.004 of the output together, and the bound of the other attention tests, 0.006, holds whatever the channel's size."""
    k = _grid_rows(cap, D, rows, [0, D - 32])[None, :, None].bfloat16()
    v = torch.randn(1, cap, 1, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    q = torch.randn(1, rows, 1, D, generator=torch.Generator().manual_seed(4))
    q[..., 0] = size
    q[:, ::2, :, D - 32] = -size
    q = q.bfloat16().cuda()
    cache = flow.KVCache(1, 1, D, cap)
    flow.af_cache_write(cache, k.cuda(), v.cuda())
    K, V = U.cache_values(cache.storage, 1, 1, D, cap)
    np.testing.assert_array_equal(K[0, 0], k[0, :, 0].double().numpy())
    ref, tol = U.attention64(q, K, V, [cap], None, True, D ** -0.5)
    got = flow.af_cache_attention(cache, q, ints([cap])).double().cpu().numpy()
    err = np.abs(got - ref)
    assert (err <= tol).all()
    assert np.linalg.norm(err) <= 6e-3 * np.linalg.norm(ref), np.linalg.norm(err) / np.linalg.norm(ref)


@pytest.mark.parametrize("D", [64, 128])
def test_a_query_does_not_depend_on_the_rows_beside_it(flow, D):
    """One query alone (few-row kernel) and as the last of many (tensor cores): both within the roundings of the other."""
    cap, rows = 4000, 300
    g = torch.Generator().manual_seed(8)
    cache = flow.KVCache(1, 2, D, cap)
    flow.af_cache_write(cache, _grid_rows(2 * cap, D, 5, [0]).view(1, cap, 2, D).bfloat16().cuda(),
                        torch.randn(1, cap, 2, D, generator=g).bfloat16().cuda())
    q = torch.randn(1, rows, 2, D, generator=g)
    q[..., 0] = 700.0
    q = q.bfloat16().cuda()
    many = flow.af_cache_attention(cache, q, ints([cap]))[:, -1:].double()
    one = flow.af_cache_attention(cache, q[:, -1:].contiguous(), ints([cap])).double()
    assert (many - one).norm() <= 2 * 6e-3 * many.norm()


# ------------------------------------------------------------------ waits past the limit

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [100, 300])                # 128 rows a CTA and 256
def test_a_wait_past_the_limit_is_given_up_and_reported(flow, D, rows):
    """Calls long enough that some wait is not over when it is first looked at: with a limit of a nanosecond one gives up
    (code 4), the CTAs drain (never code 2) and end, and the next call is as before."""
    H, cap = 16, 46800
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = flow.KVCache(1, H, D, cap)
    flow.af_cache_write(cache, *(torch.randn(1, cap, H, D, generator=g, device="cuda").bfloat16() for _ in range(2)))
    q = torch.randn(1, rows, H, D, generator=g, device="cuda").bfloat16()
    want = flow.af_cache_attention(cache, q, ints([cap]))
    assert flow.operator_error() == 0
    flow.operator_wait_limit(1e-9)
    try:
        codes = []
        for _ in range(8):
            flow.af_cache_attention(cache, q, ints([cap]))
            codes.append(flow.operator_error())
    finally:
        flow.operator_wait_limit(2.0)
    assert set(codes) <= {0, 4} and 4 in codes
    assert torch.equal(flow.af_cache_attention(cache, q, ints([cap])), want)
    assert flow.operator_error() == 0
