"""Paged decode attention where scores are far beyond what FP16 or a small
FP32 error can hold: the weights are then one token's, and stay finite."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_22_b200 import binding as nb
from tests import paged_ref as R
from tests.test_gpu_attention_paged import Cache, _query

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dim,heads,page", [(64, 4, 16), (128, 2, 16), (128, 1, 20), (256, 1, 16)])
@pytest.mark.parametrize("exponent", [24, 28, 40, 100])
def test_large_scores_choose_their_token(dim, heads, page, exponent):
    """A head's scores are off by eps_s (paged_ref.attention_bounds), so that
    the weights are those of its largest score where the next is 2 eps_s + 50
    less (what is left then, exp(-50) a token, is far below a BF16 step), and
    anything between the tokens' values elsewhere; BF16 rounds once."""
    cache = Cache([700, 1, 40], heads, dim, page, exponent)
    q = _query(3, heads * 8, dim, 50, 2.0 ** exponent)
    o, lse = cache.attend(q.to(DEV))
    chosen = 0
    for b, n in enumerate(cache.lens):
        k, v = cache.host[b]
        x = R.f64(q[b]).reshape(heads, -1, dim)
        _, want_lse, ao, sa = R.attention(x, k, v, dim ** -0.5)
        got = R.f64(o[b]).reshape(x.shape)
        low, high = (np.broadcast_to(m(v, 0)[:, None], got.shape) for m in (np.min, np.max))
        step = 2.0 ** -8 * np.maximum(np.abs(low), np.abs(high))
        assert np.all((got >= low - step) & (got <= high + step))
        s = np.einsum("hgd,thd->hgt", x, k) * dim ** -0.5
        eps = (8.5 * dim / 16 + 4) * R.U * sa
        order = np.sort(s, -1)
        clear = np.ones(eps.shape, bool) if n == 1 else order[..., -1] - order[..., -2] > 2 * eps + 50
        top = np.take_along_axis(v.transpose(1, 0, 2), s.argmax(-1)[..., None], 1)
        assert np.all(np.abs(got - top)[clear] <= (2.0 ** -8 * np.abs(top) + 1e-12)[clear])
        # the log of the sum: the score's error, and 4 roundings of it
        assert np.all(np.abs(R.f64(lse[b]).reshape(want_lse.shape) - want_lse) <= eps + 4 * R.U * np.abs(want_lse) + 1e-3)
        chosen += clear.sum()
    assert chosen > 0.9 * 3 * heads * 8
    assert nb.nvfp4_check_status() == 0


def test_scores_past_fp32_are_nan_in_their_head():
    cache = Cache([50, 60], 2, 128, 16, 51)
    q = _query(2, 8, 128, 52)
    q[0, 3] *= 2.0 ** 120                                  # times the scale: past 2^128, of either sign
    scale = 2.0 ** 10
    o, lse = cache.attend(q.to(DEV), scale=scale)
    bad = torch.zeros(2, 8, dtype=torch.bool)
    bad[0, 3] = True
    assert torch.isnan(o.float()).all(-1).cpu().equal(bad) and torch.isnan(lse).cpu().equal(bad)


@pytest.mark.parametrize("dim,heads", [(64, 4), (128, 2), (256, 1)])
@pytest.mark.parametrize("exponent", [-126, -128, -131])
def test_queries_of_subnormal_values(dim, heads, exponent):
    """What BF16 still holds of such a query, with a scale that brings its
    scores back to the order of one."""
    cache = Cache([300, 7], heads, dim, 16, 53)
    q = _query(2, heads * 8, dim, 54, 2.0 ** exponent)
    scale = 2.0 ** -exponent * dim ** -0.5 / 4
    o, lse = cache.attend(q.to(DEV), scale=scale)
    for b, n in enumerate(cache.lens):
        k, v = cache.host[b]
        want, wl, ao, sa = R.attention(R.f64(q[b]).reshape(heads, -1, dim), k, v, float(np.float32(scale)))
        ob, lb = R.attention_bounds(want, wl, ao, sa, n, dim, np.abs(v).max())
        assert np.ptp(wl) > 10 * lb.max()                      # scores that are all 0 would show
        assert np.all(np.abs(R.f64(o[b]).reshape(want.shape) - want) <= ob)
        assert np.all(np.abs(R.f64(lse[b]).reshape(wl.shape) - wl) <= lb)


@pytest.mark.parametrize("dim,heads,page", [(64, 4, 16), (128, 2, 20), (256, 1, 16)])
@pytest.mark.parametrize("exponent", [-100, 60, 61, 100, 118])
def test_value_scales_of_the_whole_range(dim, heads, page, exponent):
    """A tensor scale of V is up to 2^118 (nvfp4_quantize) and down to 2^-116
    (of BF16's largest values): a power of two in it is one in the output,
    for a sequence of one CTA and for one that is joined."""
    cache = Cache([9000, 20, 1], heads, dim, page, 55)
    q = _query(3, heads * 8, dim, 56)
    cache.v.global_scale.fill_(1.5)
    want, want_lse = cache.attend(q.to(DEV))
    cache.v.global_scale.fill_(0.75 * 2.0 ** exponent if exponent > 0 else 1.5 * 2.0 ** exponent)
    o, lse = cache.attend(q.to(DEV))
    factor = 2.0 ** (1 - exponent) if exponent > 0 else 2.0 ** -exponent
    # BF16 rounds less than 2^-126 to coarser steps (zeros are the many codes of 0 of the sequence of one token)
    normal = ((want.double() * factor).abs() >= 2.0 ** -126) | (want == 0)
    assert torch.equal((want.double() * factor)[normal], o.double()[normal]) and torch.equal(lse, want_lse)
    assert normal.double().mean() > 0.99
