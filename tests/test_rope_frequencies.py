"""Rotary frequencies of every scaling against their formulas, one pair at a
time in Python floats, with and without a GPU in the machine; on a GPU the
tables made from them as well."""
import math

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_22_b200 import binding as nb

KINDS = [dict(), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0), dict(scaling="linear", factor=0.5),
         dict(scaling="bands", factor=8.0, original_positions=8192.0, low=1.0, high=4.0),
         dict(scaling="bands", factor=32.0, original_positions=2048.0, low=2.0, high=2.5),
         dict(scaling="ramp", factor=16.0, original_positions=4096.0, low=1.0, high=32.0),
         dict(scaling="ramp", factor=40.0, original_positions=32768.0, low=0.5, high=64.0)]


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        from nvfp4_block_scaled_22_b200.build import build
        build()
    nb.lib()


def _formula(r, base, scaling="plain", factor=1.0, original_positions=0.0, low=1.0, high=32.0):
    if scaling == "ntk":
        base = base * factor ** (r / (r - 2))
    out = []
    for i in range(r // 2):
        f = base ** (-2 * i / r)
        kept = {"plain": 1.0, "ntk": 1.0, "linear": 0.0}.get(scaling)
        if scaling == "bands":
            turns = original_positions * f / (2 * math.pi)
            kept = (min(max(turns, low), high) - low) / (high - low)
        if scaling == "ramp":
            first, last = (r * math.log(original_positions / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (high, low))
            first, last = max(math.floor(first), 0), min(math.ceil(last), r - 1)
            kept = 1 - (min(max(i, first), last) - first) / (last - first)
        out.append(kept * f + (1 - kept) * f / factor)
    return np.array(out)


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: f"{k.get('scaling', 'plain')} {k.get('factor', 1)}")
@pytest.mark.parametrize("r,base", [(128, 1e4), (64, 5e5), (96, 1e6)])
def test_frequencies(kind, r, base):
    got = nb.nvfp4_rope_inv_freq(r, base, **kind).numpy()
    assert got.dtype == np.float64
    # a power (2 ulp or so of an exponent up to 14, twice), then a few operations: 2^-52 each
    assert np.allclose(got, _formula(r, base, **kind), rtol=64 * 2.0 ** -52, atol=0)


def test_refusals():
    for bad in (dict(rotary_dim=63), dict(rotary_dim=0), dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, base=float("nan")),
                dict(rotary_dim=64, scaling="linear", factor=0.0), dict(rotary_dim=2, scaling="ntk", factor=2.0),
                dict(rotary_dim=64, scaling="bands", factor=2.0), dict(rotary_dim=64, scaling="ramp", factor=2.0, original_positions=4096.0, low=4.0, high=4.0)):
        with pytest.raises(nb.NVFP4Error):
            nb.nvfp4_rope_inv_freq(**bad)
    with pytest.raises(ValueError, match="scaling"):
        nb.nvfp4_rope_inv_freq(64, scaling="none")


def test_host_tensors_are_refused():
    x, pos, table = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.zeros(8, 32, 2)
    cache = nb.NVFP4Tensor(torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(128, dtype=torch.uint8), torch.ones(1), 16, 128, nb.SF_LINEAR)
    for call in (lambda: nb.nvfp4_rope(x, pos, table), lambda: nb.nvfp4_kv_write(x, x, pos, cache, cache), lambda: nb.nvfp4_kv_read(cache, cache, pos),
                 lambda: nb.nvfp4_attention_decode_paged(x, cache, cache, 2, torch.zeros(4, 1, dtype=torch.int32), pos, 16)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: f"{k.get('scaling', 'plain')} {k.get('factor', 1)}")
def test_table_of_scaled_frequencies(kind):
    r, base, first, rows = 96, 5e5, 100_000, 700
    f = nb.nvfp4_rope_inv_freq(r, base, **kind)
    formula = _formula(r, base, **kind)
    assert np.allclose(f.numpy(), formula, rtol=64 * 2.0 ** -52, atol=0)
    got = nb.nvfp4_rope_table(f, rows, 1.0, first, "cuda").cpu().numpy()
    a = (first + np.arange(rows)).astype(np.longdouble)[:, None] * formula.astype(np.longdouble)
    want = np.stack([np.cos(a), np.sin(a)], -1)
    # FP32 once; the frequency's error above, the product's rounding and 2 ulp of sincos in 64 bits
    tol = 2.0 ** -24 * np.abs(want) + (np.abs(a) * 66 * 2.0 ** -52)[..., None] + 2.0 ** -51
    assert np.all(np.abs(got - want) <= tol)
