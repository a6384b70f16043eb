"""Host side of the paged-cache operators: rotary frequencies, refusals before
any CUDA call, and the binding's argument checks.  No kernel runs."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_22_b200 import binding as nb
from nvfp4_block_scaled_22_b200.build import build

OK, ARG, ALIGN, SHAPE, WS = 0, 1, 2, 3, 6
DEVICE = (8, 9)                 # checks passed, then no usable device here


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("the calls' pointers are made up: only for a host without a GPU")
    build()
    return nb.lib()


def _plain(r, base=1e4):
    return base ** (-2.0 * np.arange(r // 2) / r)


# ------------------------------------------------------------ frequencies
@pytest.mark.parametrize("r", [2, 6, 64, 128])
def test_plain_linear_and_ntk_frequencies(lib, r):
    f = nb.nvfp4_rope_inv_freq(r, 1e4).numpy()
    assert np.allclose(f, _plain(r), rtol=1e-14, atol=0)
    lin = nb.nvfp4_rope_inv_freq(r, 1e4, "linear", factor=8.0).numpy()
    assert np.allclose(lin, _plain(r) / 8, rtol=1e-14, atol=0)
    if r > 2:
        ntk = nb.nvfp4_rope_inv_freq(r, 1e4, "ntk", factor=4.0).numpy()
        # the first pair keeps its frequency, the last is divided by the factor
        assert ntk[0] == 1.0
        assert np.isclose(ntk[-1], _plain(r)[-1] / 4, rtol=1e-12)


def test_bands_keep_fast_pairs_and_divide_slow_ones(lib):
    r, length, s, low, high = 128, 8192, 8.0, 1.0, 4.0
    f = nb.nvfp4_rope_inv_freq(r, 5e5, "bands", s, length, low, high).numpy()
    p = _plain(r, 5e5)
    for i in range(r // 2):
        turns = length * p[i] / (2 * math.pi)
        if turns >= high:
            want = p[i]
        elif turns <= low:
            want = p[i] / s
        else:
            a = (turns - low) / (high - low)
            want = a * p[i] + (1 - a) * p[i] / s
        assert math.isclose(f[i], want, rel_tol=1e-13), i


def test_ramp_runs_between_two_pairs(lib):
    r, length, s, base = 128, 4096, 16.0, 1e4
    f = nb.nvfp4_rope_inv_freq(r, base, "ramp", s, length, 1.0, 32.0).numpy()
    p = _plain(r, base)

    def pair_of(turns):
        return r * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))

    i0, i1 = max(math.floor(pair_of(32)), 0), min(math.ceil(pair_of(1)), r - 1)
    for i in range(r // 2):
        g = min(max((i - i0) / (i1 - i0), 0.0), 1.0)
        assert math.isclose(f[i], p[i] * (1 - g) + p[i] / s * g, rel_tol=1e-13), i


def test_frequency_refusals(lib):
    out = (C.c_double * 64)()

    def call(r=128, base=1e4, kind=0, factor=2.0, length=4096.0, low=1.0, high=4.0, to=out):
        return lib.nvfp4_rope_inv_freq(r, base, kind, factor, length, low, high, to)

    assert call() == OK
    assert call(to=None) == ARG
    assert call(r=127) == SHAPE and call(r=0) == SHAPE and call(r=-2) == SHAPE
    assert call(kind=5) == ARG and call(kind=-1) == ARG
    assert call(base=1.0) == ARG and call(base=float("nan")) == ARG and call(base=float("inf")) == ARG
    assert call(kind=1, factor=0.0) == ARG and call(kind=1, factor=float("nan")) == ARG
    assert call(r=2, kind=2) == SHAPE
    assert call(kind=3, length=0.0) == ARG and call(kind=3, low=4.0) == ARG
    assert call(kind=4, high=float("inf")) == ARG
    with pytest.raises(ValueError, match="scaling"):
        nb.nvfp4_rope_inv_freq(64, 1e4, "other")


# --------------------------------------------------------------- refusals
def test_table_refusals(lib):
    def call(f=16, r=64, first=0, rows=10, m=1.0, t=16):
        return lib.nvfp4_rope_table(f, r, first, rows, m, t, None)

    assert call() in DEVICE
    assert call(rows=0, f=0, t=0) == OK
    assert call(r=63) == SHAPE and call(rows=-1) == ARG and call(first=-1) == ARG
    assert call(first=2 ** 31 - 5) == ARG and call(rows=2 ** 31) == ARG
    assert call(m=float("inf")) == ARG
    assert call(f=0) == ARG and call(t=0) == ARG
    assert call(f=20) == ALIGN and call(t=24) == ALIGN


def test_rope_refusals(lib):
    def call(x=16, xt=256, xh=128, n=4, h=2, d=128, pos=16, tab=16, rows=10, r=128, inter=0, inv=0,
             y=4096, yt=256, yh=128, ws=16, wsn=256):
        return lib.nvfp4_rope(x, xt, xh, n, h, d, pos, tab, rows, r, inter, inv, y, yt, yh, ws, wsn, None)

    assert call() in DEVICE
    assert call(n=0) == OK and call(h=0) == OK
    assert call(n=-1) == ARG and call(xt=-8) == ARG and call(yh=-8) == ARG
    assert call(inter=2) == ARG and call(inv=-1) == ARG and call(rows=0) == ARG
    assert call(r=130) == SHAPE and call(r=63) == SHAPE and call(r=0) == SHAPE
    assert call(x=0) == ARG and call(y=0) == ARG and call(pos=0) == ARG and call(tab=0) == ARG
    assert call(x=17) == ALIGN and call(tab=24) == ALIGN and call(pos=18) == ALIGN
    assert call(ws=0) == WS and call(wsn=255) == WS
    # output rows that overlap: heads, tokens, or heads of one token in the next
    assert call(yh=64) == SHAPE and call(yt=0) == SHAPE and call(yt=130) == SHAPE
    assert call(xt=0, xh=0) in DEVICE                       # an input may repeat
    assert call(yt=128, yh=512) in DEVICE                   # head-major output
    assert call(y=16) in DEVICE                             # in place
    assert call(y=16, yt=512) == ARG                        # "in place" with other strides
    assert call(n=2 ** 31, h=2 ** 20, yt=2 ** 28) == SHAPE  # too many items


def _pools(rows=64, cols=256, layout=1, p=16):
    return nb.CTensor(p, p, 16, rows, cols, layout)


def test_write_refusals(lib):
    def call(k=16, kt=256, kh=128, v=8192, vt=256, vh=128, n=4, h=2, d=128, slots=16, K=None, V=None,
             pos=16, tab=16, rows=10, r=128, inter=0, ws=16, wsn=256):
        return lib.nvfp4_kv_write(k, kt, kh, v, vt, vh, n, h, d, slots, K or _pools(), V or _pools(), pos,
                                  tab, rows, r, inter, ws, wsn, None)

    assert call() in DEVICE and call(tab=0, pos=0, r=0) in DEVICE
    assert call(n=0) == OK and call(n=0, k=0, v=0, slots=0, pos=0) == OK
    assert call(n=-1) == ARG and call(h=0) == ARG and call(kt=-8) == ARG
    assert call(d=120) == SHAPE and call(h=3) == SHAPE
    assert call(K=_pools(layout=0)) == SHAPE and call(V=_pools(rows=32)) == SHAPE
    assert call(K=nb.CTensor(16, 16, 0, 64, 256, 1)) == ARG
    assert call(k=0) == ARG and call(slots=0) == ARG
    assert call(k=24) == ALIGN and call(kt=260) == ALIGN and call(slots=18) == ALIGN
    assert call(pos=0) == ARG and call(r=130) == SHAPE and call(tab=20) == ALIGN
    assert call(wsn=100) == WS
    assert call(n=2 ** 31) == SHAPE


def test_read_refusals(lib):
    def call(K=None, V=None, slots=16, rows=8, k=16, ldk=256, v=8192, ldv=256, ws=16, wsn=256):
        return lib.nvfp4_kv_read(K or _pools(), V or _pools(), slots, rows, k, ldk, v, ldv, ws, wsn, None)

    assert call() in DEVICE
    assert call(rows=0, slots=0, k=0, v=0) == OK
    assert call(rows=-1) == ARG and call(slots=0) == ARG and call(v=0) == ARG
    assert call(k=24) == ALIGN and call(ldv=260) == ALIGN
    assert call(ldk=248) == SHAPE and call(K=_pools(layout=0)) == SHAPE and call(rows=2 ** 31) == SHAPE
    assert call(ws=0) == WS
    assert call(v=16) == ARG                                # one output for both


def test_attention_refusals(lib):
    big = 1 << 30

    def call(q=16, qb=512, qh=128, n=4, hq=4, K=None, V=None, hk=2, bt=16, bts=8, pages=8, lens=16, page=16,
             scale=0.1, o=8192, ob=512, oh=128, lse=16, ws=16, wsn=256, sc=16, scn=big):
        return lib.nvfp4_attention_decode_paged(q, qb, qh, n, hq, K or _pools(), V or _pools(), hk, bt, bts,
                                                pages, lens, page, scale, o, ob, oh, lse, ws, wsn, sc, scn, None)

    assert call() in DEVICE and call(lse=0) in DEVICE
    assert call(n=0) == OK
    assert call(n=-1) == ARG and call(hq=0) == ARG and call(hk=0) == ARG and call(page=0) == ARG
    assert call(scale=float("nan")) == ARG and call(scale=float("inf")) == ARG
    assert call(hq=5) == SHAPE and call(hk=1, hq=2, oh=256) in DEVICE and call(hk=4) in DEVICE
    assert call(hk=8, hq=8) == SHAPE                                     # head_dim 32
    assert call(page=24) == SHAPE                                        # 64 rows are no whole pages
    assert call(bts=4) == SHAPE and call(n=1, bts=0) in DEVICE
    assert call(pages=2 ** 28) == SHAPE                                  # more tokens than 31 bits count
    assert call(K=_pools(layout=0)) == SHAPE and call(V=_pools(rows=32)) == SHAPE
    assert call(q=0) == ARG and call(o=0) == ARG and call(lens=0) == ARG and call(bt=0) == ARG
    assert call(pages=0, bt=0) in DEVICE                                 # no pages: every sequence is empty
    assert call(q=24) == ALIGN and call(qb=516) == ALIGN and call(lens=18) == ALIGN and call(lse=18) == ALIGN
    assert call(ob=0) == SHAPE and call(oh=64) == SHAPE and call(qb=0, qh=0) in DEVICE
    assert call(o=16) in DEVICE and call(n=1, o=16, ob=1024) in DEVICE   # in place
    assert call(o=16, ob=1024) == ARG and call(o=16, oh=256, ob=1024) == ARG
    assert call(hq=2 ** 16, qb=2 ** 23, ob=2 ** 23) == SHAPE
    assert lib.nvfp4_attention_paged_scratch_bytes(2 ** 16, 1, 128) == 0
    assert call(wsn=10) == WS
    need = lib.nvfp4_attention_paged_scratch_bytes(4, 2, 128)
    if need:
        assert call(scn=need - 1) == WS and call(scn=need) in DEVICE and call(sc=0) == WS
        assert call(sc=24) == ALIGN


def test_binding_refuses_host_tensors_and_wrong_types(lib):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pos, table = torch.zeros(4, dtype=torch.int32), torch.zeros(8, 32, 2)
    with pytest.raises(ValueError, match="CUDA"):
        nb.nvfp4_rope(x, pos, table)
    with pytest.raises(ValueError, match="BF16"):
        nb.nvfp4_rope(x.float(), pos, table)
    cache = nb.NVFP4Tensor(torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(16 * 8, dtype=torch.uint8),
                           torch.ones(1), 16, 128, nb.SF_LINEAR)
    with pytest.raises(ValueError, match="CUDA"):
        nb.nvfp4_kv_write(x, x, pos, cache, cache)
    with pytest.raises(ValueError, match="CUDA"):
        nb.nvfp4_kv_read(cache, cache, pos)
    with pytest.raises(ValueError, match="CUDA"):
        nb.nvfp4_attention_decode_paged(x, cache, cache, 2, torch.zeros(4, 1, dtype=torch.int32), pos, 16)
