"""The paged cache's write and read on the GPU, bit for bit against the
oracle: the bytes of a written row are those of quantizing the (rotated) row
with the pool's tensor scale, a row read back is the oracle's dequantize."""
import numpy as np
import pytest
import torch

import oracle
from nvfp4_block_scaled_22_b200 import binding as nb
from tests import paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _clean():
    nb.lib()
    yield
    assert nb.nvfp4_check_status() == 0


def _pool(rows, cols, seed, g=2688 / 6.0):
    """A pool of arbitrary earlier content."""
    t = nb.NVFP4Tensor.empty(rows, cols, nb.SF_LINEAR, DEV)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t.codes.copy_(torch.randint(0, 256, t.codes.shape, generator=gen, device=DEV, dtype=torch.uint8))
    t.scales.copy_(torch.randint(0, 127, t.scales.shape, generator=gen, device=DEV, dtype=torch.uint8))
    t.global_scale.fill_(g)
    return t


def _rows(t):
    return t.codes.cpu().numpy().copy(), t.scales.view(t.rows, -1).cpu().numpy().copy()


def _expect(before, x, slots, g):
    codes, scales = before[0].copy(), before[1].copy()
    keep = [i for i, s in enumerate(slots) if s >= 0]
    if keep:
        q = oracle.quantize_with_global(x[keep].reshape(len(keep), -1), g, oracle.SF_LINEAR)
        codes[[slots[i] for i in keep]] = q.codes
        scales[[slots[i] for i in keep]] = q.scales.reshape(len(keep), -1)
    return codes, scales


def _check(pool, want):
    got = _rows(pool)
    assert np.array_equal(got[1], want[1]), "scales"
    assert np.array_equal(got[0], want[0]), "codes"


def _tokens(n, heads, dim, seed, outliers=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, heads, dim))
    if outliers:
        x[..., :: 37] *= 10.0
    return R.bf16(x)


@pytest.mark.parametrize("tokens,heads,dim", [(1, 8, 128), (67, 8, 128), (130, 5, 64), (33, 1, 256), (9, 3, 48), (700, 2, 16)])
@pytest.mark.parametrize("rope", ["none", "half", "interleaved", "half quarter", "interleaved odd", "half odd"])
def test_write_then_read(tokens, heads, dim, rope):
    rng = np.random.default_rng(tokens + dim)
    rows = tokens + 50
    slots = rng.permutation(rows)[:tokens].astype(np.int32)
    slots[tokens // 2: tokens // 2 + tokens // 10] = -1                       # padding inside of the batch
    k, v = _tokens(tokens, heads, dim, 1), _tokens(tokens, heads, dim, 2)
    kc, vc = _pool(rows, heads * dim, 3, 300.0), _pool(rows, heads * dim, 4, 2688 / 45.0)
    before = _rows(kc), _rows(vc)
    args, rotated = {}, k
    if rope != "none":
        rotary = {"half": dim, "interleaved": dim, "half quarter": max(2, dim // 4), "interleaved odd": 6, "half odd": 10}[rope]
        pos = torch.from_numpy(rng.integers(0, 1000, tokens).astype(np.int32))
        table = nb.nvfp4_rope_table(nb.nvfp4_rope_inv_freq(rotary), 1000, device=DEV)
        inter = rope.startswith("interleaved")
        args = dict(positions=pos.to(DEV), table=table, interleaved=inter)
        cs = table.cpu().numpy()[pos.numpy()]
        rotated = torch.from_numpy(R.rope(k.float().numpy(), cs[..., 0], cs[..., 1], inter)).to(torch.bfloat16)
    dslots = torch.from_numpy(slots).to(DEV)
    nb.nvfp4_kv_write(k.to(DEV), v.to(DEV), dslots, kc, vc, **args)
    want = _expect(before[0], rotated, slots, 300.0), _expect(before[1], v, slots, 2688 / 45.0)
    _check(kc, want[0])
    _check(vc, want[1])
    got = nb.nvfp4_kv_read(kc, vc, dslots)
    for y, (codes, scales), g in zip(got, want, (300.0, 2688 / 45.0)):
        safe = np.maximum(slots, 0)
        ref = oracle.dequantize(np.ascontiguousarray(codes[safe]), np.ascontiguousarray(scales[safe]).ravel(), oracle.SF_LINEAR, g, tokens, heads * dim)
        ref = np.where(slots[:, None] >= 0, ref, np.uint16(0))
        assert np.array_equal(y.cpu().view(torch.int16).numpy().view(np.uint16), ref)


def test_written_bytes_are_those_of_quantize():
    """The whole-tensor entry point with the same tensor scale, outliers past
    the scale's range (saturated), zeros and subnormals among the values."""
    n, heads, dim = 64, 4, 128
    x = _tokens(n, heads, dim, 5).float()
    x[3] = 0.0
    x[4, :, ::2] = -0.0
    x[5] *= 1e-6
    x[6] *= 1e-39
    x[7] *= 1e4
    x = x.to(torch.bfloat16).to(DEV)
    kc, vc = _pool(n, heads * dim, 6, 448.0), _pool(n, heads * dim, 7, 448.0)
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    nb.nvfp4_kv_write(x, x, slots, kc, vc)
    ref = nb.NVFP4Tensor.empty(n, heads * dim, nb.SF_LINEAR, DEV)
    ref.global_scale.fill_(448.0)
    nb.nvfp4_quantize(x.view(n, -1), out=ref, layout=nb.SF_LINEAR, global_supplied=True)
    y = nb.nvfp4_dequantize(ref)
    for pool, got in zip((kc, vc), nb.nvfp4_kv_read(kc, vc, slots)):
        assert torch.equal(pool.codes, ref.codes) and torch.equal(pool.scales, ref.scales)
        assert torch.equal(R.bits(got), R.bits(y))


def test_fused_projection_strides_and_output_pitch():
    """k and v as slices of one projection [tokens, (q + k + v) heads, dim];
    rows read into a wider buffer, 16-byte but not 32-byte aligned."""
    n, heads, dim = 21, 2, 64
    fused = _tokens(n, 8 + 2 * heads, dim, 8).to(DEV)
    k, v = fused[:, 8:8 + heads], fused[:, 8 + heads:]
    kc, vc = _pool(40, heads * dim, 9), _pool(40, heads * dim, 10)
    slots = torch.arange(39, 39 - n, -1, dtype=torch.int32, device=DEV)
    before = _rows(kc), _rows(vc)
    nb.nvfp4_kv_write(k, v, slots, kc, vc)
    s = slots.cpu().numpy()
    _check(kc, _expect(before[0], k.cpu().contiguous(), s, 2688 / 6.0))
    _check(vc, _expect(before[1], v.cpu().contiguous(), s, 2688 / 6.0))
    ref = nb.nvfp4_kv_read(kc, vc, slots)
    wide = [torch.full((n, heads * dim + 16), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    nb.nvfp4_kv_read(kc, vc, slots, out=tuple(w[:, 8:8 + heads * dim] for w in wide))
    for w, r in zip(wide, ref):
        assert torch.equal(R.bits(w[:, 8:-8]), R.bits(r))
        assert (w[:, :8] == 3).all() and (w[:, -8:] == 3).all()


def test_bad_slots_positions_and_values_are_recorded():
    n, heads, dim = 8, 2, 64
    x = _tokens(n, heads, dim, 11)
    ws = nb.Workspace(DEV, 256)
    table = nb.nvfp4_rope_table(nb.nvfp4_rope_inv_freq(dim), 10, device=DEV)
    for slot, position, status in [(16, 3, 1), (-2, 3, 1), (2 ** 31 - 1, 3, 1), (5, 10, 1), (5, -1, 0), (5, -7, 1)]:
        kc, vc = _pool(16, heads * dim, 12), _pool(16, heads * dim, 13)
        before = _rows(kc), _rows(vc)
        slots = np.arange(n, dtype=np.int32)
        pos = np.zeros(n, np.int32)
        slots[5], pos[5] = slot, position
        nb.nvfp4_kv_write(x.to(DEV), x.to(DEV), torch.from_numpy(slots).to(DEV), kc, vc, torch.from_numpy(pos).to(DEV), table, workspace=ws)
        assert nb.nvfp4_check_status(ws) == status, (slot, position)
        slots[5] = -1
        _check(kc, _expect(before[0], x, slots, 2688 / 6.0))                   # position 0: the rotation is the identity
        _check(vc, _expect(before[1], x, slots, 2688 / 6.0))
    out = nb.nvfp4_kv_read(kc, vc, torch.tensor([0, 16, -1, -9], dtype=torch.int32, device=DEV), workspace=ws)
    assert nb.nvfp4_check_status(ws) == 1
    assert not out[0][1:].any() and not out[1][1:].any() and out[0][0].any()
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[2, 1, 20] = bad
        kc, vc = _pool(16, heads * dim, 12), _pool(16, heads * dim, 13)
        before = _rows(kc)
        slots = np.arange(n, dtype=np.int32)
        nb.nvfp4_kv_write(y.to(DEV), x.to(DEV), torch.from_numpy(slots).to(DEV), kc, vc, workspace=ws)
        assert nb.nvfp4_check_status(ws) == 4
        want, got = _expect(before, x, slots, 2688 / 6.0), _rows(kc)
        blk = dim // 16 + 1
        got[0][2, 8 * blk:8 * blk + 8], got[1][2, blk] = want[0][2, 8 * blk:8 * blk + 8], want[1][2, blk]
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])     # only that block differs


def test_rows_past_32_bit_offsets():
    """The last rows of a pool whose codes pass 4 GiB."""
    heads, dim = 32, 256
    cols = heads * dim
    rows = (1 << 32) // (cols // 2) + 40
    kc = nb.NVFP4Tensor(torch.zeros(rows, cols // 2, dtype=torch.uint8, device=DEV), torch.zeros(rows * cols // 16, dtype=torch.uint8, device=DEV),
                        torch.full((1,), 448.0, device=DEV), rows, cols, nb.SF_LINEAR)
    x = _tokens(3, heads, dim, 14)
    slots = np.array([rows - 1, 7, rows - 33], np.int32)
    d = torch.from_numpy(slots).to(DEV)
    nb.nvfp4_kv_write(x.to(DEV), x.to(DEV), d, kc, kc)
    q = oracle.quantize_with_global(x.reshape(3, -1), 448.0, oracle.SF_LINEAR)
    scales = kc.scales.view(rows, -1)
    assert np.array_equal(kc.codes[d.long()].cpu().numpy(), q.codes)
    assert np.array_equal(scales[d.long()].cpu().numpy().ravel(), q.scales)
    assert int((scales.any(dim=1)).sum()) == 3                                 # and no other row
    got = nb.nvfp4_kv_read(kc, kc, d)[1].cpu().view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(got, q.dequantize())


def test_empty_calls_and_binding_refusals():
    kc, vc = _pool(16, 128, 15), _pool(16, 128, 16)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    x = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    nb.nvfp4_kv_write(x, x, none, kc, vc)
    nb.nvfp4_kv_write(x, x, none, kc, vc, positions=none, table=torch.zeros(4, 32, 2, device=DEV))
    assert nb.nvfp4_kv_read(kc, vc, none)[0].shape == (0, 128)
    x, slots = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="slots"):
        nb.nvfp4_kv_write(x, x, slots.long(), kc, vc)
    with pytest.raises(ValueError, match="v:"):
        nb.nvfp4_kv_write(x, x[:2], slots, kc, vc)
    with pytest.raises(ValueError, match="positions"):
        nb.nvfp4_kv_write(x, x, slots, kc, vc, table=torch.zeros(4, 32, 2, device=DEV))
    with pytest.raises(ValueError, match="linear"):
        t = nb.NVFP4Tensor.empty(16, 128, nb.SF_SWIZZLED, DEV)
        nb.nvfp4_kv_write(x, x, slots, t, vc)
    with pytest.raises(ValueError, match="codes"):
        t = nb.NVFP4Tensor(kc.codes[:8], kc.scales, kc.global_scale, 16, 128, nb.SF_LINEAR)
        nb.nvfp4_kv_read(kc, t, slots)
    with pytest.raises(ValueError, match="out"):
        nb.nvfp4_kv_read(kc, vc, slots, out=(torch.zeros(3, 64, dtype=torch.bfloat16, device=DEV),) * 2)
    with pytest.raises(nb.NVFP4Error):                                          # 3 heads of 64 in a pool of 2
        y = torch.zeros(3, 3, 64, dtype=torch.bfloat16, device=DEV)
        nb.nvfp4_kv_write(y, y, slots, kc, vc)
