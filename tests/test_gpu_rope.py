"""Rotary positions on the GPU: the table against 80-bit angles, the rotation
bit for bit against the same FP32 operations in numpy, within rounding of the
64-bit formula, and its inverse as the gradient.

Bound against the formula: cos and sin are rounded once (2^-24 of each), so
are both products and their sum, which adds up to at most 4 * 2^-24 of |x1| +
|x2| (|cos|, |sin| <= 1); BF16 then takes 2^-8 of the result."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_22_b200 import binding as nb
from tests import paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _clean():
    nb.lib()
    yield
    assert nb.nvfp4_check_status() == 0


def _case(tokens, heads, dim, rotary, seed, far=131072):
    rng = np.random.default_rng(seed)
    x = R.bf16(rng.standard_normal((tokens, heads, dim)))
    pos = torch.from_numpy(rng.integers(0, far, tokens).astype(np.int32))
    table = nb.nvfp4_rope_table(nb.nvfp4_rope_inv_freq(rotary, 1e4), far, device=DEV)
    return x, pos, table


def _same_steps(x, pos, table, interleaved, inverse=False):
    cs = table.cpu().numpy()[pos.numpy()]
    y = R.rope(x.float().numpy(), cs[..., 0], cs[..., 1], interleaved, inverse)
    assert y.dtype == np.float32
    return torch.from_numpy(y).to(torch.bfloat16)


@pytest.mark.parametrize("rotary,first,rows,magnitude", [(128, 0, 1000, 1.0), (64, 1 << 20, 77, 1.25),
                                                         (2, 2 ** 31 - 8, 7, 1.0), (20, 5, 1, 0.5)])
def test_table_against_extended_precision(rotary, first, rows, magnitude):
    f = nb.nvfp4_rope_inv_freq(rotary, 1e4)
    got = nb.nvfp4_rope_table(f, rows, magnitude, first, DEV).cpu().numpy()
    a = (first + np.arange(rows)).astype(np.longdouble)[:, None] * f.numpy().astype(np.longdouble)
    want = np.stack([np.cos(a), np.sin(a)], -1) * np.longdouble(magnitude)
    # the angle's own rounding in FP64 (2^-53 of it), 2 ulp of sincos, then FP32
    tol = 2.0 ** -24 * np.abs(want) + magnitude * (np.abs(a)[..., None] * 2.0 ** -52 + 2.0 ** -51)
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("tokens,heads,dim,rotary", [
    (1, 1, 128, 128), (3, 72, 128, 128), (37, 5, 64, 64), (130, 8, 256, 128), (9, 3, 128, 16), (5, 7, 64, 2),
    (11, 4, 80, 40), (6, 2, 96, 20), (4, 3, 10, 6), (2, 1, 129, 128), (1000, 40, 128, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_matches_formula_and_steps(tokens, heads, dim, rotary, interleaved):
    x, pos, table = _case(tokens, heads, dim, rotary, tokens * 7 + dim, far=4096)
    y = nb.nvfp4_rope(x.to(DEV), pos.to(DEV), table, interleaved)
    assert torch.equal(R.bits(y.cpu()), R.bits(_same_steps(x, pos, table, interleaved)))
    a = pos.numpy()[:, None] * R.inv_freq(rotary, 1e4)
    exact = R.rope(R.f64(x), np.cos(a), np.sin(a), interleaved)
    slack = 4 * R.U * R.turned_bound(R.f64(x), rotary, interleaved)
    assert np.all(np.abs(R.f64(y) - exact) <= 2.0 ** -8 * (np.abs(exact) + slack) + slack)


@pytest.mark.parametrize("tokens,heads,dim,rotary", [
    (9, 5, 128, 2), (7, 6, 64, 54), (5, 9, 256, 206), (6, 1, 72, 38), (300, 3, 128, 30), (2, 4, 8, 2), (3, 5, 16, 14),
    (4, 8, 128, 126), (8, 2, 24, 20), (2, 3, 8, 8), (5, 7, 256, 250)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_pair_counts_that_cut_a_piece(tokens, heads, dim, rotary, interleaved):
    """Rotated parts that end inside of 16 bytes: apart, inverse, in place,
    head-major, and with what is not finite kept to its pair."""
    x, pos, table = _case(tokens, heads, dim, rotary, dim + rotary, far=4096)
    x[0, 0, dim - 1], x[-1, -1, 0] = float("nan"), float("inf")
    want = _same_steps(x, pos, table, interleaved)

    def same(got, want):
        nan = torch.isnan(want.float())
        return torch.equal(torch.isnan(got.float()), nan) and torch.equal(R.bits(got)[~nan], R.bits(want)[~nan])

    d = x.to(DEV)
    assert same(nb.nvfp4_rope(d, pos.to(DEV), table, interleaved).cpu(), want)
    assert same(nb.nvfp4_rope(d, pos.to(DEV), table, interleaved, inverse=True).cpu(), _same_steps(x, pos, table, interleaved, True))
    flip = torch.empty(heads, tokens, dim, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    assert same(nb.nvfp4_rope(d, pos.to(DEV), table, interleaved, out=flip).cpu(), want)
    assert same(nb.nvfp4_rope(d, pos.to(DEV), table, interleaved, out=d).cpu(), want)


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    """<R x, g> = <x, R^T g>, against differences of the formula as well."""
    tokens, heads, dim, rotary = 5, 3, 64, 32
    x, pos, table = _case(tokens, heads, dim, rotary, 3, far=512)
    g = R.bf16(np.random.default_rng(4).standard_normal((tokens, heads, dim)))
    gx = nb.nvfp4_rope(g.to(DEV), pos.to(DEV), table, interleaved, inverse=True)
    assert torch.equal(R.bits(gx.cpu()), R.bits(_same_steps(g, pos, table, interleaved, True)))
    a = pos.numpy()[:, None] * R.inv_freq(rotary, 1e4)
    c, s = np.cos(a), np.sin(a)

    def loss(v):
        return (R.rope(v, c, s, interleaved) * R.f64(g)).sum()

    x0, want = R.f64(x), np.zeros((tokens, heads, dim))
    for at in np.ndindex(tokens, heads, dim):          # the loss is linear: a difference is exact but for rounding
        d = np.zeros_like(x0)
        d[at] = 0.5
        want[at] = loss(x0 + d) - loss(x0 - d)
    slack = 4 * R.U * R.turned_bound(R.f64(g), rotary, interleaved) + 1e-11
    assert np.all(np.abs(R.f64(gx) - want) <= 2.0 ** -8 * (np.abs(want) + slack) + slack)


@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_in_place_and_padding(interleaved):
    tokens, heads, dim, rotary = 33, 6, 128, 64
    x, pos, table = _case(tokens, heads, dim, rotary, 8)
    want = _same_steps(x, pos, table, interleaved)
    fused = torch.zeros(tokens, (heads + 3) * dim, dtype=torch.bfloat16, device=DEV)     # a slice of a wider projection
    part = fused[:, dim:dim + heads * dim].view(tokens, heads, dim)
    part.copy_(x)
    out = nb.nvfp4_rope(part, pos.to(DEV), table, interleaved)
    assert torch.equal(R.bits(out.cpu()), R.bits(want))
    flip = torch.empty(heads, tokens, dim, dtype=torch.bfloat16, device=DEV)             # head-major output
    nb.nvfp4_rope(part, pos.to(DEV), table, interleaved, out=flip.transpose(0, 1))
    assert torch.equal(R.bits(flip.cpu().transpose(0, 1)), R.bits(want))
    pad = pos.clone()
    pad[-4:] = -1
    before = fused.clone()
    nb.nvfp4_rope(part, pad.to(DEV), table, interleaved, out=part)                       # in place, padded batch
    assert torch.equal(R.bits(part[:-4].cpu()), R.bits(want[:-4]))
    assert torch.equal(fused[-4:], before[-4:])
    assert torch.equal(fused[:, :dim], before[:, :dim]) and torch.equal(fused[:, -2 * dim:], before[:, -2 * dim:])
    odd = torch.zeros(tokens * heads * dim + 1, dtype=torch.bfloat16, device=DEV)[1:].view(tokens, heads, dim)
    odd.copy_(x)                                                                         # 2-byte aligned
    assert torch.equal(R.bits(nb.nvfp4_rope(odd, pos.to(DEV), table, interleaved).cpu()), R.bits(want))
    one = x[:1].to(DEV).expand(tokens, heads, dim)                                       # one row for every token
    got = nb.nvfp4_rope(one, pos.to(DEV), table, interleaved)
    assert torch.equal(R.bits(got.cpu()), R.bits(_same_steps(x[:1].expand(tokens, heads, dim), pos, table, interleaved)))


def test_positions_outside_of_the_table_are_recorded():
    x, pos, table = _case(6, 2, 64, 64, 9, far=100)
    ws = nb.Workspace(DEV, 256)
    for bad in (100, -2, 2 ** 31 - 1):
        p = pos.clone()
        p[2] = bad
        out = torch.full((6, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        nb.nvfp4_rope(x.to(DEV), p.to(DEV), table, out=out, workspace=ws)
        assert nb.nvfp4_check_status(ws) == 1
        want = _same_steps(x, pos, table, False)
        want[2] = 7.0
        assert torch.equal(R.bits(out.cpu()), R.bits(want))
    assert nb.nvfp4_check_status(ws) == 0


def test_nonfinite_values_stay_in_their_pair():
    x, pos, table = _case(2, 2, 64, 64, 10)
    x[0, 0, 3], x[1, 1, 40] = float("nan"), float("inf")
    got = nb.nvfp4_rope(x.to(DEV), pos.to(DEV), table).cpu()
    fine = torch.ones(2, 2, 64, dtype=torch.bool)
    fine[0, 0, 3] = fine[0, 0, 35] = fine[1, 1, 40] = fine[1, 1, 8] = False
    assert torch.isfinite(got[fine]).all() and not torch.isfinite(got[~fine]).any()


def test_no_tokens_and_binding_refusals():
    table = nb.nvfp4_rope_table(nb.nvfp4_rope_inv_freq(64), 16, device=DEV)
    x = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    assert nb.nvfp4_rope(x, torch.zeros(0, dtype=torch.int32, device=DEV), table).shape == (0, 4, 64)
    x, pos = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="positions"):
        nb.nvfp4_rope(x, pos.long(), table)
    with pytest.raises(ValueError, match="positions"):
        nb.nvfp4_rope(x, pos[:1], table)
    with pytest.raises(ValueError, match="device"):
        nb.nvfp4_rope(x, pos.cpu(), table)
    with pytest.raises(ValueError, match="table"):
        nb.nvfp4_rope(x, pos, table.double())
    with pytest.raises(ValueError, match="innermost"):
        nb.nvfp4_rope(x.transpose(1, 2), pos, table)
    with pytest.raises(ValueError, match="out"):
        nb.nvfp4_rope(x, pos, table, out=x[:1])
    with pytest.raises(nb.NVFP4Error):                                   # table wider than the head
        nb.nvfp4_rope(x[..., :32], pos, table)
