"""Paged decode attention where each CTA takes many more tiles than its ring of
shared memory has stages: stages are handed back and filled again, whole
sequences lie within a range, and sequences end in the middle of the ring.

The pools hold random codes and scales, what they stand for is restored in 64
bits on the GPU by plain torch operations; bounds as in
paged_ref.attention_bounds.  Queries are scaled so that a head's weights lie
on a few dozen tokens, which differ from head to head: a tile that is lost,
taken twice or overwritten too early moves some head's output far past its
bound."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_22_b200 import binding as nb
from tests import paged_plan
from tests import paged_ref as R

DEV = "cuda"

#: head size, KV heads, tokens a page: a case for every way of copying (TMA for
#: pages of whole 16 tokens with scale rows of whole 16-byte groups, else
#: cp.async) and number of warps that share a unit (2, 4, 8)
FORMS = [(64, 40, 16), (64, 40, 20), (64, 38, 16), (64, 37, 32),
         (128, 40, 64), (128, 38, 16), (128, 40, 20), (128, 38, 1), (128, 37, 16),
         (256, 24, 16), (256, 22, 32), (256, 21, 16), (256, 24, 20), (256, 22, 5), (256, 21, 20)]
GROUP = 8


def _lengths(dim, heads, kind):
    """Lengths that give each range 3 times the ring's stages, or more."""
    tokens, ranges, stages, _ = paged_plan.plan(heads * GROUP, heads, dim)
    tiles = (3 * stages + 8) * ranges
    if kind == "long":                                                 # one sequence, and a short one behind it
        return [tiles * tokens - 5, 3]
    rng = np.random.default_rng(dim + heads)
    lens = [0, 1]
    while sum(max(1, -(-n // tokens)) for n in lens) < tiles:
        lens.append(int(rng.integers(0, 2 * stages * tokens)))
    return lens


@pytest.mark.parametrize("kind", ["long", "ragged"])
@pytest.mark.parametrize("dim,heads,page", FORMS)
def test_ranges_hold_more_tiles_than_the_ring(dim, heads, page, kind):
    """What the cases below rest on, from the library's own plan."""
    lens = _lengths(dim, heads, kind)
    _, ranges, stages, _ = paged_plan.plan(heads * GROUP, heads, dim)
    taken = paged_plan.tiles_of_ranges(lens, heads * GROUP, heads, dim)
    assert len(taken) == ranges
    counts = [len(t) for t in taken]
    if kind == "long":
        assert min(counts) >= 3 * stages
    else:
        assert min(counts) >= 2 * stages and np.mean(counts) >= 3 * stages
        ends = [i for t in taken for i, (b, n) in enumerate(t) if i + 1 < len(t) and t[i + 1][0] != b]
        assert len({(i + 1) % stages for i in ends}) == stages         # ends at every place of the ring
        assert max(ends) > 2 * stages


def test_plan_matches_the_scratch_size():
    """The compiled header is the library's: 2 parts a range and unit, a join a range."""
    if not torch.cuda.is_available():
        from nvfp4_block_scaled_22_b200.build import build
        build()
    for dim, heads, _ in FORMS:
        _, ranges, _, _ = paged_plan.plan(heads * GROUP, heads, dim)
        assert nb.lib().nvfp4_attention_paged_scratch_bytes(heads * GROUP, heads, dim) == ranges * (2 * heads * (8 * dim + 16) * 4 + 16)


class Pool:
    """Random pages of a batch; rows that no sequence holds have NaN scales."""

    def __init__(self, lens, dim, heads, page, seed):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.dim, self.heads, self.page = lens, dim, heads, page
        used = [-(-n // page) for n in lens]
        pages, width = sum(used) + 3, max(used)
        rows, cols = pages * page, heads * dim
        order = torch.randperm(pages, generator=gen, device=DEV, dtype=torch.int32)
        self.table = torch.full((len(lens), width), 10 ** 9, dtype=torch.int32, device=DEV)
        column = torch.arange(width, device=DEV)
        self.table[column < torch.tensor(used, device=DEV)[:, None]] = order[:sum(used)]
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.rows = [self.table[b, torch.arange(n, device=DEV) // page].long() * page + torch.arange(n, device=DEV) % page
                     for b, n in enumerate(lens)]
        self.caches = []
        for g in (8.0, 4.0):
            codes = torch.full((rows, cols // 2), 0xFF, dtype=torch.uint8, device=DEV)
            scales = torch.full((rows, cols // 16), 0x7F, dtype=torch.uint8, device=DEV)
            for r in self.rows:                                        # scales from 0.5 to 3.75
                codes[r] = torch.randint(0, 256, (len(r), cols // 2), generator=gen, device=DEV, dtype=torch.uint8)
                scales[r] = torch.randint(48, 72, (len(r), cols // 16), generator=gen, device=DEV, dtype=torch.uint8)
            self.caches.append(nb.NVFP4Tensor(codes, scales.flatten(), torch.full((1,), g, device=DEV), rows, cols, nb.SF_LINEAR))

    def restored(self, which, b):
        t = self.caches[which]
        grid = torch.from_numpy(np.concatenate([R.GRID, -R.GRID])).to(DEV)
        e4m3 = torch.from_numpy(R.E4M3).to(DEV)
        c, s = t.codes[self.rows[b]].long(), t.scales.view(t.rows, -1)[self.rows[b]].long()
        v = grid[torch.stack((c & 15, c >> 4), -1).flatten(1)] * e4m3[s].repeat_interleave(16, 1)
        return (v / t.global_scale.double()).view(-1, self.heads, self.dim)

    def attend(self, q, **more):
        return nb.nvfp4_attention_decode_paged(q, *self.caches, self.heads, self.table, self.seq_lens, self.page, return_lse=True, **more)

    def check(self, q, o, lse, scale):
        for b, n in enumerate(self.lens):
            if n == 0:
                assert not o[b].any() and torch.isneginf(lse[b]).all()
                continue
            k, v = self.restored(0, b), self.restored(1, b)
            x = q[b].double().view(self.heads, -1, self.dim)
            s = scale * torch.einsum("hgd,thd->hgt", x, k)
            sa = abs(scale) * torch.einsum("hgd,thd->hgt", x.abs(), k.abs()).amax(-1)
            wl = torch.logsumexp(s, -1)
            p = torch.exp(s - wl[..., None])
            want, ao = (torch.einsum("hgt,thd->hgd", p, y) for y in (v, v.abs()))
            ob, lb = R.attention_bounds(*(R.f64(t) for t in (want, wl, ao, sa)), n, self.dim, float(v.abs().max()))
            err = np.abs(R.f64(o[b]).reshape(ob.shape) - R.f64(want))
            assert np.all(err <= ob), f"sequence {b} of {n}: o off by {np.nanmax(err - ob)} more than allowed"
            off = np.abs(R.f64(lse[b]).reshape(lb.shape) - R.f64(wl))
            assert np.all(off <= lb), f"sequence {b} of {n}: lse {np.nanmax(off)}"


def _query(n, heads, dim, seed):
    """Scores (times dim ** -0.5) with a deviation of about 2.5: keys have one of about 1."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (2.5 * torch.randn(n, heads * GROUP, dim, generator=gen, device=DEV)).bfloat16()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["long", "ragged"])
@pytest.mark.parametrize("dim,heads,page", FORMS)
def test_stages_are_used_again(dim, heads, page, kind):
    lens = _lengths(dim, heads, kind)
    pool = Pool(lens, dim, heads, page, dim + heads + page)
    q = _query(len(lens), heads, dim, 1)
    ws = nb.Workspace(DEV, 256)
    o, lse = pool.attend(q, workspace=ws)
    assert nb.nvfp4_check_status(ws) == 0
    pool.check(q, o, lse, dim ** -0.5)
    again, l2 = pool.attend(q, workspace=ws)
    assert torch.equal(R.bits(o), R.bits(again)) and torch.equal(lse, l2)


@pytest.mark.gpu
@pytest.mark.parametrize("limit", [1, 1000, 20000])
@pytest.mark.parametrize("dim,heads,page", [(128, 40, 16), (256, 21, 16), (64, 40, 20), (128, 37, 16)])   # TMA, TMA, cp.async, cp.async
def test_a_wait_that_gives_up_with_stages_in_use(dim, heads, page, limit):
    """Ranges of many times the ring's stages, and waits that are cut short at
    their start, or may be in their middle: the call records what gave up (a
    long limit may do for all waits) and ends by itself, its copies awaited;
    the next call is right."""
    lens = _lengths(dim, heads, "ragged")
    pool = Pool(lens, dim, heads, page, 7)
    q = _query(len(lens), heads, dim, 2)
    ws = nb.Workspace(DEV, 256)
    nb.nvfp4_set_wait_limit_cycles(limit)
    try:
        o, lse = pool.attend(q, workspace=ws)
        status = nb.nvfp4_check_status(ws)
    finally:
        nb.nvfp4_set_wait_limit_cycles(0)
    assert status in ((7,) if limit == 1 else (0, 7))
    if status == 0:
        pool.check(q, o, lse, dim ** -0.5)
    o, lse = pool.attend(q, workspace=ws)
    assert nb.nvfp4_check_status(ws) == 0
    pool.check(q, o, lse, dim ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,heads,page", [(64, 40, 16), (128, 38, 16), (128, 37, 16), (256, 22, 5)])
def test_output_in_place_of_the_queries_of_many_sequences(dim, heads, page):
    """CTAs that take several sequences fetch a query while they write the
    result before it; sequences that are cut leave theirs to the join."""
    lens = _lengths(dim, heads, "ragged")
    pool = Pool(lens, dim, heads, page, 11)
    rows = torch.full((len(lens), heads * GROUP * dim + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    q = rows[:, 8:-16].view(len(lens), heads * GROUP, dim)                 # rows that share cache lines with their neighbours
    q.copy_(_query(len(lens), heads, dim, 3))
    o, lse = pool.attend(q)
    got, got_lse = pool.attend(q, out=q)
    assert got is q and torch.equal(R.bits(q), R.bits(o)) and torch.equal(got_lse, lse)
    assert (rows[:, :8] == 7).all() and (rows[:, -16:] == 7).all()
