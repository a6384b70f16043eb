"""Decode attention over the paged cache on the GPU against the 64-bit formula
on the exact restored values; bounds derived in paged_ref.attention_bounds."""
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


class Cache:
    """Quantized K and V of ragged sequences in pages of any order.  Rows that
    no sequence holds are filled with NaN scales: reading one shows."""

    def __init__(self, lens, heads, dim, page, seed, spare=3, make=None):
        rng = np.random.default_rng(seed)
        self.lens, self.heads, self.dim, self.page = list(lens), heads, dim, page
        cols = heads * dim
        used = [-(-n // page) for n in lens]
        self.pages = sum(used) + spare
        rows = self.pages * page
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), max(max(used), 1) + 1), 10 ** 9, np.int32)   # no such page
        at, self.host = 0, []
        pools = [(np.full((rows, cols // 2), 0xFF, np.uint8), np.full((rows, cols // 16), 0x7F, np.uint8)) for _ in range(2)]
        for b, n in enumerate(lens):
            self.table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
            t = np.arange(n)
            dest = self.table[b, t // page].astype(np.int64) * page + t % page
            kv = make(b, n, rng) if make else (rng.standard_normal((n, cols)), rng.standard_normal((n, cols)) + 0.25)
            held = []
            for x, (codes, scales), g in zip(kv, pools, (500.0, 300.0)):
                q = oracle.quantize_with_global(R.bf16(x), g, oracle.SF_LINEAR) if n else None
                if n:
                    codes[dest], scales[dest] = q.codes, q.scales.reshape(n, -1)
                    held.append((R.restore(q.codes, q.scales.reshape(n, -1)) / g).reshape(n, heads, dim))
                else:
                    held.append(np.zeros((0, heads, dim)))
            self.host.append(held)
        self.k, self.v = (nb.NVFP4Tensor(torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV).flatten(), torch.full((1,), g, device=DEV),
                                         rows, cols, nb.SF_LINEAR) for (c, s), g in zip(pools, (500.0, 300.0)))
        self.block_table = torch.from_numpy(self.table).to(DEV)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def attend(self, q, **more):
        more.setdefault("return_lse", True)
        table, lens = more.pop("block_table", self.block_table), more.pop("seq_lens", self.seq_lens)
        return nb.nvfp4_attention_decode_paged(q, self.k, self.v, self.heads, table, lens, self.page, **more)


def _query(n, heads, dim, seed, factor=1.0):
    return R.bf16(np.random.default_rng(seed).standard_normal((n, heads, dim)) * factor)


def _check(cache, q, o, lse, scale, what=""):
    heads, dim = cache.heads, cache.dim
    for b, n in enumerate(cache.lens):
        k, v = cache.host[b]
        want, wl, ao, sa = R.attention(R.f64(q[b]).reshape(heads, -1, dim), k, v, scale)
        ob, lb = R.attention_bounds(want, wl, ao, sa, n, dim, np.abs(v).max() if n else 0.0)
        got, gl = R.f64(o[b]).reshape(want.shape), R.f64(lse[b]).reshape(wl.shape)
        err = np.abs(got - want)
        assert np.all(err <= ob), f"{what} sequence {b} of {n}: o off by {np.nanmax(err - ob)} more than allowed"
        if n:
            assert np.all(np.abs(gl - wl) <= lb), f"{what} sequence {b} of {n}: lse {np.abs(gl - wl).max()} > {lb.min()}"
        else:
            assert np.all(np.isneginf(gl)) and not got.any()


@pytest.mark.parametrize("lens,heads,group,dim,page", [
    ([1], 1, 1, 128, 16), ([1, 2, 3], 2, 3, 64, 1), ([0], 1, 8, 128, 16), ([0, 0, 5, 0], 3, 2, 128, 4),
    ([15, 16, 17, 31, 32, 33], 4, 8, 128, 16), ([63, 64, 65, 127, 128, 129], 8, 8, 128, 64), ([100, 7, 300], 5, 3, 64, 20),
    ([1000], 8, 8, 128, 16), ([777, 1], 2, 7, 256, 48), ([513, 0, 40], 1, 20, 128, 256), ([260, 3], 1, 16, 64, 5),
    ([90, 91], 16, 1, 128, 16), ([40, 300], 6, 9, 64, 7), ([2500, 17], 4, 4, 128, 16), ([600, 20], 3, 33, 256, 16)])
def test_ragged_batches(lens, heads, group, dim, page):
    cache = Cache(lens, heads, dim, page, sum(lens) + dim)
    q = _query(len(lens), heads * group, dim, 1)
    o, lse = cache.attend(q.to(DEV))
    _check(cache, q, o, lse, dim ** -0.5)


# The kernel has a form per head size, per way of copying (TMA where 16 tokens
# share a page and a row's scales are whole 16-byte groups) and per warps of a
# unit (2, 4, 8); the cases above and below meet each of them.
@pytest.mark.parametrize("lens,heads,group,dim,page", [
    ([700, 33, 16], 4, 8, 64, 16), ([129, 0, 90], 8, 12, 64, 32), ([300, 41], 1, 40, 64, 16), ([260], 4, 30, 128, 20),
    ([350, 70], 2, 32, 128, 16), ([90, 200, 5], 2, 16, 128, 48), ([400, 8], 6, 2, 128, 16), ([77, 500], 4, 4, 256, 16),
    ([300, 30], 1, 5, 256, 32), ([200, 64], 4, 8, 256, 20), ([150, 6], 2, 1, 256, 9), ([330, 11], 1, 8, 256, 7),
    ([130, 1], 1, 9, 256, 24), ([610, 2, 48], 3, 16, 256, 16)])
def test_every_form_of_the_kernel(lens, heads, group, dim, page):
    cache = Cache(lens, heads, dim, page, sum(lens) + group)
    q = _query(len(lens), heads * group, dim, 31)
    o, lse = cache.attend(q.to(DEV))
    _check(cache, q, o, lse, dim ** -0.5)


def test_batch_of_sequences_that_are_all_cut():
    """60 sequences (more than a warp schedules by itself) over 148 ranges:
    each is cut and joined, some from two parts, some from more."""
    rng = np.random.default_rng(33)
    lens = [int(v) for v in rng.integers(150, 900, 60)]
    lens[7], lens[8] = 0, 3000
    cache = Cache(lens, 4, 64, 16, 34)
    q = _query(60, 16, 64, 35)
    o, lse = cache.attend(q.to(DEV))
    _check(cache, q, o, lse, 0.125)


@pytest.mark.parametrize("n,heads,dim", [(20000, 2, 128), (9001, 1, 64), (5000, 2, 256)])
def test_one_long_sequence_split_over_the_device(n, heads, dim):
    """Also peaked weights in the last tokens, after which all that was summed
    before has to be scaled down, and a ramp in V that a dropped or doubled
    part would move."""
    def make(b, n, rng):
        k, v = rng.standard_normal((n, heads * dim)), rng.standard_normal((n, heads * dim)) * 0.1
        v += np.linspace(-4, 4, n)[:, None]
        k[n - 5:] *= 3.0
        return k, v

    cache = Cache([n, 10], heads, dim, 16, n, make=make)
    for factor in (0.0, 1.0, 8.0):
        q = _query(2, heads * 8, dim, 2, factor)
        o, lse = cache.attend(q.to(DEV))
        _check(cache, q, o, lse, dim ** -0.5, f"query times {factor}")


def test_many_sequences():
    rng = np.random.default_rng(3)
    lens = [int(v) for v in np.exp(rng.uniform(0, np.log(400), 300))]
    lens[:4] = [0, 1, 900, 0]
    cache = Cache(lens, 2, 64, 16, 4)
    q = _query(300, 8, 64, 5)
    o, lse = cache.attend(q.to(DEV))
    _check(cache, q, o, lse, 0.125)
    again, l2 = cache.attend(q.to(DEV))
    assert torch.equal(R.bits(o), R.bits(again)) and torch.equal(lse, l2)      # the same bits every time


@pytest.mark.parametrize("n,heads", [(31, 8), (32, 1), (32, 40), (33, 1), (33, 40)])
def test_sequences_around_the_number_a_warp_schedules(n, heads):
    """Up to 32 sequences each warp schedules for itself; 40 heads leave fewer
    ranges (29) than sequences, so that the joins are by range."""
    lens = [(7 * b * b + b) % 90 for b in range(n)]
    cache = Cache(lens, heads, 128, 16, n + heads)
    q = _query(n, heads * 3, 128, 33)
    o, lse = cache.attend(q.to(DEV))
    _check(cache, q, o, lse, 128 ** -0.5)


@pytest.mark.parametrize("lens,heads,group,dim,page", [
    ([9000, 0, 30], 2, 8, 128, 16), ([40, 3, 17, 160], 4, 20, 64, 10), ([700, 50], 1, 6, 256, 32)])
def test_output_in_place_of_the_query(lens, heads, group, dim, page):
    cache = Cache(lens, heads, dim, page, 34)
    q = _query(len(lens), heads * group, dim, 35).to(DEV)
    o, lse = cache.attend(q)
    rows = torch.full((len(lens), heads * group + 2, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    for x in (q.clone(), rows[:, 1:-1].copy_(q)):
        got, got_lse = cache.attend(x, out=x)
        assert got is x and torch.equal(R.bits(x), R.bits(o)) and torch.equal(got_lse, lse)
    assert (rows[:, 0] == 7).all() and (rows[:, -1] == 7).all()


def test_matches_the_contiguous_read():
    """The identity table over one pool is nvfp4_attention_decode; both are
    within their bounds, so they differ by at most two BF16 roundings and the
    weights' FP16 rounding."""
    n, heads = 3000, 4
    cache = Cache([n], heads, 128, 1, 6, spare=0)
    rows = torch.from_numpy(cache.table[0, :n].astype(np.int64)).to(DEV)
    k, v = (nb.NVFP4Tensor(t.codes[rows].contiguous(), t.scales.view(t.rows, -1)[rows].flatten(), t.global_scale, n, t.cols, nb.SF_LINEAR) for t in (cache.k, cache.v))
    q = _query(1, heads * 8, 128, 7)
    flat = nb.nvfp4_attention_decode(q[0].to(DEV), k, v, heads)
    table = torch.arange(n, dtype=torch.int32, device=DEV)[None]
    paged = nb.nvfp4_attention_decode_paged(q.to(DEV), k, v, heads, table, cache.seq_lens, 1)
    want, wl, ao, sa = R.attention(R.f64(q[0]).reshape(heads, 8, 128), *cache.host[0], 128 ** -0.5)
    bound, _ = R.attention_bounds(want, wl, ao, sa, n, 128, np.abs(cache.host[0][1]).max())
    assert np.all(np.abs(R.f64(flat) - R.f64(paged[0])) <= 2 * bound.reshape(heads * 8, 128))


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(scale):
    cache = Cache([200, 33], 2, 128, 16, 8)
    q = _query(2, 6, 128, 9)
    o, lse = cache.attend(q.to(DEV), scale=scale)
    _check(cache, q, o, lse, scale)


@pytest.mark.parametrize("factor", [1e-30, 1e30, 2.0 ** 20])
def test_queries_far_from_one(factor):
    """BF16 queries beyond FP16's range (the scale brings the scores back)."""
    cache = Cache([150], 2, 128, 16, 10)
    q = _query(1, 16, 128, 11, factor)
    o, lse = cache.attend(q.to(DEV), scale=0.1 / factor)
    _check(cache, q, o, lse, float(np.float32(0.1 / factor)))


def test_strided_query_output_and_table():
    lens, heads, group, dim = [50, 0, 130], 2, 4, 128
    cache = Cache(lens, heads, dim, 16, 12)
    q = _query(3, heads * group, dim, 13)
    ref, lref = cache.attend(q.to(DEV))
    wide = torch.zeros(3, heads * group + 5, dim, dtype=torch.bfloat16, device=DEV)       # q beside k and v
    wide[:, 2:2 + heads * group] = q.to(DEV)
    out = torch.full((3, heads * group, 2 * dim), 5.0, dtype=torch.bfloat16, device=DEV)
    table = torch.full((3, cache.block_table.shape[1] + 9), -7, dtype=torch.int32, device=DEV)
    table[:, :cache.block_table.shape[1]] = cache.block_table
    o, lse = cache.attend(wide[:, 2:2 + heads * group], out=out[..., :dim], block_table=table[:, :cache.block_table.shape[1]])
    assert torch.equal(R.bits(o), R.bits(ref)) and torch.equal(lse, lref)
    assert (out[..., dim:] == 5).all()
    major = torch.zeros(heads * group, 3, dim, dtype=torch.bfloat16, device=DEV)           # head-major
    cache.attend(q.to(DEV), out=major.transpose(0, 1), return_lse=False)
    assert torch.equal(R.bits(major.transpose(0, 1)), R.bits(ref))
    same = q[:1].to(DEV).expand(3, heads * group, dim)                                     # one query for all
    o, lse = cache.attend(same)
    _check(cache, q[:1].expand(3, heads * group, dim), o, lse, dim ** -0.5)


def test_nan_stays_in_its_sequence_and_head():
    cache = Cache([70, 300, 20], 2, 128, 16, 14)
    q = _query(3, 8, 128, 15)
    q[1, 5, 77] = float("nan")
    q[2, 0, 0] = float("inf")
    o, lse = cache.attend(q.to(DEV))
    bad = torch.zeros(3, 8, dtype=torch.bool)
    bad[1, 5] = bad[2, 0] = True
    assert torch.isnan(o.float()).any(-1).cpu().equal(bad) and not torch.isfinite(lse.cpu()[bad]).any()
    q[1, 5] = q[2, 0] = 0.0
    clean, _ = cache.attend(q.to(DEV))
    assert torch.equal(R.bits(clean)[~bad.to(DEV)], R.bits(o)[~bad.to(DEV)])


def test_bad_pages_and_lengths_are_recorded():
    ws = nb.Workspace(DEV, 256)
    cache = Cache([100, 40], 2, 128, 16, 16)
    q = _query(2, 4, 128, 17)
    for bad in (-1, cache.pages, 2 ** 31 - 1):
        table = cache.block_table.clone()
        table[0, 2] = bad                                                    # tokens 32 .. 47 take no part
        o, lse = cache.attend(q.to(DEV), block_table=table, workspace=ws)
        assert nb.nvfp4_check_status(ws) == 1
        cut = Cache.__new__(Cache)
        cut.heads, cut.dim, cut.lens = 2, 128, [84, 40]
        cut.host = [[np.delete(x, np.s_[32:48], 0) for x in cache.host[0]], cache.host[1]]
        _check(cut, q, o, lse, 128 ** -0.5, f"page {bad}")
    table = cache.block_table.clone()
    table[0, :] = -1
    o, lse = cache.attend(q.to(DEV), block_table=table, workspace=ws)
    assert nb.nvfp4_check_status(ws) == 1 and not o[0].any() and torch.isneginf(lse[0]).all()
    # a length past the table's pages is cut to them, a negative one to 0
    short = cache.block_table[:, :3].contiguous()
    o, lse = cache.attend(q.to(DEV), block_table=short, seq_lens=torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32, device=DEV), workspace=ws)
    assert nb.nvfp4_check_status(ws) == 1
    cut.lens, cut.host = [48, 0], [[x[:48] for x in cache.host[0]], [x[:0] for x in cache.host[1]]]
    _check(cut, q, o, lse, 128 ** -0.5, "cut")
    none = torch.zeros(2, 0, dtype=torch.int32, device=DEV)                    # no pages at all
    o, lse = cache.attend(q.to(DEV), block_table=none, seq_lens=torch.zeros(2, dtype=torch.int32, device=DEV), workspace=ws)
    assert nb.nvfp4_check_status(ws) == 0 and not o.any() and torch.isneginf(lse).all()
    assert nb.nvfp4_check_status(ws) == 0


def test_pool_past_32_bit_offsets():
    heads, dim, page = 32, 256, 16
    cols = heads * dim
    pages = (1 << 32) // (cols // 2) // page + 20
    rows = pages * page
    small = Cache([40], heads, dim, page, 18, spare=0)
    pools = []
    for t in (small.k, small.v):
        big = nb.NVFP4Tensor(torch.zeros(rows, cols // 2, dtype=torch.uint8, device=DEV), torch.zeros(rows * cols // 16, dtype=torch.uint8, device=DEV),
                             t.global_scale, rows, cols, nb.SF_LINEAR)
        big.codes[-t.rows:] = t.codes
        big.scales[-t.scales.numel():] = t.scales
        pools.append(big)
    q = _query(1, heads * 2, dim, 19)
    table = small.block_table.clone()
    table[:, :3] += pages - small.pages
    small.k, small.v = pools
    o, lse = small.attend(q.to(DEV), block_table=table)
    _check(small, q, o, lse, dim ** -0.5)


def test_two_streams_at_once():
    """Calls on two streams share the workspace, not the scratch."""
    a, b = Cache([6000, 100], 2, 128, 16, 20), Cache([3000, 2000, 5], 2, 128, 16, 21)
    qa, qb = _query(2, 16, 128, 22).to(DEV), _query(3, 16, 128, 23).to(DEV)
    ra, rb = a.attend(qa), b.attend(qb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        got.append((a.attend(qa, stream=s1), b.attend(qb, stream=s2.cuda_stream)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(R.bits(x[0]), R.bits(ra[0])) and torch.equal(x[1], ra[1])
        assert torch.equal(R.bits(y[0]), R.bits(rb[0])) and torch.equal(y[1], rb[1])


def test_captured_step_replayed_with_other_lengths_and_pages():
    """Rotate, write and attend captured once; each replay has new tokens, new
    lengths and slots (two graphs alternate), as a serving loop has them."""
    heads, group, dim, page, n = 2, 4, 128, 16, 5
    rng = np.random.default_rng(24)
    lens = np.array([0, 15, 16, 200, 37])
    cache = Cache([260] * n, heads, dim, page, 25)
    table = nb.nvfp4_rope_table(nb.nvfp4_rope_inv_freq(dim), 512, device=DEV)
    q, k, v = (torch.zeros(n, h, dim, dtype=torch.bfloat16, device=DEV) for h in (heads * group, heads, heads))
    pos, slots, seq = (torch.full((n,), -1, dtype=torch.int32, device=DEV) for _ in range(3))
    seq.fill_(0)

    def step():
        r = nb.nvfp4_rope(q, pos, table)
        nb.nvfp4_kv_write(k, v, slots, cache.k, cache.v, pos, table)
        return cache.attend(r, seq_lens=seq)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        graphs.append((g, outs))
    host = [[x.copy() for x in h] for h in cache.host]
    for i in range(6):
        hq, hk, hv = (R.bf16(rng.standard_normal((n, h, dim))) for h in (heads * group, heads, heads))
        p = lens.astype(np.int32)
        s = np.array([cache.table[b, t // page] * page + t % page for b, t in enumerate(p)], np.int32)
        for d, x in ((q, hq), (k, hk), (v, hv), (pos, torch.from_numpy(p)), (slots, torch.from_numpy(s)), (seq, torch.from_numpy(p + 1))):
            d.copy_(x)
        g, (o, lse) = graphs[i % 2]
        g.replay()
        torch.cuda.synchronize()
        cs = table.cpu().numpy()[p]
        turned = [torch.from_numpy(R.rope(x.float().numpy(), cs[..., 0], cs[..., 1], False)).to(torch.bfloat16) for x in (hq, hk)]
        for x, gscale, j in ((turned[1], 500.0, 0), (hv, 300.0, 1)):
            w = oracle.quantize_with_global(x.reshape(n, -1), gscale, oracle.SF_LINEAR)
            rows = (R.restore(w.codes, w.scales.reshape(n, -1)) / gscale).reshape(n, heads, dim)
            for b in range(n):
                host[b][j][p[b]] = rows[b]
        view = Cache.__new__(Cache)
        view.heads, view.dim, view.lens = heads, dim, [int(t) + 1 for t in p]
        view.host = [[x[:t + 1] for x in host[b]] for b, t in enumerate(p)]
        _check(view, turned[0], o, lse, dim ** -0.5, f"replay {i}")
        lens += 1
    assert nb.nvfp4_check_status() == 0


@pytest.mark.parametrize("heads,dim,page", [(4, 128, 16), (1, 64, 16)])      # TMA, and copies without it
def test_a_wait_that_gives_up_is_recorded(heads, dim, page):
    """The wait limit cut to one cycle: the first wait that does not find its
    tile there gives up, the call records it and ends by itself; the next
    call is right."""
    cache = Cache([3000, 500], heads, dim, page, 40)
    q = _query(2, heads * 4, dim, 41)
    ws = nb.Workspace(DEV, 256)
    nb.nvfp4_set_wait_limit_cycles(1)
    try:
        cache.attend(q.to(DEV), workspace=ws)
        assert nb.nvfp4_check_status(ws) == 7
    finally:
        nb.nvfp4_set_wait_limit_cycles(0)
    o, lse = cache.attend(q.to(DEV), workspace=ws)
    assert nb.nvfp4_check_status(ws) == 0
    _check(cache, q, o, lse, dim ** -0.5)


def test_binding_refusals():
    cache = Cache([20], 2, 64, 16, 26)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="block_table"):
        cache.attend(q, block_table=cache.block_table.long())
    with pytest.raises(ValueError, match="seq_lens"):
        cache.attend(q, seq_lens=cache.seq_lens.long())
    with pytest.raises(ValueError, match="seq_lens"):
        cache.attend(q, seq_lens=torch.zeros(2, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError, match="columns"):
        cache.attend(torch.zeros(1, 4, 128, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError, match="q:"):
        cache.attend(q.float())
    with pytest.raises(ValueError, match="out"):
        cache.attend(q, out=torch.zeros(1, 4, 64, device=DEV))
    with pytest.raises(ValueError, match="device"):
        cache.attend(q, seq_lens=cache.seq_lens.cpu())
    with pytest.raises(nb.NVFP4Error):                                       # 3 query heads over 2
        cache.attend(q[:, :3])
    o, lse = cache.attend(torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV), block_table=cache.block_table[:0], seq_lens=cache.seq_lens[:0])
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
