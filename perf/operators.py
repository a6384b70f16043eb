"""The paged NVFP4 key-value cache of a serving loop, as work to be measured:
rotary positions, the cache's write and read, and decode attention over it.

A cache is a pool of token rows (pages of ``page`` tokens); a row holds the
E2M1 codes (two a byte) and the E4M3 block scales of heads * dim values under
one FP32 scale for the pool.  ``run`` computes either the plain form (torch,
32 bits) or, where ``own`` is true, calls the library.
"""
import random

import torch

own = False

DEV = "cuda"
#: positions that the rotary table of a case covers
TABLE_ROWS = 131072


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of one sequence: 64 query and 8 key heads rotated in place of the projection's output
        dict(name="rope one token", op="rope", tokens=1, heads=72, dim=128, rotary=128, interleaved=False, inverse=False, base=1e4),
        # a prompt of 8192 tokens, queries and keys together
        dict(name="rope prompt", op="rope", tokens=8192, heads=72, dim=128, rotary=128, interleaved=False, inverse=False, base=5e5),
        # the gradient of a training step, neighbouring pairs, half of the head rotated, odd token count
        dict(name="rope gradient", op="rope", tokens=4099, heads=40, dim=128, rotary=64, interleaved=True, inverse=True, base=1e4),
        # the new keys and values of a decode step of 64 sequences (the last 3 rows pad the batch)
        dict(name="write decode", op="write", tokens=67, pad=3, heads=8, dim=128, rotary=128, interleaved=False, page=16, base=1e4),
        # a prompt's keys and values into the cache
        dict(name="write prompt", op="write", tokens=16384, pad=0, heads=8, dim=128, rotary=128, interleaved=False, page=64, base=5e5),
        # a ragged prefill chunk of a smaller model: 5 heads of 64, a quarter of the head rotated, pages of 48 tokens
        dict(name="write ragged", op="write", tokens=5003, pad=11, heads=5, dim=64, rotary=16, interleaved=True, page=48, base=1e4),
        # a short shared prefix restored for a new prompt's dense attention
        dict(name="read prefix", op="read", rows=777, heads=8, dim=128, page=16),
        # a whole 128K context restored for a prompt chunk's dense attention
        dict(name="read context", op="read", rows=131072, heads=8, dim=128, page=64),
        # one sequence of ordinary length: latency
        dict(name="attend one", op="attend", seqs=1, low=1000, high=1000, heads=8, group=8, dim=128, page=16),
        # one sequence over the whole 128K cache
        dict(name="attend long", op="attend", seqs=1, low=131072, high=131072, heads=8, group=8, dim=128, page=64),
        # a serving batch, lengths from empty to 8192
        dict(name="attend batch", op="attend", seqs=96, low=256, high=8192, heads=8, group=8, dim=128, page=16),
        # odd sizes: 3 query heads a key head, heads of 64, pages that end inside a tile
        dict(name="attend odd", op="attend", seqs=37, low=1, high=3001, heads=5, group=3, dim=64, page=20),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([1, 16, 16, 20, 32, 48, 64, 256])
    if op == "rope":
        heads = rng.randint(1, 72)
        most = 8192 * 72 * 128 // (heads * dim)
        return dict(op=op, tokens=_log(rng, 1, min(16384, most)), heads=heads, dim=dim, rotary=2 * rng.randint(1, dim // 2) if rng.random() < 0.3
                    else dim // rng.choice([1, 1, 2, 4]), interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, base=rng.choice([1e4, 5e5, 1e6]))
    heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    if op == "write":
        tokens = _log(rng, 1, min(16384, 16384 * 1024 // (heads * dim)))
        return dict(op=op, tokens=tokens, pad=rng.randint(0, tokens // 8), heads=heads, dim=dim, rotary=rng.choice([0, dim, dim, dim // 2, dim // 4]),
                    interleaved=rng.random() < 0.5, page=page, base=rng.choice([1e4, 5e5, 1e6]))
    if op == "read":
        return dict(op=op, rows=_log(rng, 1, 131072 * 1024 // (heads * dim)), heads=heads, dim=dim, page=page)
    seqs = _log(rng, 1, 192)
    high = _log(rng, 16, min(131072, 96 * 8192 * 1024 // (heads * dim) // seqs))
    return dict(op=op, seqs=seqs, low=_log(rng, 1, high), high=high, heads=heads, group=rng.choice([1, 2, 3, 4, 7, 8, 8, 16]), dim=dim, page=page)


def _lengths(case):
    """The sequences' lengths, spread over their logarithm; a larger batch has an empty sequence and one of a single token among them."""
    n, low, high = case["seqs"], case["low"], case["high"]
    r = random.Random(n * 1000003 + low * 1009 + high)
    lens = [_log(r, low, high) for _ in range(n)]
    lens[0] = high
    if n > 8:
        lens[1], lens[2] = 0, 1
    return lens


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 4.0 * n + 4 * case["tokens"] * (1 + case["rotary"]), "flops": 3.0 * case["tokens"] * case["heads"] * case["rotary"]}
    cols = case["heads"] * case["dim"]
    if case["op"] == "write":  # keys and values in, codes and scales out, and those restored for the caller
        t = case["tokens"] - case["pad"]
        return {"bytes": t * (2 * cols * (2 + 2 * 0.5625 + 2) + 4 * case["rotary"] + 8.0), "flops": 2.0 * t * cols * 4}
    if case["op"] == "read":
        return {"bytes": case["rows"] * (2 * cols * (0.5625 + 2) + 4.0), "flops": 2.0 * case["rows"] * cols}
    tokens, out = sum(_lengths(case)), case["seqs"] * cols * case["group"]
    return {"bytes": tokens * cols * 2 * 0.5625 + out * 4.0, "flops": 4.0 * tokens * cols * case["group"]}


# --------------------------------------------------------------- formats
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
#: borders between neighbouring codes; a value on one goes to the even code
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _values(codes, scales, dtype=torch.float32):
    """e2m1(code) * e4m3(scale), [..., n / 2] and [..., n / 16] bytes to [..., n]."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device, dtype=dtype)
    c = grid[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    s = scales.view(torch.float8_e4m3fn).to(dtype)
    return (c.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _restored(codes, scales, g, dtype=torch.float32):
    """The values that rows stand for, e2m1(code) * (e4m3(scale) / g)."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device, dtype=dtype)
    c = grid[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    s = scales.view(torch.float8_e4m3fn).to(dtype) / g.to(dtype)
    return (c.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _quantized(x, g):
    """Codes and scales of the rows of x under the tensor scale g: a scale for
    16 values from their largest magnitude, then each value to the nearest code."""
    b = x.unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / 6 * g).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.to(x.dtype)
    y = b * torch.where(sf > 0, g / sf, 0.0).unsqueeze(-1)
    a = y.abs()
    code = ((a > BORDERS[0]).byte() + (a >= BORDERS[1]).byte() + (a > BORDERS[2]).byte() + (a >= BORDERS[3]).byte()
            + (a > BORDERS[4]).byte() + (a >= BORDERS[5]).byte() + (a > BORDERS[6]).byte())
    code = (code + 8 * torch.signbit(b).byte()).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], s.view(torch.uint8)


def _table(rotary, base):
    """(cos, sin) of each position and pair, angles in 64 bits, held in 32."""
    f = base ** (-torch.arange(0, rotary, 2, device=DEV, dtype=torch.float64) / rotary)
    a = torch.arange(TABLE_ROWS, device=DEV, dtype=torch.float64).unsqueeze(1) * f
    return torch.stack((a.cos(), a.sin()), -1).float()


def _rotated(x, cs, interleaved, inverse):
    """The first 2 * cs.shape[-2] values of each head rotated; x [T, H, D], cs [T, pairs, 2], in cs's precision."""
    n = cs.shape[-2]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1] * (-1.0 if inverse else 1.0)
    r, rest = x[..., : 2 * n].to(cs.dtype), x[..., 2 * n:].to(cs.dtype)
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :n], r[..., n:])
    a, b = a * c - b * s, b * c + a * s
    return torch.cat((torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1), rest), -1)


# --------------------------------------------------------------- prepare
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.bfloat16)


def _pool(gen, pages, page, heads, dim):
    """A cache pool that holds quantized rows: normal values, with a few channels ten times larger."""
    rows, cols = pages * page, heads * dim
    factor = torch.ones(cols, device=DEV)
    factor[torch.randperm(cols, generator=gen, device=DEV)[:5]] = 10.0
    g = torch.full((1,), 448 * 6 / 64.0, device=DEV)
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, cols // 16, dtype=torch.uint8, device=DEV)
    for a in range(0, rows, 32768):
        codes[a:a + 32768], scales[a:a + 32768] = _quantized(_normal(gen, min(32768, rows - a), cols).float() * factor, g)
    return dict(codes=codes, scales=scales, g=g)


def _slots(gen, pages, page, tokens):
    """Rows of `tokens` consecutive tokens in pages of any order."""
    order = torch.randperm(pages, generator=gen, device=DEV, dtype=torch.int32)
    t = torch.arange(tokens, device=DEV, dtype=torch.int32)
    return (order[(t // page).long()] * page + t % page).int()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "rope":
        t, h = case["tokens"], case["heads"]
        s["x"] = _normal(gen, t, h, case["dim"])
        first = torch.randint(0, TABLE_ROWS - t, (1,), generator=gen, device=DEV, dtype=torch.int32)
        s["positions"] = first + torch.arange(t, device=DEV, dtype=torch.int32)
        s["table"] = _table(case["rotary"], case["base"])
        return s
    heads, dim, page = case["heads"], case["dim"], case["page"]
    if op in ("write", "read"):
        n = case["tokens"] if op == "write" else case["rows"]
        pages = -(-n // page) + 2
        s["k_cache"], s["v_cache"] = _pool(gen, pages, page, heads, dim), _pool(gen, pages, page, heads, dim)
        s["slots"] = _slots(gen, pages, page, n)
        if op == "write":
            s["k"], s["v"] = _normal(gen, n, heads, dim), _normal(gen, n, heads, dim)
            s["positions"] = torch.randint(0, TABLE_ROWS - n, (1,), generator=gen, device=DEV, dtype=torch.int32) + torch.arange(n, device=DEV, dtype=torch.int32)
            s["table"] = _table(case["rotary"], case["base"]) if case["rotary"] else None
            s["slots"][n - case["pad"]:] = -1
        return s
    lens = _lengths(case)
    random.Random(seed).shuffle(lens)
    width = max(1, -(-max(lens) // page))
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 3
    s["k_cache"], s["v_cache"] = _pool(gen, pages, page, heads, dim), _pool(gen, pages, page, heads, dim)
    order = torch.randperm(pages, generator=gen, device=DEV, dtype=torch.int32)
    table = torch.zeros(case["seqs"], width, dtype=torch.int32, device=DEV)
    column = torch.arange(width, device=DEV)
    taken = torch.tensor(used, device=DEV)
    table[column < taken[:, None]] = order[: sum(used)]
    s["block_table"], s["seq_lens"] = table, torch.tensor(lens, device=DEV, dtype=torch.int32)
    s["q"] = _normal(gen, case["seqs"], heads * case["group"], dim)
    s["scale"] = dim ** -0.5
    return s


def _cache(c):
    from nvfp4_block_scaled_22_b200 import binding as nb
    return nb.NVFP4Tensor(c["codes"], c["scales"], c["g"], c["codes"].shape[0], c["codes"].shape[1] * 2, nb.SF_LINEAR)


# ------------------------------------------------------------------- run
def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "rope":
        y = _rotated(s["x"], s["table"][s["positions"].long()], s["interleaved"], s["inverse"])
        return y.bfloat16()
    if op == "write":
        k = s["k"]
        if s["table"] is not None:
            k = _rotated(k, s["table"][s["positions"].clamp(min=0).long()], s["interleaved"], False).bfloat16()
        n = s["tokens"] - s["pad"]                                                # the padding rows are the last ones
        rows = s["slots"][:n].long()
        kc, vc = s["k_cache"], s["v_cache"]
        kc["codes"][rows], kc["scales"][rows] = _quantized(k[:n].flatten(1).float(), kc["g"])
        vc["codes"][rows], vc["scales"][rows] = _quantized(s["v"][:n].flatten(1).float(), vc["g"])
        return [_read_plain(kc, s["slots"]), _read_plain(vc, s["slots"])]
    if op == "read":
        return [_read_plain(s["k_cache"], s["slots"]), _read_plain(s["v_cache"], s["slots"])]
    return _attend_plain(s)


def _read_plain(c, slots):
    """Rows of a pool as BF16; zeros for slot -1."""
    rows = slots.clamp(min=0).long()
    x = _restored(c["codes"][rows], c["scales"][rows], c["g"])
    return torch.where(slots[:, None] >= 0, x, 0.0).bfloat16()


def _gathered(s, dtype):
    """Keys and values of all sequences [B, L, H, D] and which of them are there [B, L]."""
    page, table, lens = s["page"], s["block_table"], s["seq_lens"]
    t = torch.arange(table.shape[1] * page, device=DEV)
    there = t < lens[:, None]
    rows = torch.where(there, table[:, t // page].long() * page + t % page, 0)
    shape = (s["heads"], s["dim"])
    k = _values(s["k_cache"]["codes"][rows], s["k_cache"]["scales"][rows], dtype).unflatten(-1, shape)
    v = _values(s["v_cache"]["codes"][rows], s["v_cache"]["scales"][rows], dtype).unflatten(-1, shape)
    return k, v, there


def _attended(s, dtype):
    k, v, there = _gathered(s, dtype)
    q = s["q"].to(dtype).unflatten(1, (s["heads"], s["group"]))                   # [B, H, G, D]
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * (s["scale"] / s["k_cache"]["g"].to(dtype))
    x = x.masked_fill(~there[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(dtype).min)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / total.clamp(min=torch.finfo(dtype).tiny) / s["v_cache"]["g"].to(dtype)
    return o.flatten(1, 2), (top + torch.log(total)).flatten(1)


def _attend_plain(s):
    o, lse = _attended(s, torch.float32)
    return {"o": o.bfloat16(), "lse": lse}


def _run_own(s):
    from nvfp4_block_scaled_22_b200 import binding as nb
    op = s["op"]
    if op == "rope":
        return nb.nvfp4_rope(s["x"], s["positions"], s["table"], interleaved=s["interleaved"], inverse=s["inverse"])
    kc, vc = _cache(s["k_cache"]), _cache(s["v_cache"])
    if op == "write":
        nb.nvfp4_kv_write(s["k"], s["v"], s["slots"], kc, vc, positions=s["positions"], table=s["table"], interleaved=s["interleaved"])
        return list(nb.nvfp4_kv_read(kc, vc, s["slots"]))
    if op == "read":
        return list(nb.nvfp4_kv_read(kc, vc, s["slots"]))
    o, lse = nb.nvfp4_attention_decode_paged(s["q"], kc, vc, s["heads"], s["block_table"], s["seq_lens"], s["page"], scale=s["scale"], return_lse=True)
    return {"o": o, "lse": lse}


# ----------------------------------------------------------------- exact
def exact(case, seed):
    """The operators' definitions in 64 bits, one head or one sequence at a time."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "rope":
        return _turned(s["x"], s["positions"], case, -1.0 if case["inverse"] else 1.0)
    if case["op"] == "write":
        k = s["k"]
        if case["rotary"]:
            k = _turned(k, s["positions"], case, 1.0).bfloat16()
        there = (s["slots"] >= 0)[:, None]
        return [_nearest(k.flatten(1), s["k_cache"]["g"]) * there, _nearest(s["v"].flatten(1), s["v_cache"]["g"]) * there]
    if case["op"] == "read":
        return [_meant(s[c], s["slots"].long()) / s[c]["g"].to(f64) for c in ("k_cache", "v_cache")]
    out, lses = [], []
    for b, n in enumerate(s["seq_lens"].tolist()):
        t = torch.arange(n, device=DEV)
        rows = s["block_table"][b].long()[t // case["page"]] * case["page"] + t % case["page"]
        for h in range(case["heads"]):
            cut = slice(h * case["dim"], (h + 1) * case["dim"])
            k = _meant(s["k_cache"], rows, cut) / s["k_cache"]["g"].to(f64)
            v = _meant(s["v_cache"], rows, cut) / s["v_cache"]["g"].to(f64)
            x = s["q"][b, h * case["group"]:(h + 1) * case["group"]].to(f64) @ k.T * s["scale"]
            lse = torch.logsumexp(x, -1) if n else torch.full((case["group"],), float("-inf"), device=DEV, dtype=f64)
            out.append(torch.exp(x - lse[:, None]) @ v if n else torch.zeros(case["group"], case["dim"], device=DEV, dtype=f64))
            lses.append(lse)
    return {"o": torch.cat(out).view(case["seqs"], -1, case["dim"]), "lse": torch.cat(lses).view(case["seqs"], -1)}


def _turned(x, positions, case, sign):
    """Rotation as a product of complex numbers, of the pairs one after another."""
    y, n, f64 = x.double(), case["rotary"] // 2, torch.float64
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + n)
        angle = sign * positions.to(f64) * case["base"] ** (-2.0 * i / case["rotary"])
        z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.ones_like(angle), angle)[:, None]
        y[..., a], y[..., b] = z.real, z.imag
    return y


def _nearest(x, g):
    """What the rows stand for once they are held in 4 bits: each block's scale, then each value's nearest grid point, found by distance."""
    b, g = x.double().unflatten(-1, (-1, 16)), g.double()
    s = (b.abs().amax(-1, keepdim=True) * g / 6).clamp(max=448.0).float().to(torch.float8_e4m3fn).double()
    y = (b * g / s).nan_to_num(0.0)
    best, far = torch.zeros_like(y), torch.full_like(y, float("inf"))
    for v in (0.0, 1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0):                     # even codes first: they win a tie
        d = (y.abs() - v).abs()
        best, far = torch.where(d < far, v, best), torch.minimum(d, far)
    return (torch.copysign(best, b) * s / g).flatten(-2)


def _meant(c, rows, cut=slice(None)):
    """e2m1 * e4m3 of some rows (and columns) of a pool, from the bits of each code."""
    codes = c["codes"][rows, (cut.start or 0) // 2: cut.stop and cut.stop // 2].long()
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(1)
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1)) * (1 - 2.0 * (n >> 3))
    byte = c["scales"][rows, (cut.start or 0) // 16: cut.stop and cut.stop // 16].long()
    e, m = byte >> 3, (byte & 7).double() / 8
    return v * torch.where(e == 0, m * 2.0 ** -6, (1 + m) * torch.exp2(e.double() - 7)).repeat_interleave(16, 1)
