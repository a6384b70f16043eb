"""Plain 64-bit forms of the paged-cache operators (test infrastructure):
rotary positions, decode attention over gathered rows, and the error bounds
that the GPU tests use."""
import numpy as np
import torch

U = 2.0 ** -24
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(b & 7) / 8 * 2.0 ** -6 if b >> 3 == 0 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7)
                 for b in range(128)])
E4M3[127] = np.nan


def bf16(a):
    """BF16 tensor of a 64-bit array (rounded through FP32)."""
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


def bits(t):
    return t.detach().contiguous().view(torch.int16)


def restore(codes, scales):
    """e2m1 * e4m3 of rows [n, c/2], [n, c/16] of bytes, exact in 64 bits."""
    n = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), np.int64)
    n[..., 0::2], n[..., 1::2] = codes & 15, codes >> 4
    return GRID[n & 7] * np.where(n & 8, -1.0, 1.0) * np.repeat(E4M3[scales & 127], 16, axis=-1)


def rope(x, cos, sin, interleaved, inverse=False):
    """x [T, H, D], cos and sin [T, pairs], all in one precision."""
    n = cos.shape[1]
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    c, s = cos[:, None], -sin[:, None] if inverse else sin[:, None]
    y = x.copy()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def attention(q, k, v, scale):
    """One sequence: q [H, G, D], k and v [T, H, D] in 64 bits.  Returns o,
    lse, sum p |v| / sum p and the largest |scale| sum |q k| of each head."""
    heads, group, dim = q.shape
    o, ao = np.zeros(q.shape), np.zeros(q.shape)
    lse, sa = np.full((heads, group), -np.inf), np.zeros((heads, group))
    if k.shape[0]:
        s = scale * np.einsum("hgd,thd->hgt", q, k)
        sa = abs(scale) * np.einsum("hgd,thd->hgt", np.abs(q), np.abs(k)).max(-1)
        top = s.max(-1, keepdims=True)
        p = np.exp(s - top)
        total = p.sum(-1, keepdims=True)
        o = np.einsum("hgt,thd->hgd", p / total, v)
        ao = np.einsum("hgt,thd->hgd", p / total, np.abs(v))
        lse = (top + np.log(total))[..., 0]
    return o, lse, ao, sa


def attention_bounds(o, lse, ao, sa, tokens, dim, vmax):
    """Allowed errors of o and lse.

    Scores: exact products of the FP16 query (BF16 values scaled by a power
    of two: exact down to 2^-29 of the largest of a head) and the restored
    key, dim / 16 tensor-core steps of 16 terms, each off by at most 2 ulp of
    its terms' magnitudes (8.5 u of the sum of magnitudes a step is more than
    all lose), then one fused multiply-add: eps_s = (8.5 dim / 16 + 4) u sa.
    Weights: 2^x in FP32 (2 ulp and the rescales: 8 u) and, for the product
    with V, rounded to FP16: 2^-11 of the weight, or 2^-25 where it is
    subnormal, which is 2^-31 of the largest weight (they are scaled so that
    the largest is at least 2^6).
    Sums: FP32, at most one accumulation chain of tokens / 16 steps off by
    2 ulp each in parts joined in FP32: (tokens / 8 + 64) u of the magnitudes,
    for the weighted and the plain sum.  The final divisions: 4 u.
    A weighted mean moves by at most 2 eps of its magnitudes when the weights
    move by eps; the output is rounded to BF16 (2^-8)."""
    eps_s = (8.5 * dim / 16 + 4) * U * sa[..., None]
    rest = (tokens / 8 + 64) * U
    eps = 2 * (eps_s + 8 * U) + 2.0 ** -11 + 2 * rest + 4 * U
    o_bound = eps * ao + tokens * 2.0 ** -31 * vmax
    o_bound = o_bound + 2.0 ** -8 * (np.abs(o) + o_bound) + 1e-38
    lse_bound = eps_s[..., 0] + 8 * U + rest + 4 * U * np.abs(np.where(np.isfinite(lse), lse, 0.0)) + 4 * U
    return o_bound, lse_bound


def inv_freq(rotary, base):
    return base ** (-2.0 * np.arange(rotary // 2) / rotary)


def turned_bound(x, rotary, interleaved):
    """sum of |x1| + |x2| of each value's pair: the magnitudes a rotation adds."""
    n = rotary // 2
    a = np.abs(x)
    m = a.copy()
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    m[..., i] = m[..., j] = a[..., i] + a[..., j]
    return m
