"""Definition of the paged FP8 cache and of attention over it in 64 bits, for
the tests: written from the format (E4M3 codes, power-of-two scales)."""
import math

import numpy as np
import torch


def e4m3_values():
    b = np.arange(256)
    exp, man = (b >> 3) & 15, b & 7
    val = np.where(exp == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (exp - 10.0)) * np.where(b & 128, -1.0, 1.0)
    val[[127, 255]] = np.nan
    return val


GRID = e4m3_values()
SCALES = np.concatenate([np.ldexp(1.0, np.arange(255) - 127), [np.nan]])


def quantise(x):
    """Codes [..., 128] and scale bytes [...] of an array of vectors, element by element from the definition."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(-1)
    y = np.where(bad[..., None], 0.0, x)
    amax = np.abs(y).max(-1)
    byte = np.searchsorted(448.0 * SCALES[:255], amax)          # the first scale that reaches amax
    byte = np.where(amax == 0, 127, byte)
    z = y / SCALES[byte][..., None]
    mid = (GRID[:126] + GRID[1:127]) / 2
    i = np.searchsorted(mid, np.abs(z))
    i = np.where((np.abs(z) == mid[np.minimum(i, 125)]) & (i % 2 == 1), i + 1, i)    # a tie goes to the even code
    codes = (i | np.where(np.signbit(z), 128, 0)).astype(np.uint8)
    codes[bad] = 0
    return codes, np.where(bad, 255, byte).astype(np.uint8)


def values(codes, scales):
    """64-bit values of codes [..., 128] (uint8 tensor) and scale bytes [...]."""
    g = torch.tensor(GRID, device=codes.device)[codes.long()]
    return g * torch.tensor(SCALES, device=codes.device)[scales.long()].unsqueeze(-1)


def attention(q, kv, q_lens, kv_lens, group, *, causal=True, window=None, scale=None):
    """O, log-sum, and what the error bounds need, in 64 bits.

    kv: per sequence a pair (K, V) of [len, heads, 128].  Returns (o, lse, av,
    sq) over all rows: av = sum_j p_j |v_j| per channel, sq = the largest
    scale * sum_i |q_i k_ij| over the keys seen."""
    scale = scale or 1.0 / math.sqrt(128)
    res = [[], [], [], []]
    at = 0
    for (k, v), ql, kl in zip(kv, q_lens, kv_lens):
        x = q[at:at + ql].double()
        at += ql
        hq = x.shape[1]
        k, v = (torch.nan_to_num(t[:kl], nan=math.nan).double().repeat_interleave(group, 1) for t in (k, v))
        if kl == 0:
            z = torch.zeros((ql, hq, 128), dtype=torch.float64, device=q.device)
            low = torch.full((ql, hq), -math.inf, dtype=torch.float64, device=q.device)
            for r, t in zip(res, (z, low, z, z[..., 0])):
                r.append(t)
            continue
        s = torch.einsum("thd,jhd->htj", x, k) * scale
        mag = torch.einsum("thd,jhd->htj", x.abs(), k.abs()) * scale
        seen = torch.ones((ql, kl), dtype=torch.bool, device=q.device)
        if causal:
            pos = torch.arange(kl - ql, kl, device=q.device).unsqueeze(1)
            j = torch.arange(kl, device=q.device)
            seen = j <= pos
            if window:
                seen &= j > pos - window
        s = torch.where(seen, s, -math.inf)
        lse = torch.logsumexp(s, -1)
        p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse).unsqueeze(-1))
        p = torch.where(seen, p, 0.0)
        # a row sees only its own keys: what others hold, NaN too, is not multiplied in
        vz = torch.nan_to_num(v, nan=0.0)
        o = torch.einsum("htj,jhd->thd", p, vz)
        poison = torch.einsum("tj,jhd->thd", seen.double(), torch.isnan(v).double()) > 0
        o = torch.where(poison, math.nan, o)
        av = torch.einsum("htj,jhd->thd", p, vz.abs())
        sq = torch.where(seen, mag, 0.0).amax(-1).T
        for r, t in zip(res, (o, lse.T, av, sq)):
            r.append(t)
    return tuple(torch.cat(r) for r in res)


def error_bounds(o, lse, av, sq):
    """How far a kernel's O (BF16) and log-sum (FP32) may be from the above.

    Scores: their products are exact, the query enters in full (8 or 11 bits),
    and 128 of them are added in FP32 or wider blocks of it, each step off by
    2^-22 of the largest partial sum at most: |ds| <= 128 * 2^-22 * sq = 2^-15
    sq, and a few roundings of the final products, 2^-22 |s|.  A weight is off by
    e^ds - 1 (twice ds for numerator and sum together), by 2^-20 (exponent and
    sums in FP32), and by 2^-11 (half a step of FP16) where it meets V.  O is
    rounded to BF16 once: 2^-8 of what is rounded, which is itself off by the
    above."""
    ds = (2.0 ** -15 + 2.0 ** -22) * sq
    inner = (2.0 ** -11 + 2.0 ** -19 + 2.0 * ds.unsqueeze(-1)) * av
    eo = 2.0 ** -8 * (o.abs() + inner) + inner + 1e-38
    el = ds + 2.0 ** -20 + 2.0 ** -22 * torch.nan_to_num(lse, neginf=0.0).abs()
    return eo, el
