"""Attention inputs whose outputs say which keys were counted.

Key j has a whole level L_j in 0..12 (scores are levels: q = (1, 0, ...), k_j =
(sign * L_j, 0, ...), scale = sign * log 2), so its weight is 2^L_j, a number
that every 16-bit type holds.  In a window of 16 * dim keys, its value is
2^(12 - L_j) in one channel and 0 elsewhere: each key of the window adds the
same 2^12 to one channel's sum, a channel has 16 of them, and

    y[c] = 2^12 * (keys of the window that the row sees in c) / sum_j 2^L_j.

One key that is lost, counted twice, weighted or placed wrongly moves a channel
by 1/17 or more, far past the rounding; a head's windows of all passes cover all
keys.  No input is random but the levels."""
import math

import torch

TOP = 12
PER_CHANNEL = 16
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
PATTERNS = ["flat", "rising", "falling", "blocks", "first", "last"]


def levels(n, pattern, seed=0):
    """The levels of n keys: equal, moving the maximum all the way or never, by blocks of 32 keys at random, or one key
    far above the others."""
    at = torch.arange(n)
    if pattern == "rising":
        return at * TOP // max(1, n - 1)
    if pattern == "falling":
        return TOP - at * TOP // max(1, n - 1)
    if pattern == "blocks":
        g = torch.Generator().manual_seed(seed)
        return torch.randint(0, TOP + 1, (n // 32 + 1,), generator=g)[at // 32]
    out = torch.zeros(n, dtype=torch.long)
    if n and pattern in ("first", "last"):
        out[0 if pattern == "first" else -1] = TOP
    return out


def windows(n, dim):
    """Passes that it takes until every head's windows have covered n keys."""
    return max(1, -(-n // (PER_CHANNEL * dim)))


def keys_and_values(lev, kv_heads, dim, which, sign=1.0, device="cpu"):
    """k, v (n, kv_heads, dim), exact in fp32: pass `which` of windows()."""
    n = lev.shape[0]
    k = torch.zeros((n, kv_heads, dim), device=device)
    v = torch.zeros((n, kv_heads, dim), device=device)
    lev = lev.to(device)
    k[:, :, 0] = (sign * lev).float()[:, None]
    for h in range(kv_heads):
        a = (which + h) % windows(n, dim) * PER_CHANNEL * dim
        j = torch.arange(a, max(a, min(n, a + PER_CHANNEL * dim)), device=device)
        v[j, h, (j + 17 * h) % dim] = 2.0 ** (TOP - lev[j]).float()
    return k, v


def queries(rows, heads, dim, dtype, device):
    q = torch.zeros((rows, heads, dim), dtype=dtype, device=device)
    q[:, :, 0] = 1.0
    return q


def expected(lev, v, n_q, causal=True):
    """y (n_q, kv_heads, dim) in 64 bits for rows that see their keys (bottom right); v as keys_and_values gives it."""
    n = lev.shape[0]
    w = 2.0 ** lev.to(v.device).double()
    numer = torch.cat([torch.zeros((1, *v.shape[1:]), dtype=torch.float64, device=v.device),
                       (w[:, None, None] * v.double()).cumsum(0)])
    denom = torch.cat([torch.zeros(1, dtype=torch.float64, device=v.device), w.cumsum(0)])
    seen = torch.arange(n_q, device=v.device) + 1 + n - n_q if causal else torch.full((n_q,), n, device=v.device)
    seen = seen.clamp(0, n)
    return numer[seen] / denom[seen].clamp(min=1.0)[:, None, None]


def check(got, lev, v, causal=True):
    """got (n_q, q_heads, dim).  A score is off by at most 2 * 12 * 2^-23 (scale * log2 e, one fma), a weight by that
    and a step of exp2, under 2^-18; the maximum moves at most 12 times in a wave and the sums are joined at most three
    times, under 2^-13 for both sums of the quotient; adding n weights in fp32 at most n * 2^-24.  Weights rounded to
    the type are exact, and y is rounded once; 2^-25 is half a subnormal step of fp16."""
    n, dtype = lev.shape[0], got.dtype
    want = expected(lev, v, got.shape[0], causal)
    group = got.shape[1] // v.shape[1]
    want = want.repeat_interleave(group, 1)
    limit = want * (HALF_STEP[dtype] + 2.0 ** -12 + (n + 64) * 2.0 ** -24)
    limit = limit + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    off = (got.double() - want).abs()
    wrong = ~(off <= limit)
    assert not bool(wrong.any()), (
        f"{int(wrong.sum())} values of {wrong.numel()} wrong, first at (row, head, channel) "
        f"{torch.nonzero(wrong)[0].tolist()}: {float(got[wrong][0]):.6g}, {float(want[wrong][0]):.6g} expected")


LOG2 = math.log(2.0)
