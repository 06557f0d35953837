"""The inputs of _shares.py in a four-bit cache, written as codes and pairs so that every number in them is exact, and
which form of the decode kernel a call takes.

A key's level is its code in channel 0 (scale 1, low 0; or, for a negative scale of the scores, low -12 and the code
12 - level), where the query is 1; its other channels hold any codes.  A value 2^(12 - level) in one channel is that
scale with codes of 9 there and 8 elsewhere over a low of -8 scales ("centred": low + 8 scale is 0), or with codes of 1
and 0 over a low of 0 ("plain": the sums over codes less 8 and over low + 8 scale cancel)."""
import os
import re

import torch

import _kv4
import _shares as sh

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rotation_int4_weight_amd", "csrc")


def rows_of(lev, kv_heads, dim, which, sign=1.0, centred=True, device="cpu"):
    """(codes (n, kv_heads, dim), pairs (n, kv_heads, dim / 64, 2)) of K and of V, and V's values in fp32."""
    lev = lev.to(device)
    n = lev.shape[0]
    _, v = sh.keys_and_values(lev, kv_heads, dim, which, device=device)
    codes = (torch.arange(n, device=device)[:, None, None] * 7 + torch.arange(dim, device=device) * 5 + 3) % 16
    codes = codes.expand(n, kv_heads, dim).clone()
    codes[:, :, 0] = (lev if sign > 0 else sh.TOP - lev)[:, None]
    pairs = torch.ones((n, kv_heads, dim // 64, 2), device=device)
    pairs[..., 1] = 0.0 if sign > 0 else -float(sh.TOP)
    step = (2.0 ** (sh.TOP - lev).float())[:, None, None, None].expand(n, kv_heads, dim // 64, 1)
    low = -8.0 * step if centred else 0.0 * step
    vc = (v > 0).long() + (8 if centred else 0)
    return (codes, pairs), (vc, torch.cat([step, low], -1)), v


def pages(codes, pairs, page, dtype, key):
    """Codes and pairs of n rows as the bytes of their pages (m, heads, page, 9 dim / 16); behind the last row codes of
    15 and pairs of NaN."""
    n, heads, dim = codes.shape
    m = -(-n // page)
    c = torch.full((m * page, heads, dim), 15, dtype=torch.long, device=codes.device)
    p = torch.full((m * page, *pairs.shape[1:]), float("nan"), device=codes.device)
    c[:n], p[:n] = codes, pairs
    c = c.view(m, page, heads, dim).transpose(1, 2)
    byte, bit = (t.to(codes.device) for t in _kv4.places(page, dim, key))
    out = torch.zeros((m, heads, page * dim // 2), dtype=torch.long, device=codes.device)
    out.index_add_(2, byte.flatten(), (c << bit).flatten(2))
    p = p.view(m, page, heads, -1).transpose(1, 2).to(dtype).contiguous().view(torch.uint8).flatten(2)
    return torch.cat([out.to(torch.uint8), p], -1).view(m, heads, page, dim * 9 // 16)


def expected(lev, v, q_heads, dtype, centred=True):
    """(y, limit) (1, q_heads, dim) of a row that sees all keys, in 64 bits; v of rows_of.

    Scores are exact products of the level with scale * log2 e, a weight is off by less than 2^-18 of itself (_shares.py),
    and weight times scale, a power of two but for that, rounds to it; the codes' sums are whole numbers of it.  As there
    2^-12 covers moved maxima and joins for both sums, n 2^-24 the sum of the weights, one rounding y.  Plain: each
    key's 8 weight * scale are added exactly and taken off to 2^-18."""
    w, n = 2.0 ** lev.to(v.device).double(), lev.shape[0]
    y = (w[:, None, None] * v.double()).sum(0) / w.sum()
    y = y.repeat_interleave(q_heads // v.shape[1], 0)[None]
    limit = y * (sh.HALF_STEP[dtype] + 2.0 ** -12 + (n + 64) * 2.0 ** -24)
    limit = limit + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    if not centred:
        limit = limit + 8 * n * 2.0 ** (sh.TOP - 18) / w.sum()
    return y, limit


def wrong(got, y, limit):
    """Where got (rows, q_heads, dim) of rows over the same keys is off by more than it may be."""
    return ~((got.double() - y).abs() <= limit)


def check(got, lev, v, centred=True):
    y, limit = expected(lev, v, got.shape[1], got.dtype, centred)
    bad = wrong(got, y, limit)
    if bool(bad.any()):
        at = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{int(bad.sum())} values of {bad.numel()} wrong, first at (row, head, channel) {at}: "
                             f"{float(got[at]):.6g}, {float(y[0][at[1:]]):.6g} expected")


def _constant(text, name):
    return int(re.search(r"\b%s = (\d+)[;,]" % name, text).group(1))


def form(lengths, q_heads, kv_heads, max_len):
    """How the kernel deals out a call over rows of these lengths: "output" (a workgroup for each output, looked up),
    "cut" (shares, outputs cut between workgroups), "wave" (outputs to waves), "rows" (a workgroup for each output, more
    rows than are looked up); and whether it is the kernel for many outputs.  The rules of attention_decode4.hip, with
    the constants that stand there."""
    with open(os.path.join(CSRC, "attention_decode4.hip")) as f:
        text = f.read()
    with open(os.path.join(CSRC, "attention.hpp")) as f:
        text += f.read()
    unit, start = 4 * _constant(text, "kStep"), _constant(text, "kOutputUnits")
    assert "constexpr int kUnit = kStep * kDecodeWaves;" in text
    assert "p.whole = outputs <= p.workgroups ? 5 + (int)outputs / 48 : 0;" in text
    assert "p.dealt = rows <= kMaxDealtRows && most < int64_t(1) << 30;" in text
    assert "longest * kLoneLongest > of_wave * kLoneShare" in text
    of_row = kv_heads * -(-(q_heads // kv_heads) // 16)
    outputs = len(lengths) * of_row
    most = outputs * (max(1, -(-max_len // unit)) + start)
    if len(lengths) > _constant(text, "kMaxDealtRows") or most >= 1 << 30:
        return "rows", True
    workgroups = min(most, 256 * _constant(text, "kDecode4Resident"))
    units = [max(1, -(-n // unit)) for n in lengths]
    whole = 5 + outputs // 48 if outputs <= workgroups else 0
    if whole:
        return ("output" if max(units) <= whole else "cut"), False
    share = -(-sum(u + start for u in units) * of_row // workgroups)
    lone = max(units) * _constant(text, "kLoneLongest") <= -(-share // 4) * _constant(text, "kLoneShare")
    return ("wave" if lone else "cut"), True
