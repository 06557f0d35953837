"""Attention over the four-bit cache in 64 bits, with a bound that weights what each key can add by its probability, so
that keys without weight do not widen it and a lost share of the weight shows."""
import torch

import _kv4

HALF_STEP = _kv4.HALF_STEP


def held(c, layer, slot):
    """(codes (n, heads, dim), scale, low (n, heads, dim / 64)) of K and of V, in 64 bits."""
    n, page, dim = int(c.lengths[slot]), c.c.page_size, c.c.head_dim
    where = c.table[slot, :-(-n // page)].long()
    out = []
    for t, key in ((c.k, True), (c.v, False)):
        flat = t[layer, where].cpu().flatten(2)
        byte, bit = _kv4.places(page, dim, key)
        codes = flat[:, :, byte.flatten()].long().view(*flat.shape[:2], page, dim) >> bit & 15
        pairs = flat[:, :, page * dim // 2:].contiguous().view(c.dtype).view(*flat.shape[:2], page, dim // 64, 2).double()
        out.append(tuple(x.transpose(1, 2).flatten(0, 1)[:n] for x in (codes.double(), pairs[..., 0], pairs[..., 1])))
    return out


def attention(q, k, v, scale):
    """q (heads, dim) of one row; k, v: held(): (y, limit) (heads, dim) in 64 bits.

    limit, for weights p_j of head h, with code_jc, s_ju, low_ju of a value and mid = low + 8 s, is the sum of
      scores    fp32 sums of terms T_j = |scale| sum_u (s_ju sum |q_c| code_jc + |low_ju| sum |q_c|), of which the matrix
                cores may cut 2^-23 of the largest, a query that is cut at 2^-35 of its row's largest, the score's own
                roundings, the exponent's (up to 2^-24 of 300) and a few of exp2: e_j; through the quotient
                sum_j p_j e_j (|v_jc| + |y_c|)
      products  p s rounded to fp16 (half a step), times code - 8: 2^-11 sum_j p_j s_ju |code_jc - 8|; below its normal
                range 2^-25 against at least 2^5 for the largest of them, times 8
      sums      n / 16 + 64 roundings of sums of p |s (code - 8)| + p |mid|
      output    half a step, of fp16 at least 2^-25."""
    dtype = q.dtype
    q = q.detach().cpu().double()
    (kc, ks, kl), (vc, vs, vl) = k, v
    n, kv_heads, dim = kc.shape
    group = q.shape[0] // kv_heads
    wide = lambda x: x.repeat_interleave(64, -1)  # noqa: E731
    ys, limits = [], []
    for h in range(kv_heads):
        mine = q[h * group:(h + 1) * group]
        key = wide(kl[:, h]) + wide(ks[:, h]) * kc[:, h]
        s = mine @ key.t() * scale
        p = torch.softmax(s, -1)
        val, step, mid = wide(vl[:, h]) + wide(vs[:, h]) * vc[:, h], wide(vs[:, h]), wide(vl[:, h] + 8 * vs[:, h])
        y = p @ val
        a = mine.abs()
        terms = abs(scale) * (a @ (wide(ks[:, h]) * kc[:, h]).t() + a @ wide(kl[:, h].abs()).t())
        cut = abs(scale) * 2.0 ** -35 * a.amax(-1, keepdim=True) * (wide(ks[:, h]) * 15 + wide(kl[:, h].abs())).sum(-1)
        e = (dim + 16) * 2.0 ** -23 * terms + cut + (1.5 * s.abs() + 300) * 2.0 ** -22
        e = e.clamp(max=1e6)
        off = (step * (vc[:, h] - 8)).abs()
        pe = p * e
        limit = pe @ val.abs() + pe.sum(-1, keepdim=True) * y.abs()
        limit += 2.0 ** -11 * (p @ off)
        largest = torch.stack([(p * vs[:, h, u]).amax(-1) for u in range(dim // 64)], -1)
        limit += 8 * n * 2.0 ** -30 * wide(largest)
        limit += (n / 16 + 64) * 2.0 ** -23 * (p @ (off + mid.abs()))
        limit = 1.01 * limit + HALF_STEP[dtype] * y.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)
        ys.append(y)
        limits.append(limit)
    return torch.cat(ys), torch.cat(limits)


def wrong(got, y, limit):
    """Where got is off by more than it may be."""
    return ~((got.detach().cpu().double() - y).abs() <= limit)


def check(got, q, k, v, scale):
    y, limit = attention(q, k, v, scale)
    bad = wrong(got, y, limit)
    if bool(bad.any()):
        at = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{int(bad.sum())} values of {bad.numel()} wrong, first at (head, channel) {at}: "
                             f"{float(got[at]):.6g}, {float(y[at]):.6g} expected, {float(limit[at]):.2g} allowed")
