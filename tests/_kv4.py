"""Shared by the tests of the four-bit cache: its format written from the
documented layout, one address at a time, and attention over it in 64 bits."""
import math

import torch

ORDER = (0, 2, 4, 6, 1, 3, 5, 7)
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def quantise(x):
    """x (..., D) in 16 bits on the host: codes (..., D) int64, scale and low (..., D / 64) in x's type."""
    g = x.unflatten(-1, (-1, 64)).double()
    low, high = g.amin(-1), g.amax(-1)
    scale = ((high - low) / 15).float().to(x.dtype)
    bad = ~torch.isfinite(g).all(-1)
    s = scale.double()[..., None]
    codes = torch.where(s > 0, ((g - low[..., None]) / torch.where(s > 0, s, 1.0)).round().clamp(0, 15), 0.0)
    codes = torch.where(bad[..., None], torch.zeros_like(codes), codes).long().flatten(-2)
    nan = torch.tensor(float("nan"), dtype=x.dtype)
    return codes, torch.where(bad, nan, scale), torch.where(bad, nan, low.to(x.dtype))


def stands_for(codes, scale, low):
    """low + scale * code in 64 bits."""
    c = codes.unflatten(-1, (-1, 64)).double()
    return (low.double()[..., None] + scale.double()[..., None] * c).flatten(-2)


def places(page, dim, key):
    """(byte, bit) (page, dim) of every code in a head's page."""
    p, c = torch.arange(page)[:, None], torch.arange(dim)[None]
    if key:
        nibble = torch.tensor([ORDER.index(i) for i in range(8)])[c % 8].expand(page, dim)
        return 4 * ((p * 4 + c % 32 // 8) * (dim // 32) + c // 32) + nibble // 2, 4 * (nibble % 2)
    word = ((p // 4 * 16 + c % 64 // 4) * (dim // 64) + c // 64) * 4 + p % 4
    return 2 * word + c % 4 // 2, (4 * (c % 2)).expand(page, dim)


def pages_of(x, key):
    """x (n, heads, page, dim) on the host as the bytes of its pages (n, heads, page, 9 dim / 16)."""
    n, heads, page, dim = x.shape
    codes, scale, low = quantise(x)
    byte, bit = places(page, dim, key)
    out = torch.zeros((n, heads, page * dim // 2), dtype=torch.int64)
    out.index_add_(2, byte.flatten(), (codes << bit).flatten(2))
    pairs = torch.stack([scale, low], -1).contiguous().view(torch.uint8).flatten(2)
    return torch.cat([out.to(torch.uint8), pairs], -1).view(n, heads, page, dim * 9 // 16)


def values_of(pages, dtype, key):
    """The bytes of pages (n, heads, page, 9 dim / 16) as the values they hold, (n, heads, page, dim) in 64 bits."""
    pages = pages.cpu()
    n, heads, page, row = pages.shape
    dim = row * 16 // 9
    flat = pages.flatten(2)
    byte, bit = places(page, dim, key)
    codes = flat[:, :, byte.flatten()].long().view(n, heads, page, dim) >> bit & 15
    pairs = flat[:, :, page * dim // 2:].contiguous().view(dtype).view(n, heads, page, dim // 64, 2)
    return stands_for(codes, pairs[..., 0], pairs[..., 1])


def held_rows(c, layer, slot, n=None):
    """K and V (n, kv_heads, dim) in 64 bits of what a slot of a four-bit cache holds."""
    n = int(c.lengths[slot]) if n is None else n
    page = c.k.shape[3]
    where = c.table[slot, :-(-n // page)].long()
    return tuple(values_of(t[layer, where], c.dtype, key).transpose(1, 2).flatten(0, 1)[:n]
                 for t, key in ((c.k, True), (c.v, False)))


def fill(paro, lengths, page_size, kv_heads, dim, dtype, seed, layers=1, spare=5, extra=2, k_scale=1.0, v_scale=1.0,
         garbage=0xFF):
    """A four-bit cache whose slot i holds lengths[i] random positions in randomly ordered pages; everything behind a
    sequence's end, and free pages, is `garbage` (0xFF: pairs of NaN, codes of 15)."""
    counts = [-(-n // page_size) for n in lengths]
    pages = sum(counts) + spare
    g = torch.Generator().manual_seed(seed)
    c = paro.KVCache.empty(layers, pages, kv_heads, page_size, dim, len(lengths), max(counts + [0]) + extra, dtype,
                           bits=4)
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full(c.table.shape, -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    size = page_size * dim // 2
    pools = []
    for key, scale in ((True, k_scale), (False, v_scale)):
        x = scale * torch.randn((layers * pages, kv_heads, page_size, dim), generator=g)
        pools.append(pages_of(x.to(dtype), key).view(layers, pages, kv_heads, page_size, -1))
    behind = [torch.full_like(p, garbage) for p in pools]
    for i, n in enumerate(lengths):
        for j in range(counts[i]):
            page = order.pop()
            table[i, j], refs[page] = page, 1
            rows = min(page_size, n - j * page_size)
            for pool, out, key in ((pools[0], behind[0], True), (pools[1], behind[1], False)):
                a, b = pool[:, page].flatten(2), out[:, page].flatten(2).clone()
                b[..., size:size + rows * dim // 16] = a[..., size:size + rows * dim // 16]
                # bytes of codes belong to one position each
                byte = places(page_size, dim, key)[0][:rows].flatten().unique()
                b[..., byte] = a[..., byte]
                out[:, page] = b.view(out[:, page].shape)
    c.k.copy_(behind[0])
    c.v.copy_(behind[1])
    c.table.copy_(table)
    c.refs.copy_(refs)
    c.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
    return c


def check_decode(got, q, k, v, scale):
    """got, q (Hq, D) of one row; k, v (n, Hkv, D) in 64 bits, as the cache holds them.

    The bound: fp32 scores (terms of |q| times the largest |low| + 15 scale that values of size vmax can have, at most
    three times their size, summed by the matrix cores, which may cut terms at 2^-23 of the largest); weights times
    scales rounded to fp16 (half a step each, multiplied by codes less 8: at most 8 / 15 of a group's range, which is at
    most 2 vmax; an absolute 2^-40 of the largest scale below the type's normal range); the sums of n terms; the
    output's rounding."""
    dtype = got.dtype
    got, q = got.detach().cpu().double(), q.detach().cpu().double()
    n, kv_heads, dim = k.shape
    if n == 0:
        assert bool((got == 0).all())
        return
    group = q.shape[0] // kv_heads
    u = HALF_STEP[dtype]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    for h in range(kv_heads):
        mine = slice(h * group, (h + 1) * group)
        s = q[mine] @ k[:, h].t() * scale
        y = torch.softmax(s, -1) @ v[:, h]
        vmax, kmax = float(v[:, h].abs().max()), float(k[:, h].abs().max())
        terms = abs(scale) * q[mine].abs().sum(-1, keepdim=True) * 3 * kmax
        ds = (dim + 16) * 2.0 ** -23 * terms + (s.abs().amax(-1, keepdim=True) * 1.5 + 160) * 2.0 ** -23
        weights = 2 * vmax * (2.0 ** -11 + n * 2.0 ** -36)
        limit = u * y.abs() + tiny + 1.01 * (weights + vmax * (4 * ds + (n + 40) * 2.0 ** -22))
        off = (got[mine] - y).abs()
        assert bool((off <= limit).all()), (
            f"kv head {h}: off by {float(off.max()):.3e}, at most {float(limit.max()):.3e} allowed "
            f"({int((~(off <= limit)).sum())} values)")


def default_scale(dim):
    return 1.0 / math.sqrt(dim)
