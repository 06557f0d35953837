"""Shared by the attention and cache tests: the definition in 64 bits on the
host, the error bound that the arithmetic gives, and caches with random pages."""
import math

import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def attention_f64(q, k, v, scale, causal=True):
    """One sequence, one key-value head: q (Hg, n_q, D), k, v (n_k, D), all float64 on the host.

    Masked places are left out, not multiplied by zero.  Returns y (Hg, n_q, D) and the bound of |y - result|."""
    heads, n_q, dim = q.shape
    n_k = k.shape[0]
    y = torch.zeros((heads, n_q, dim), dtype=torch.float64)
    spread = torch.zeros((heads, n_q, 1), dtype=torch.float64)
    for i in range(n_q):
        seen = min(n_k, i + 1 + n_k - n_q) if causal else n_k
        if seen <= 0:
            continue
        s = (q[:, i] @ k[:seen].t()) * scale
        p = torch.softmax(s, -1)
        y[:, i] = p @ v[:seen]
        # fp32 scores: products exact, a sum of `dim` terms and a few roundings more
        ds = (dim + 8) * 2.0 ** -24 * scale * (q[:, i].abs() @ k[:seen].abs().t()).amax(-1, keepdim=True)
        vmax = v[:seen].abs().max()
        spread[:, i] = vmax * (4 * ds + (seen + 16) * 2.0 ** -24)
    return y, spread


def bound(y, spread, vmax, dtype):
    """Weights rounded to the type (half a step each, on both sides of the division) and the output's rounding; a
    16-bit float's steps below its normal range are absolute."""
    u = HALF_STEP[dtype]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    return u * y.abs() + 2 * (u + tiny) * vmax + 1.01 * spread + tiny


def check_rows(got, q, k, v, scale, causal=True):
    """got, q: (n_q, Hq, D), k, v: (n_k, Hkv, D) of one sequence, any device."""
    dtype = got.dtype
    got, q, k, v = (t.detach().cpu().double() for t in (got, q, k, v))
    group = q.shape[1] // max(1, k.shape[1])
    for h in range(k.shape[1]):
        hs = slice(h * group, (h + 1) * group)
        y, spread = attention_f64(q[:, hs].transpose(0, 1), k[:, h], v[:, h], scale, causal)
        vmax = v[:, h].abs().max() if v.shape[0] else 0.0
        off = (got[:, hs].transpose(0, 1) - y).abs()
        limit = bound(y, spread, vmax, dtype)
        assert bool((off <= limit).all()), (
            f"kv head {h}: off by {float(off.max()):.3e}, at most {float(limit[off > limit].min()):.3e} allowed "
            f"({int((~(off <= limit)).sum())} values)")


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, device="cuda", generator=g)).to(dtype)


def offsets(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return torch.tensor(out, dtype=torch.int64, device="cuda")


def filled_cache(paro, lengths, page_size, kv_heads, dim, dtype, seed, layers=1, spare=5, extra=2):
    """A cache whose slot i holds lengths[i] positions in randomly ordered pages; what lies behind a sequence's end
    in its last page, and in free pages, is NaN."""
    counts = [-(-n // page_size) for n in lengths]
    pages = sum(counts) + spare
    c = paro.KVCache.empty(layers, pages, kv_heads, page_size, dim, len(lengths), max(counts + [0]) + extra, dtype)
    c.k.fill_(float("nan"))
    c.v.fill_(float("nan"))
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full(c.table.shape, -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    for i, n in enumerate(lengths):
        for j in range(counts[i]):
            page = order.pop()
            table[i, j] = page
            refs[page] = 1
            rows = min(page_size, n - j * page_size)
            for layer in range(layers):
                c.k[layer, page, :, :rows] = randn((kv_heads, rows, dim), dtype, seed + 7 * page + layer)
                c.v[layer, page, :, :rows] = randn((kv_heads, rows, dim), dtype, seed + 7 * page + layer + 3)
    c.table.copy_(table)
    c.refs.copy_(refs)
    c.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
    return c


def cached_rows(c, layer, slot, n=None):
    """K and V rows (n, kv_heads, dim) that slot holds, gathered by the host's reading of the table."""
    n = int(c.lengths[slot]) if n is None else n
    page = c.k.shape[3]
    at = torch.arange(n, device=c.k.device)
    where = c.table[slot].long()[at // page]
    return c.k[layer, where, :, at % page], c.v[layer, where, :, at % page]


def default_scale(dim):
    return 1.0 / math.sqrt(dim)
