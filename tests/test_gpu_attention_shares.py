"""Every key is counted once, by its own weight and with its own value: the
inputs of _shares.py through every form of the attention kernels (packed and
cached prompts, whole, in halves, split between waves and over workgroups;
decode with one part, two and many)."""
import pytest

import _shares as sh
from _attention import offsets

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]
NAN = float("nan")


def packed(counts, k_counts, heads, kv_heads, dim, dtype, pattern, causal=True, passes=None):
    levs = [sh.levels(n, pattern, n + i) for i, n in enumerate(k_counts)]
    q = sh.queries(sum(counts), heads, dim, dtype, "cuda")
    for p in range(passes or sh.windows(max(k_counts), dim)):
        parts = [sh.keys_and_values(lev, kv_heads, dim, p, device="cuda") for lev in levs]
        k, v = (torch.cat(x).to(dtype) for x in zip(*parts))
        y = torch.full_like(q, NAN)
        paro.paro_attention_prompt(q, k, v, offsets(counts), offsets(k_counts), y, scale=sh.LOG2, causal=causal)
        at = 0
        for n, lev, (_, one) in zip(counts, levs, parts):
            sh.check(y[at:at + n], lev, one, causal)
            at += n


def paged(lengths, page, kv_heads, dim, dtype, seed, extra=2):
    """An empty cache whose slots have room for `lengths`, in pages of random order; NaN everywhere."""
    counts = [-(-n // page) for n in lengths]
    pages = sum(counts) + 3
    c = paro.KVCache.empty(1, pages, kv_heads, page, dim, len(lengths), max(counts) + extra, dtype)
    c.k.fill_(NAN)
    c.v.fill_(NAN)
    order, at = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int().cuda(), 0
    for i, m in enumerate(counts):
        c.table[i, :m] = order[at:at + m]
        c.refs[order[at:at + m].long()] = 1
        at += m
    c.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
    return c


def fill(c, slot, k, v):
    at = torch.arange(k.shape[0], device="cuda")
    page = c.k.shape[3]
    where = c.table[slot].long()[at // page]
    c.k[0, where, :, at % page], c.v[0, where, :, at % page] = k.to(c.dtype), v.to(c.dtype)


def cached(lengths, new, heads, kv_heads, dim, page, dtype, pattern, causal=True, split=False):
    c = paged(lengths, page, kv_heads, dim, dtype, len(lengths))
    levs = [sh.levels(n, pattern, n + i) for i, n in enumerate(lengths)]
    q = sh.queries(sum(new), heads, dim, dtype, "cuda")
    need = paro.paro_attention_prompt_cached_workspace_bytes(c, len(new), sum(new), heads)
    assert need > 0 or not split
    ws = paro.make_workspace(need) if split else None
    slots = torch.arange(len(new), dtype=torch.int32, device="cuda")
    for p in range(sh.windows(max(lengths), dim)):
        parts = [sh.keys_and_values(lev, kv_heads, dim, p, device="cuda") for lev in levs]
        for s, (k, v) in enumerate(parts):
            fill(c, s, k, v)
        y = torch.full_like(q, NAN)
        paro.paro_attention_prompt_cached(c, 0, q, slots, offsets(new), y, scale=sh.LOG2, causal=causal, workspace=ws)
        at = 0
        for n, lev, (_, v) in zip(new, levs, parts):
            sh.check(y[at:at + n], lev, v, causal)
            at += n


def decode(lengths, heads, kv_heads, dim, page, dtype, pattern, extra=2, passes=None):
    c = paged(lengths, page, kv_heads, dim, dtype, len(lengths), extra)
    levs = [sh.levels(n, pattern, n + i) for i, n in enumerate(lengths)]
    rows = len(lengths)
    q = sh.queries(rows, heads, dim, dtype, "cuda")
    slots = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda")
    ws = paro.make_workspace(paro.paro_attention_decode_workspace_bytes(c, rows, heads))
    for p in range(passes or sh.windows(max(lengths), dim)):
        parts = [sh.keys_and_values(lev, kv_heads, dim, p, device="cuda") for lev in levs]
        for s, (k, v) in enumerate(parts):
            fill(c, s, k, v)
        y = torch.full_like(q, NAN)
        paro.paro_attention_decode(c, 0, q, slots, y, ws, scale=sh.LOG2)
        for r in range(rows):
            s = rows - 1 - r
            sh.check(y[r:r + 1], levs[s], parts[s][1])


# workgroups of 32 rows whose waves share the keys; of 128 rows with four waves; the same with eight, keys in halves
PACKED = [([700], [700], 4, 1), ([3, 40], [2222, 1000], 4, 1),
          ([400, 129, 65, 1], [400, 129, 65, 1], 16, 8), ([150, 200, 3], [1033, 270, 3], 56, 8),
          ([800], [800], 16, 8), ([600, 65, 1], [640, 1500, 1300], 16, 8), ([900], [780], 16, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("counts,k_counts,heads,kv_heads", PACKED)
def test_prompt_counts_each_key_once(counts, k_counts, heads, kv_heads, dim, dtype):
    for pattern in sh.PATTERNS:
        packed(counts, k_counts, heads, kv_heads, dim, dtype, pattern)
    packed(counts, k_counts, heads, kv_heads, dim, dtype, "blocks", causal=False)


def test_long_prompt_counts_each_key_once():
    for dtype, dim, pattern in ((torch.bfloat16, 128, "blocks"), (torch.float16, 64, "rising")):
        packed([4100], [4100], 32, 8, dim, dtype, pattern, passes=2)


CACHED = [([700, 33, 1], [5, 33, 1], 4, 1), ([1217, 300, 90], [64, 200, 90], 56, 8),
          ([900, 400, 5], [880, 270, 5], 64, 16), ([2100], [800], 16, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (128, 16), (64, 256)])
@pytest.mark.parametrize("lengths,new,heads,kv_heads", CACHED)
def test_chunk_counts_each_key_once(lengths, new, heads, kv_heads, dim, page, dtype):
    for pattern in sh.PATTERNS:
        cached(lengths, new, heads, kv_heads, dim, page, dtype, pattern)
    cached(lengths, new, heads, kv_heads, dim, page, dtype, "rising", causal=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,page,heads,kv_heads", [(64, 16, 7, 1), (128, 32, 8, 2), (128, 16, 4, 4)])
def test_chunk_in_parts_counts_each_key_once(dim, page, heads, kv_heads, dtype):
    for pattern in sh.PATTERNS:
        cached([5000], [6], heads, kv_heads, dim, page, dtype, pattern, split=True)
        cached([2300, 513, 40, 1024, 512], [33, 5, 40, 2, 1], heads, kv_heads, dim, page, dtype, pattern, split=True)
    cached([9001], [40], heads, kv_heads, dim, page, dtype, "blocks", split=True)
    cached([1500, 600], [17, 40], heads, kv_heads, dim, page, dtype, "falling", causal=False, split=True)


DECODE = [([1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 384], 4, 1),
          ([5000, 385, 384], 8, 2), ([9001, 17, 4096], 2, 2), ([3000], 17, 1),
          ([700, 385, 1100, 900] * 10, 8, 8), ([450, 1000, 33] * 22, 16, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (128, 256)])
@pytest.mark.parametrize("lengths,heads,kv_heads", DECODE)
def test_decode_counts_each_key_once(lengths, heads, kv_heads, dim, page, dtype):
    for pattern in sh.PATTERNS:
        decode(lengths, heads, kv_heads, dim, page, dtype, pattern)


@pytest.mark.parametrize("dtype", TYPES)
def test_decode_with_a_spare_table_counts_each_key_once(dtype):
    """A table far longer than the sequences: parts of the least length."""
    for pattern in sh.PATTERNS:
        decode([5000, 385, 40], 4, 1, 128, 16, dtype, pattern, extra=9000)
    decode([131072, 40], 8, 2, 64, 64, dtype, "blocks", passes=2)
