"""Prompt and decode attention through the C-ABI against the definition in 64
bits: head layouts, ragged and empty sequences, rows that see no key, strides,
masked NaN, streams, and refusals that only the binding can make."""
import pytest

from _attention import cached_rows, check_rows, default_scale, filled_cache, offsets, randn

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")

pytestmark = pytest.mark.gpu

HEADS = [(1, 1), (4, 1), (7, 1), (32, 8), (6, 2), (40, 2)]
TYPES = [torch.float16, torch.bfloat16]
NAN = float("nan")


def run_prompt(q_counts, k_counts, heads, kv_heads, dim, dtype, causal=True, scale=None, seed=0, qs=1.5):
    q = randn((sum(q_counts), heads, dim), dtype, seed, qs)
    k = randn((sum(k_counts), kv_heads, dim), dtype, seed + 1)
    v = randn((sum(k_counts), kv_heads, dim), dtype, seed + 2)
    y = torch.full_like(q, NAN)
    paro.paro_attention_prompt(q, k, v, offsets(q_counts), offsets(k_counts), y, scale=scale, causal=causal)
    torch.cuda.synchronize()
    q0 = k0 = 0
    for a, b in zip(q_counts, k_counts):
        check_rows(y[q0:q0 + a], q[q0:q0 + a], k[k0:k0 + b], v[k0:k0 + b],
                   default_scale(dim) if scale is None else scale, causal)
        q0, k0 = q0 + a, k0 + b


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", HEADS)
def test_prompt_heads(heads, dim, dtype):
    run_prompt([33, 1, 70], [33, 1, 70], *heads, dim, dtype)


@pytest.mark.parametrize("dim,dtype", [(64, torch.bfloat16), (128, torch.float16)])
@pytest.mark.parametrize("counts", [[1], [2], [31], [32], [33], [63, 64, 65], [127, 128, 129], [0, 5, 0, 0, 1, 0],
                                    [257, 1, 3, 300], [1] * 70, [700]])
def test_prompt_lengths(counts, dim, dtype):
    run_prompt(counts, counts, 4, 1, dim, dtype, seed=len(counts))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_counts,k_counts", [([5, 3, 0, 7, 70], [2, 3, 4, 0, 300]), ([65], [64]), ([300], [10]),
                                               ([1, 1, 1], [129, 64, 0]), ([40], [1000]), ([0, 0], [5, 0])])
def test_prompt_fewer_and_more_keys_than_rows(q_counts, k_counts, causal):
    for dim, dtype, heads in ((128, torch.bfloat16, (8, 2)), (64, torch.float16, (3, 3))):
        run_prompt(q_counts, k_counts, *heads, dim, dtype, causal=causal, seed=3)


def test_prompt_scales_and_large_scores():
    for scale in (0.0, -0.3, 1.0):  # 1.0: scores to about +-100, weights concentrate on one key
        run_prompt([90], [90], 4, 2, 128, torch.bfloat16, scale=scale, qs=1.0, seed=5)
    run_prompt([90], [90], 4, 2, 64, torch.float16, scale=3.0, qs=1.0, seed=6)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,dtype", [(64, torch.bfloat16), (64, torch.float16), (128, torch.bfloat16),
                                       (128, torch.float16)])
def test_prompt_many_row_tiles(dim, dtype, causal):
    """More than 96 row tiles and key-value heads: workgroups of 128 rows that share their keys."""
    run_prompt([400, 129, 65, 1], [400, 129, 65, 1], 16, 8, dim, dtype, causal=causal, seed=11)
    run_prompt([150, 200, 3], [333, 70, 3], 56, 8, dim, dtype, causal=causal, seed=12)


@pytest.mark.parametrize("dim,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("q_counts,k_counts,causal", [([800], [800], True), ([769, 900], [769, 900], True),
                                                      ([600, 65, 1], [640, 1500, 300], True), ([800], [833], False),
                                                      ([900], [780], True)])
def test_prompt_keys_in_halves(q_counts, k_counts, causal, dim, dtype):
    """About one workgroup of 128 rows per CU and long sequences: its waves take the key tiles in two halves."""
    run_prompt(q_counts, k_counts, 16, 8, dim, dtype, causal=causal, seed=21)


@pytest.mark.parametrize("layout", ["fused", "heads_first"])
def test_prompt_strides_many_row_tiles(layout):
    n, heads, kv_heads, dim, dtype = 340, 64, 16, 64, torch.bfloat16
    if layout == "fused":
        rows = randn((n, heads + 2 * kv_heads, dim), dtype, 1)
        q, k, v = rows[:, :heads], rows[:, heads:heads + kv_heads], rows[:, heads + kv_heads:]
        y = torch.full((n, heads, dim + 8), NAN, dtype=dtype, device="cuda")[..., :dim]
    else:
        q, k, v = (randn((h, n, dim), dtype, i).transpose(0, 1) for i, h in enumerate((heads, kv_heads, kv_heads)))
        y = torch.full((heads, n, dim), NAN, dtype=dtype, device="cuda").transpose(0, 1)
    cu = offsets([140, 200])
    paro.paro_attention_prompt(q, k, v, cu, cu, y)
    for a, b in ((0, 140), (140, 340)):
        check_rows(y[a:b], q[a:b], k[a:b], v[a:b], default_scale(dim))


@pytest.mark.parametrize("layout", ["fused", "heads_first", "broadcast"])
def test_prompt_strides(layout):
    n, heads, kv_heads, dim, dtype = 75, 6, 2, 64, torch.float16
    if layout == "fused":  # q, k, v are slices of one projection's rows
        rows = randn((n, heads + 2 * kv_heads, dim), dtype, 1)
        q, k, v = rows[:, :heads], rows[:, heads:heads + kv_heads], rows[:, heads + kv_heads:]
        y = torch.full((n, heads, dim + 8), NAN, dtype=dtype, device="cuda")[..., :dim]
    elif layout == "heads_first":
        q, k, v = (randn((h, n, dim), dtype, i).transpose(0, 1) for i, h in enumerate((heads, kv_heads, kv_heads)))
        y = torch.full((heads, n, dim), NAN, dtype=dtype, device="cuda").transpose(0, 1)
    else:  # one key-value head seen as two, one query row seen as all
        q = randn((1, heads, dim), dtype, 0).expand(n, heads, dim)
        k, v = (randn((n, 1, dim), dtype, i).expand(n, kv_heads, dim) for i in (1, 2))
        y = torch.full((n, heads, dim), NAN, dtype=dtype, device="cuda")
    cu = offsets([40, 35])
    paro.paro_attention_prompt(q, k, v, cu, cu, y)
    for a, b in ((0, 40), (40, 75)):
        check_rows(y[a:b], q[a:b], k[a:b], v[a:b], default_scale(dim))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bad", [NAN, float("inf"), float("-inf"), "lowest"])
def test_prompt_masked_places_do_not_reach_a_row(bad, dim):
    """Keys and values that only later rows see hold NaN, infinities or the type's lowest value."""
    dtype, counts, heads = torch.bfloat16, [100, 70], 4
    bad = torch.finfo(dtype).min if bad == "lowest" else bad
    q, k, v = randn((170, heads, dim), dtype, 0), randn((170, 1, dim), dtype, 1), randn((170, 1, dim), dtype, 2)
    cut = [60, 100 + 33]  # first bad row of each sequence
    for lo, hi in ((cut[0], 100), (cut[1], 170)):
        k[lo:hi] = bad
        v[lo:hi] = bad
    y = torch.full_like(q, 7.0)
    paro.paro_attention_prompt(q, k, v, offsets(counts), offsets(counts), y)
    for lo, hi in ((0, cut[0]), (100, cut[1])):
        check_rows(y[lo:hi], q[lo:hi], k[lo:hi], v[lo:hi], default_scale(dim))


@pytest.mark.parametrize("bad", [NAN, float("inf"), "lowest"])
def test_prompt_masked_places_many_row_tiles(bad):
    """The same with more than 96 row tiles and key-value heads, packed and over the cache."""
    dtype, n, heads, kv_heads, dim = torch.float16, 420, 32, 8, 64
    bad = torch.finfo(dtype).min if bad == "lowest" else bad
    q, k, v = (randn((n, h, dim), dtype, i) for i, h in enumerate((heads, kv_heads, kv_heads)))
    cut = 201  # first bad row
    k[cut:], v[cut:] = bad, bad
    y = torch.full_like(q, 7.0)
    paro.paro_attention_prompt(q, k, v, offsets([n]), offsets([n]), y)
    z = torch.full_like(q, 7.0)
    c = paro.KVCache.empty(1, 20, kv_heads, 32, dim, 1, 16, dtype)
    c.table[0, :14] = torch.arange(14, 0, -1, dtype=torch.int32)
    c.refs[1:15] = 1
    c.lengths[0] = n
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    paro.paro_kv_append(c, 0, k, v, slots, offsets([n]))
    paro.paro_attention_prompt_cached(c, 0, q, slots, offsets([n]), z)
    for got in (y, z):
        check_rows(got[:cut], q[:cut], k[:cut], v[:cut], default_scale(dim))


def test_prompt_bad_values_reach_the_rows_that_see_them():
    dtype, n, dim = torch.float16, 50, 64
    q, k, v = randn((n, 2, dim), dtype, 0), randn((n, 1, dim), dtype, 1), randn((n, 1, dim), dtype, 2)
    v[20, 0, 5] = float("inf")
    v[30, 0, 9] = NAN
    y = torch.empty_like(q)
    paro.paro_attention_prompt(q, k, v, offsets([n]), offsets([n]), y)
    inf, nan = torch.isinf(y), torch.isnan(y)
    assert not inf[:20].any() and not nan[:30].any()
    assert bool((inf[20:, :, 5] | nan[20:, :, 5]).all()) and bool(nan[30:, :, 9].all())
    inf[20:, :, 5] = nan[20:, :, 5] = nan[30:, :, 9] = False
    assert not inf.any() and not nan.any()


@pytest.mark.parametrize("n,heads,kv_heads", [(300, 4, 1), (300, 64, 16), (800, 16, 8)])
def test_prompt_bad_value_beside_and_before_masked_ones(n, heads, kv_heads):
    """Every tile and wave that a bad value can share with rows that may not see it: one at a time, moved along a tile."""
    dtype, dim = torch.bfloat16, 64
    q, k, clean = (randn((n, h, dim), dtype, i) for i, h in enumerate((heads, kv_heads, kv_heads)))
    cu, good = offsets([n]), torch.empty_like(q)
    paro.paro_attention_prompt(q, k, clean, cu, cu, good)
    for at in (0, 63, 64, 100, 127, 128, 131, 190, 298, 299):
        v = clean.clone()
        v[at, :, 7] = NAN
        y = torch.full_like(q, 5.0)
        paro.paro_attention_prompt(q, k, v, cu, cu, y)
        assert bool(torch.isnan(y[at:, :, 7]).all())
        y[at:, :, 7] = good[at:, :, 7]
        # rows computed again sum in another order: both within the bound, so at most two of them apart
        assert not torch.isnan(y).any()
        check_rows(y[max(0, at - 40):at + 2], q[max(0, at - 40):at + 2], k[:at + 2], clean[:at + 2], default_scale(dim))
        same = torch.cat([y[:max(0, at - 130)], y[at + 130:]])
        assert torch.equal(same, torch.cat([good[:max(0, at - 130)], good[at + 130:]]))


def test_prompt_rows_outside_the_sequences_stay():
    q, k, v = randn((60, 4, 64), torch.float16, 0), randn((60, 2, 64), torch.float16, 1), randn((60, 2, 64),
                                                                                               torch.float16, 2)
    y = torch.full_like(q, 3.0)
    cu = torch.tensor([10, 25, 25, 40], dtype=torch.int64, device="cuda")
    paro.paro_attention_prompt(q, k, v, cu, cu, y)
    assert bool((y[:10] == 3).all()) and bool((y[40:] == 3).all())
    for a, b in ((10, 25), (25, 40)):
        check_rows(y[a:b], q[a:b], k[a:b], v[a:b], default_scale(64))


@pytest.mark.parametrize("cu", [[-5, 30, 20, 400], [0, 200, 100], [50, 0], [-9, -3], [10 ** 12, 10 ** 13]])
def test_prompt_malformed_offsets_stay_in_bounds(cu):
    """Wrong numbers are allowed; what is not covered by a sequence is not written, and nothing else is touched."""
    big = torch.full((3, 120, 4, 64), 3.0, dtype=torch.float16, device="cuda")
    q, k, v = randn((120, 4, 64), torch.float16, 0), randn((120, 2, 64), torch.float16, 1), randn((120, 2, 64),
                                                                                                 torch.float16, 2)
    cu = torch.tensor(cu, dtype=torch.int64, device="cuda")
    paro.paro_attention_prompt(q, k, v, cu, cu, big[1])
    torch.cuda.synchronize()
    assert bool((big[0] == 3).all()) and bool((big[2] == 3).all())


def test_prompt_no_rows_and_no_sequences():
    q = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    k = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    paro.paro_attention_prompt(q, k, k, offsets([0]), offsets([0]), q)
    y = torch.full((5, 4, 64), 2.0, dtype=torch.float16, device="cuda")
    paro.paro_attention_prompt(torch.zeros_like(y), k, k, offsets([]), offsets([]), y)
    assert bool((y == 2).all())
    # rows but no key at all
    paro.paro_attention_prompt(torch.zeros_like(y), k, k, offsets([5]), offsets([0]), y)
    assert bool((y == 0).all())


@pytest.mark.parametrize("n", [255, 256, 257, 1030])
def test_prompt_many_sequences(n):
    """More sequences than one step of the sequence scan: short, empty and longer ones."""
    counts = [(i * 7) % 4 for i in range(n)]
    counts[n // 2] = counts[-1] = 140
    for cached in (False, True):
        heads, kv_heads, dim, dtype = 6, 2, 64, torch.float16
        rows = sum(counts)
        q = randn((rows, heads, dim), dtype, n, 1.5)
        y = torch.full_like(q, NAN)
        if cached:
            c = filled_cache(paro, counts, 16, kv_heads, dim, dtype, n)
            paro.paro_attention_prompt_cached(c, 0, q, torch.arange(n, dtype=torch.int32, device="cuda"),
                                              offsets(counts), y)
            k, v = (torch.cat([x[i] for x in (cached_rows(c, 0, s) for s in range(n) if counts[s])]) for i in (0, 1))
        else:
            k, v = randn((rows, kv_heads, dim), dtype, 1), randn((rows, kv_heads, dim), dtype, 2)
            paro.paro_attention_prompt(q, k, v, offsets(counts), offsets(counts), y)
        at = 0
        for i, m in enumerate(counts):
            if m and (i < 8 or m > 3 or i % 37 == 0 or i > n - 5):
                check_rows(y[at:at + m], q[at:at + m], k[at:at + m], v[at:at + m], default_scale(dim))
            at += m
        assert not torch.isnan(y).any()


def test_prompt_repeats_to_the_bit_and_on_another_stream():
    q, k, v = randn((333, 8, 128), torch.bfloat16, 0), randn((333, 2, 128), torch.bfloat16, 1), randn(
        (333, 2, 128), torch.bfloat16, 2)
    cu = offsets([200, 133])
    first = torch.empty_like(q)
    paro.paro_attention_prompt(q, k, v, cu, cu, first)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(3):
        y = torch.full_like(q, NAN)
        torch.cuda.synchronize()
        paro.paro_attention_prompt(q, k, v, cu, cu, y, stream=other)
        torch.cuda.synchronize()
        assert torch.equal(y, first)


def faint_case(dtype, n, dim, gap):
    """One key far above all others (gap: in powers of two), with a value of 0 where the others have 1: y is the sum of
    the n - 1 small weights.  Scores are exact: q = (1, 0, ...), k = (score, 0, ...), scale = log(2)."""
    q, k, v = (torch.zeros((r, 1, dim), dtype=dtype, device="cuda") for r in (1, n, n))
    q[:, :, 0], k[n // 3, :, 0] = 1.0, float(gap)
    v.fill_(1.0)
    v[n // 3] = 0.0
    small = (n - 1) * 2.0 ** -gap
    return q, k, v, small / (1.0 + small)


def check_faint(y, want, dtype):
    # scores to gap * 2^-22 (log 2 in fp32 and two products); weights and y by half a
    # step of fp16 each, the sums by fp32 steps; an fp16 y below 2^-14 by half a subnormal step
    err = (y.double() - want).abs().max()
    assert float(err) <= want * (2 * 2.0 ** -11 + 64 * 2.0 ** -22) + 2.0 ** -25


@pytest.mark.parametrize("n,heads", [(3000, 1), (3000, 64)])
def test_prompt_small_weights_in_fp16(n, heads):
    q, k, v, want = faint_case(torch.float16, n, 64, 20.5)
    q = q.expand(130, heads, 64).contiguous()
    k, v = k.expand(n, heads, 64).contiguous(), v.expand(n, heads, 64).contiguous()
    y = torch.empty_like(q)
    paro.paro_attention_prompt(q, k, v, offsets([130]), offsets([n]), y, scale=0.6931471805599453, causal=False)
    check_faint(y, want, torch.float16)


# ---- over the cache ----

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_chunk_pages(page, dtype):
    lengths, new = [1, 40, 0, 130, 300, 64, 517], [1, 7, 0, 130, 65, 64, 100]
    heads, kv_heads, dim = (7, 1, 64) if page % 3 else (8, 2, 128)
    c = filled_cache(paro, lengths, page, kv_heads, dim, dtype, page)
    order = [3, 0, 6, 2, 5, 1, 4]
    counts = [new[s] for s in order]
    q = randn((sum(counts), heads, dim), dtype, 1, 1.5)
    y = torch.full_like(q, NAN)
    slots = torch.tensor(order, dtype=torch.int32, device="cuda")
    paro.paro_attention_prompt_cached(c, 0, q, slots, offsets(counts), y)
    at = 0
    for s, n in zip(order, counts):
        k, v = cached_rows(c, 0, s)
        check_rows(y[at:at + n], q[at:at + n], k, v, default_scale(dim))
        at += n


def test_chunk_layers_empty_and_foreign_slots():
    c = filled_cache(paro, [20, 90, 0], 16, 2, 128, torch.float16, 1, layers=3)
    q = randn((3 + 90 + 4 + 2, 4, 128), torch.float16, 0)
    y = torch.full_like(q, NAN)
    slots = torch.tensor([0, 1, 2, 99], dtype=torch.int32, device="cuda")
    paro.paro_attention_prompt_cached(c, 2, q, slots, offsets([3, 90, 4, 2]), y)
    for s, (a, b) in ((0, (0, 3)), (1, (3, 93))):
        k, v = cached_rows(c, 2, s)
        check_rows(y[a:b], q[a:b], k, v, default_scale(128))
    assert bool((y[93:] == 0).all())  # no keys


@pytest.mark.parametrize("dim,page,dtype", [(64, 16, torch.bfloat16), (128, 64, torch.float16), (128, 16, torch.bfloat16)])
@pytest.mark.parametrize("lengths,new,heads,kv_heads", [([300, 90, 0, 1217, 64, 1], [200, 90, 3, 64, 30, 1], 56, 8),
                                                        ([290, 400, 5], [280, 270, 9], 64, 16)])
def test_chunk_many_row_tiles(lengths, new, heads, kv_heads, dim, page, dtype):
    """About one workgroup of 128 rows per CU (eight waves, keys in two halves), and more (four waves)."""
    c = filled_cache(paro, lengths, page, kv_heads, dim, dtype, 4)
    q = randn((sum(new), heads, dim), dtype, 5, 1.5)
    y = torch.full_like(q, NAN)
    slots = torch.arange(len(new), dtype=torch.int32, device="cuda")
    paro.paro_attention_prompt_cached(c, 0, q, slots, offsets(new), y)
    at = 0
    for s, n in enumerate(new):
        k, v = cached_rows(c, 0, s)
        check_rows(y[at:at + n], q[at:at + n], k, v, default_scale(dim))
        at += n


def run_split_chunk(lengths, new, heads, kv_heads, dim, page, dtype, causal=True, layers=1, layer=0):
    c = filled_cache(paro, lengths, page, kv_heads, dim, dtype, len(new), layers=layers)
    q = randn((sum(new), heads, dim), dtype, 5, 1.5)
    slots, cu = torch.arange(len(new), dtype=torch.int32, device="cuda"), offsets(new)
    need = paro.paro_attention_prompt_cached_workspace_bytes(c, len(new), sum(new), heads)
    assert need > 0
    ws = paro.make_workspace(need)
    first = None
    for _ in range(3):  # the workspace serves again, and the bits repeat
        y = torch.full_like(q, NAN)
        paro.paro_attention_prompt_cached(c, layer, q, slots, cu, y, causal=causal, workspace=ws)
        torch.cuda.synchronize()
        first = y if first is None else first
        assert torch.equal(y, first)
    assert not ws[:2 ** 21].any()  # the counter area
    at = 0
    for s, n in enumerate(new):
        k, v = cached_rows(c, layer, s)
        check_rows(y[at:at + n], q[at:at + n], k, v, default_scale(dim), causal)
        at += n


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,heads", [(64, (7, 1)), (128, (8, 2)), (128, (4, 4))])
def test_chunk_keys_split_over_workgroups(dim, heads, dtype):
    run_split_chunk([5000], [6], *heads, dim, 64, dtype)
    run_split_chunk([2300, 1, 0, 513, 40, 1024], [33, 1, 0, 5, 70, 2], *heads, dim, 16, dtype, layers=2, layer=1)
    run_split_chunk([1500, 3], [17, 40], *heads, dim, 32, dtype, causal=False)


def test_chunk_split_with_masked_and_visible_bad_values():
    dtype, dim, n, m = torch.float16, 64, 3000, 40
    c = filled_cache(paro, [n], 16, 1, dim, dtype, 1)
    q, slots, cu = randn((m, 4, dim), dtype, 2), torch.zeros(1, dtype=torch.int32, device="cuda"), offsets([m])
    ws = paro.make_workspace(paro.paro_attention_prompt_cached_workspace_bytes(c, 1, m, 4))
    k, v = (x.clone() for x in cached_rows(c, 0, 0))
    for at in (n - 1, n - 20):  # seen by the last rows alone
        page, row = int(c.table[0, at // 16]), at % 16
        c.v[0, page, :, row] = NAN
        y = torch.full_like(q, 3.0)
        paro.paro_attention_prompt_cached(c, 0, q, slots, cu, y, workspace=ws)
        clean = m - (n - at)
        check_rows(y[:clean], q[:clean], k[:n - m + clean], v[:n - m + clean], default_scale(dim))
        assert bool(torch.isnan(y[clean:]).all())
    c.v[0, int(c.table[0, 40]), :, 3, 9] = NAN
    paro.paro_attention_prompt_cached(c, 0, q, slots, cu, y, workspace=ws)
    assert bool(torch.isnan(y[:, :, 9]).all()) and not torch.isnan(y[:clean, :, :9]).any()


def run_decode(lengths, heads, kv_heads, dim, page, dtype, seed=0, order=None, extra=2, layers=1, layer=0):
    c = filled_cache(paro, lengths, page, kv_heads, dim, dtype, seed, extra=extra, layers=layers)
    order = list(range(len(lengths))) if order is None else order
    q = randn((len(order), heads, dim), dtype, seed + 9, 1.5)
    y = torch.full_like(q, NAN)
    slots = torch.tensor(order, dtype=torch.int32, device="cuda")
    ws = paro.make_workspace(paro.paro_attention_decode_workspace_bytes(c, len(order), heads))
    first = None
    for _ in range(3):  # the workspace serves again, and the bits repeat
        paro.paro_attention_decode(c, layer, q, slots, y, ws)
        torch.cuda.synchronize()
        first = y.clone() if first is None else first
        assert torch.equal(y, first)
    for r, s in enumerate(order):
        k, v = cached_rows(c, layer, s)
        check_rows(y[r:r + 1], q[r:r + 1], k, v, default_scale(dim))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", HEADS + [(16, 1), (17, 1), (48, 2)])
def test_decode_heads(heads, dim, dtype):
    run_decode([1, 33, 0, 200], *heads, dim, 16, dtype)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_pages_and_lengths(page):
    run_decode([1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 0, 127, 128, 129, 255, 256, 257, 500], 4, 1, 128, page,
               torch.bfloat16, page)
    run_decode([3000, 1], 8, 2, 64, page, torch.float16, page, order=[1, 0, 0, 1])


@pytest.mark.parametrize("extra", [2, 700])
def test_decode_long_and_spare_table(extra):
    """Few rows: the length is split over workgroups; a table far longer than the sequences splits more."""
    run_decode([5000], 4, 1, 128, 64, torch.float16, 1, extra=extra)
    run_decode([9001, 17, 4096], 2, 2, 64, 16, torch.bfloat16, 2, extra=extra, layers=2, layer=1)


def test_decode_workspace_serves_several_shapes():
    dtype, dim = torch.float16, 128
    caches = [filled_cache(paro, ln, 16, 2, dim, dtype, i, extra=300) for i, ln in
              enumerate(([2000], [700, 3, 900], [40] * 60))]
    need = max(paro.paro_attention_decode_workspace_bytes(c, c.table.shape[0], 8) for c in caches)
    ws = paro.make_workspace(need)
    for _ in range(2):
        for i, c in enumerate(caches):
            n = c.table.shape[0]
            q, y = randn((n, 8, dim), dtype, i), torch.full((n, 8, dim), NAN, dtype=dtype, device="cuda")
            paro.paro_attention_decode(c, 0, q, torch.arange(n, dtype=torch.int32, device="cuda"), y, ws)
            for r in range(n):
                k, v = cached_rows(c, 0, r)
                check_rows(y[r:r + 1], q[r:r + 1], k, v, default_scale(dim))


@pytest.mark.parametrize("n", [500, 50000])
def test_decode_small_weights_in_fp16(n):
    q, k, v, want = faint_case(torch.float16, n, 128, 27.5)
    pages = -(-n // 16)
    c = paro.KVCache.empty(1, pages, 1, 16, 128, 1, pages, torch.float16)
    c.table[0] = torch.arange(pages, dtype=torch.int32)
    c.refs.fill_(1)
    c.lengths[0] = n
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    paro.paro_kv_append(c, 0, k, v, slots, offsets([n]))
    y = torch.empty_like(q)
    paro.paro_attention_decode(c, 0, q, slots, y, paro.make_workspace(
        paro.paro_attention_decode_workspace_bytes(c, 1, 1)), scale=0.6931471805599453)
    check_faint(y, want, torch.float16)


def test_decode_empty_foreign_and_clamped():
    c = filled_cache(paro, [20, 0], 16, 1, 64, torch.float16, 1, extra=0)
    q = randn((4, 2, 64), torch.float16, 0)
    y = torch.full_like(q, NAN)
    ws = paro.make_workspace(paro.paro_attention_decode_workspace_bytes(c, 4, 2))
    slots = torch.tensor([1, -1, 2, 0], dtype=torch.int32, device="cuda")
    paro.paro_attention_decode(c, 0, q, slots, y, ws)
    assert bool((y[:3] == 0).all())
    k, v = cached_rows(c, 0, 0)
    check_rows(y[3:], q[3:], k, v, default_scale(64))
    # lengths and pages out of range: wrong numbers, no fault, and y alone is written
    c.lengths.copy_(torch.tensor([10 ** 9, -4]))
    c.table[0, 1] = 10 ** 9
    before = c.k.clone()
    paro.paro_attention_decode(c, 0, q, slots, y, ws)
    torch.cuda.synchronize()
    assert bool((y[:3] == 0).all()) and torch.equal(c.k.view(torch.int16), before.view(torch.int16))


def test_decode_and_chunk_strides():
    dtype, dim, lengths = torch.bfloat16, 128, [50, 300]
    c = filled_cache(paro, lengths, 32, 2, dim, dtype, 3)
    rows = randn((2, 8, dim), dtype, 4)
    q = rows[:, 2:6]
    y = torch.full((4, 2, dim), NAN, dtype=dtype, device="cuda").transpose(0, 1)
    ws = paro.make_workspace(paro.paro_attention_decode_workspace_bytes(c, 2, 4))
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    paro.paro_attention_decode(c, 0, q, slots, y, ws, scale=0.2)
    z = torch.full((2, 4, dim + 16), NAN, dtype=dtype, device="cuda")[..., 8:dim + 8]
    paro.paro_attention_prompt_cached(c, 0, q, slots, offsets([1, 1]), z, scale=0.2)
    for r, s in enumerate((1, 0)):
        k, v = cached_rows(c, 0, s)
        check_rows(y[r:r + 1], q[r:r + 1], k, v, 0.2)
        check_rows(z[r:r + 1], q[r:r + 1], k, v, 0.2)


def test_binding_refuses():
    f = torch.float16
    q, k = torch.zeros((4, 4, 64), dtype=f, device="cuda"), torch.zeros((4, 2, 64), dtype=f, device="cuda")
    cu, y = offsets([4]), torch.zeros((4, 4, 64), dtype=f, device="cuda")
    bad = [
        (q, k, k.bfloat16(), cu, cu, y), (q, k, k[:3], cu, cu, y), (q, k, k, cu.int(), cu, y),
        (q, k, k, cu, cu[:1], y), (q, k, k, cu, cu, q), (q, k, k, cu, cu, y[:3]),
        (q.transpose(1, 2), k, k, cu, cu, y), (q[:, :3], k, k, cu, cu, y[:, :3]), (q, k.cpu(), k, cu, cu, y),
        (q[..., :32], k[..., :32], k[..., :32], cu, cu, y[..., :32]), (q, k, k, cu, cu, y[:1].expand(4, 4, 64)),
    ]
    for args in bad:
        with pytest.raises(paro.ParoError):
            paro.paro_attention_prompt(*args)
    with pytest.raises(paro.ParoError):
        paro.paro_attention_prompt(q, k, k, cu, cu, y, scale=float("inf"))
    c = paro.KVCache.empty(1, 4, 2, 16, 64, 2, 2, f)
    s = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = paro.make_workspace(paro.paro_attention_decode_workspace_bytes(c, 4, 4))
    for args in [(c, 1, q, s, y, ws), (c, 0, q, s[:3], y, ws), (c, 0, q, s, y, ws[:64]), (c, 0, q, s, y, None),
                 (c, 0, q[:, :3], s, y[:, :3], ws), (c, 0, q.bfloat16(), s, y, ws), (c, 0, q, s.long(), y, ws)]:
        with pytest.raises(paro.ParoError):
            paro.paro_attention_decode(*args)
    c = paro.KVCache.empty(1, 200, 2, 16, 64, 2, 100, f)
    need = paro.paro_attention_prompt_cached_workspace_bytes(c, 1, 4, 4)
    ws = paro.make_workspace(need)
    paro.paro_attention_prompt_cached(c, 0, q, s[:1], cu, y, workspace=ws)
    for bad in (ws[:need - 16], ws.cpu(), ws[::2]):
        with pytest.raises(paro.ParoError):
            paro.paro_attention_prompt_cached(c, 0, q, s[:1], cu, y, workspace=bad)


@pytest.mark.parametrize("heads", [(256, 1), (256, 256), (255, 85)])
def test_most_heads(heads):
    run_prompt([5, 40], [5, 40], *heads, 64, torch.float16, seed=31)
    run_decode([70, 3], *heads, 64, 16, torch.bfloat16, seed=32)
    lengths, new = [90, 20], [3, 20]
    c = filled_cache(paro, lengths, 16, heads[1], 64, torch.float16, 33)
    q = randn((sum(new), heads[0], 64), torch.float16, 34)
    y = torch.full_like(q, NAN)
    paro.paro_attention_prompt_cached(c, 0, q, torch.arange(2, dtype=torch.int32, device="cuda"), offsets(new), y)
    for s, (a, b) in enumerate(((0, 3), (3, 23))):
        check_rows(y[a:b], q[a:b], *cached_rows(c, 0, s), default_scale(64))


def test_most_sequences_and_rows():
    """16384 sequences (one key each: a row's output is its value) and 32768 decode rows over three slots."""
    n, dt = 16384, torch.bfloat16
    q, k, v = randn((n, 2, 64), dt, 1), randn((n, 1, 64), dt, 2), randn((n, 1, 64), dt, 3)
    y = torch.full_like(q, NAN)
    cu = torch.arange(n + 1, dtype=torch.int64, device="cuda")
    paro.paro_attention_prompt(q, k, v, cu, cu, y)
    assert torch.equal(y, v.expand(n, 2, 64))
    with pytest.raises(paro.ParoError):
        more = torch.arange(n + 2, dtype=torch.int64, device="cuda").clamp(max=n)
        paro.paro_attention_prompt(q, k, v, more, more, y)
    rows = 2 * n
    c = filled_cache(paro, [33, 1, 100], 16, 1, 64, dt, 4)
    q = randn((rows, 2, 64), dt, 5)
    y = torch.full_like(q, NAN)
    slots = torch.arange(rows, dtype=torch.int32, device="cuda") % 3
    ws = paro.make_workspace(paro.paro_attention_decode_workspace_bytes(c, rows, 2))
    paro.paro_attention_decode(c, 0, q, slots, y, ws)
    assert not torch.isnan(y).any()
    for r in (0, 1, 2, 12345, 20000, rows - 2, rows - 1):
        check_rows(y[r:r + 1], q[r:r + 1], *cached_rows(c, 0, r % 3), default_scale(64))
    assert torch.equal(y[1::3], cached_rows(c, 0, 1)[1].expand(y[1::3].shape[0], 2, 64))
    with pytest.raises(paro.ParoError):
        paro.paro_attention_decode(c, 0, q.repeat(2, 1, 1)[:rows + 1], slots.repeat(2)[:rows + 1],
                                   y.repeat(2, 1, 1)[:rows + 1], ws)
