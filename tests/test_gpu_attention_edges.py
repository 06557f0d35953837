"""Calls at the edges of what the attention entry points allow, on every form
of the kernels: views whose rows overlap, strides at their limit, scales of
either sign and of zero, values at the end of fp16 or not finite, two calls at
once, rows of no sequence, the largest sizes."""
import pytest

import _shares as sh
from _attention import check_rows, default_scale, offsets, randn

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]
NAN = float("nan")

# form: (query rows, keys, query heads, key-value heads)
PACKED = {
    "split": (300, 300, 4, 1),   # the waves of 32-row workgroups share the keys
    "four": (300, 300, 64, 16),  # 128 rows, four waves
    "eight": (830, 830, 16, 8),  # 128 rows, eight waves, keys in halves
}
CACHED = {
    "cached split": (30, 700, 4, 1),
    "cached parts": (6, 3000, 8, 2),  # with a workspace: the keys over workgroups first
    "cached four": (700, 900, 64, 16),
    "cached eight": (400, 900, 64, 16),
    "decode": (1, 300, 8, 2),
    "decode parts": (1, 3000, 8, 2),
}
FORMS = {**PACKED, **CACHED}


def attend(form, q, k, v, scale, causal=True):
    """One sequence through the form; the cached ones take k and v into pages first."""
    y = torch.full(q.shape, NAN, dtype=q.dtype, device="cuda")
    n, cu = k.shape[0], offsets([q.shape[0]])
    if form in PACKED:
        paro.paro_attention_prompt(q, k, v, cu, offsets([n]), y, scale=scale, causal=causal)
        return y
    page, kv_heads, dim = 16, k.shape[1], k.shape[2]
    m = -(-n // page)
    c = paro.KVCache.empty(1, m + 2, kv_heads, page, dim, 1, m, q.dtype)
    c.k.fill_(NAN)
    c.v.fill_(NAN)
    c.table[0] = torch.randperm(m + 2, generator=torch.Generator().manual_seed(n))[:m].int().cuda()
    c.lengths[0] = n
    at = torch.arange(n, device="cuda")
    where = c.table[0].long()[at // page]
    c.k[0, where, :, at % page], c.v[0, where, :, at % page] = k, v
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    if form.startswith("decode"):
        ws = paro.make_workspace(paro.paro_attention_decode_workspace_bytes(c, 1, q.shape[1]))
        paro.paro_attention_decode(c, 0, q, slots, y, ws, scale=scale)
        return y
    need = paro.paro_attention_prompt_cached_workspace_bytes(c, 1, q.shape[0], q.shape[1])
    ws = paro.make_workspace(need) if form == "cached parts" else None
    assert ws is None or need > 0
    paro.paro_attention_prompt_cached(c, 0, q, slots, cu, y, scale=scale, causal=causal, workspace=ws)
    return y


# ---- views whose rows overlap ----

@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dim,step", [(64, 8), (128, 8), (128, 64), (64, 0)])
@pytest.mark.parametrize("form", PACKED)
def test_a_bad_value_in_overlapping_value_rows_stays_in_its_channel(form, dim, step, causal):
    """V as windows that move by less than their width (or not at all), NaN in one channel of the last row."""
    n_q, n, heads, kv_heads = PACKED[form]
    dtype = torch.bfloat16
    q, k = randn((n_q, heads, dim), dtype, 1), randn((n, kv_heads, dim), dtype, 2)
    flat = randn(((n - 1) * step + dim,), dtype, 3)
    clean = flat.clone().as_strided((n, kv_heads, dim), (step, 0, 1))
    bad = dim - 5  # of the last row alone (of every row if they are one)
    flat[(n - 1) * step + bad] = NAN
    v = flat.as_strided((n, kv_heads, dim), (step, 0, 1))
    y = attend(form, q, k, v, default_scale(dim), causal)
    first = n_q - 1 if causal and step else 0  # rows that see it
    assert bool(torch.isnan(y[first:, :, bad]).all())
    y[first:, :, bad] = attend(form, q, k, clean, default_scale(dim), causal)[first:, :, bad]
    assert not torch.isnan(y).any()
    part = slice(max(0, n_q - 70), n_q)
    check_rows(y[part], q[part], k, clean, default_scale(dim), causal)


# ---- scales ----

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_negative_scales(form, dim, dtype):
    n_q, n, heads, kv_heads = FORMS[form]
    for pattern in ("blocks", "rising", "falling"):
        lev = sh.levels(n, pattern, n)
        q = sh.queries(n_q, heads, dim, dtype, "cuda")
        for p in range(sh.windows(n, dim)):
            k, v = sh.keys_and_values(lev, kv_heads, dim, p, sign=-1.0, device="cuda")
            sh.check(attend(form, q, k.to(dtype), v.to(dtype), -sh.LOG2), lev, v)


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-44, -1e-44])
@pytest.mark.parametrize("form", FORMS)
def test_a_scale_of_zero_weighs_all_keys_alike(form, scale):
    """Products q . k up to 12 * 2^124, whose scaled scores are 0 (or under 2^-17): all keys weigh the same."""
    n_q, n, heads, kv_heads = FORMS[form]
    dim, dtype = 64, torch.bfloat16
    flat = sh.levels(n, "flat")
    q = sh.queries(n_q, heads, dim, dtype, "cuda")
    for p in range(sh.windows(n, dim)):
        k, v = sh.keys_and_values(flat, kv_heads, dim, p, device="cuda")
        k[:, :, 0] = (sh.levels(n, "blocks", n).float() * 2.0 ** 124).cuda()[:, None]
        sh.check(attend(form, q, k.to(dtype), v.to(dtype), scale), flat, v)


# ---- values at the end of the type ----

@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_largest_fp16_values_do_not_become_infinities(form, dim, sign):
    """All values are the largest finite one, so y is it too; the weights' rounding may not carry it past the type.
    One key a little above all others, so that a weight that is not a power of two leads."""
    n_q, n, heads, kv_heads = FORMS[form]
    big = torch.finfo(torch.float16).max
    v = torch.full((n, kv_heads, dim), sign * big, dtype=torch.float16, device="cuda")
    q = sh.queries(n_q, heads, dim, torch.float16, "cuda")
    # 6 to 9 powers of two above, different for every row and head
    q[:, :, 0] = 1.0 + torch.arange(n_q * heads, device="cuda").view(n_q, heads) % 512 / 1024
    for at in {70, n - 40, n // 2} if n_q < n else {70}:
        k = torch.zeros((n, kv_heads, dim), dtype=torch.float16, device="cuda")
        k[at % n, :, 0] = 6.25
        y = attend(form, q, k, v, sh.LOG2).double()
        # half a step for the weights, half for y
        assert bool(((y * sign <= big) & (y * sign >= big * (1 - 2.0 ** -10))).all()), (at, float((y * sign).max()))


@pytest.mark.parametrize("form", FORMS)
def test_infinite_fp16_values_stay_infinite(form):
    n_q, n, heads, kv_heads = FORMS[form]
    q, k, v = (randn((m, h, 64), torch.float16, i) for i, (m, h) in
               enumerate(((n_q, heads), (n, kv_heads), (n, kv_heads))))
    v[0, :, 3], v[0, :, 9] = float("inf"), -float("inf")
    y = attend(form, q, k, v, 0.01)
    assert bool((y[:, :, 3] == float("inf")).all()) and bool((y[:, :, 9] == -float("inf")).all())
    assert int(torch.isinf(y).sum()) == 2 * n_q * heads and not torch.isnan(y).any()


# ---- strides ----

@pytest.mark.parametrize("dim,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("layout", ["fused", "heads_first", "broadcast"])
@pytest.mark.parametrize("form", PACKED)
def test_strided_keys_and_values(form, layout, dim, dtype):
    n_q, n, heads, kv_heads = PACKED[form]
    if layout == "fused":
        rows = torch.zeros((n, heads + 2 * kv_heads, dim), dtype=dtype, device="cuda")
        q, k, v = rows[:, :heads], rows[:, heads:heads + kv_heads], rows[:, heads + kv_heads:]
    elif layout == "heads_first":
        q, k, v = (torch.zeros((h, n, dim), dtype=dtype, device="cuda").transpose(0, 1)
                   for h in (heads, kv_heads, kv_heads))
    else:  # one head of keys and values seen as all
        q = torch.zeros((n, heads, dim), dtype=dtype, device="cuda")
        k, v = (torch.zeros((n, 1, dim), dtype=dtype, device="cuda") for _ in range(2))
    q[:, :, 0] = 1.0
    for pattern in ("blocks", "rising"):
        lev = sh.levels(n, pattern, n)
        for p in range(sh.windows(n, dim)):
            kk, vv = sh.keys_and_values(lev, k.shape[1], dim, p, device="cuda")
            k.copy_(kk)
            v.copy_(vv)
            y = attend(form, q, k.expand(n, kv_heads, dim), v.expand(n, kv_heads, dim), sh.LOG2)
            sh.check(y, lev, vv.expand(n, kv_heads, dim))


@pytest.mark.parametrize("form", PACKED)
def test_keys_and_values_a_full_stride_apart(form):
    """The longest token stride, 2^24 elements: a tile's last row lies 2 GB behind its first."""
    n_q, n, heads, kv_heads = PACKED[form]
    dim, dtype, token = 64, torch.bfloat16, 1 << 24
    store = torch.empty((n - 1) * token + 2 * kv_heads * dim, dtype=dtype, device="cuda")
    k, v = (store[i * kv_heads * dim:].as_strided((n, kv_heads, dim), (token, dim, 1)) for i in (0, 1))
    lev = sh.levels(n, "blocks", n)
    q = sh.queries(n_q, heads, dim, dtype, "cuda")
    for p in range(sh.windows(n, dim)):
        kk, vv = sh.keys_and_values(lev, kv_heads, dim, p, device="cuda")
        k.copy_(kk)
        v.copy_(vv)
        sh.check(attend(form, q, k, v, sh.LOG2), lev, vv)


# ---- values that are not finite, behind the diagonal ----

@pytest.mark.parametrize("bad", [NAN, float("inf"), "lowest"])
@pytest.mark.parametrize("form", [f for f in FORMS if not f.startswith("decode")])
def test_masked_bad_keys_and_values_do_not_reach_a_row(form, bad):
    """The last third of the query rows has keys and values that are not finite (or the type's lowest): the rows before
    count their own keys as if there were no others."""
    n_q, n, heads, kv_heads = FORMS[form]
    dim, dtype = 64, torch.float16
    bad = torch.finfo(dtype).min if bad == "lowest" else bad
    clean = n_q - max(1, n_q // 3)  # rows that see only good keys
    good = n - n_q + clean
    lev = sh.levels(good, "blocks", n)
    q = sh.queries(n_q, heads, dim, dtype, "cuda")
    for p in range(sh.windows(good, dim)):
        k, v = (torch.full((n, kv_heads, dim), bad, dtype=dtype, device="cuda") for _ in range(2))
        kk, vv = sh.keys_and_values(lev, kv_heads, dim, p, device="cuda")
        k[:good], v[:good] = kk.to(dtype), vv.to(dtype)
        sh.check(attend(form, q, k, v, sh.LOG2)[:clean], lev, vv)


# ---- two at once ----

def test_chunks_in_parts_on_two_streams():
    """Two calls over one cache at the same time, each with a workspace of its own; the bits are those of single calls."""
    dim, heads, kv_heads, page, lengths = 128, 8, 2, 16, [3000, 4500]
    m = [-(-n // page) for n in lengths]
    c = paro.KVCache.empty(1, sum(m), kv_heads, page, dim, 2, max(m), torch.bfloat16)
    c.k.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    c.v.normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    c.table[0, :m[0]] = torch.arange(m[0], device="cuda").int()
    c.table[1, :m[1]] = torch.arange(m[0], sum(m), device="cuda").int()
    c.lengths.copy_(torch.tensor(lengths))
    calls = []
    for i, rows in enumerate((6, 9)):
        need = paro.paro_attention_prompt_cached_workspace_bytes(c, 1, rows, heads)
        assert need > 0
        q = randn((rows, heads, dim), c.dtype, i)
        calls.append((torch.cuda.Stream(), q, torch.tensor([i], dtype=torch.int32, device="cuda"), offsets([rows]),
                      torch.empty_like(q), paro.make_workspace(need)))
    want = []
    for _, q, s, cu, y, ws in calls:
        paro.paro_attention_prompt_cached(c, 0, q, s, cu, y, workspace=ws)
        torch.cuda.synchronize()
        want.append(y.clone())
    for _ in range(10):
        for call in calls:
            call[4].fill_(NAN)
        torch.cuda.synchronize()
        for st, q, s, cu, y, ws in calls:
            for _ in range(4):
                paro.paro_attention_prompt_cached(c, 0, q, s, cu, y, stream=st, workspace=ws)
        torch.cuda.synchronize()
        for call, w in zip(calls, want):
            assert torch.equal(call[4], w)


# ---- rows of no sequence ----

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("form", [f for f in CACHED if not f.startswith("decode")])
def test_rows_before_between_and_behind_the_sequences_stay(form, dtype):
    """Over the cache; the offsets leave out the first five rows and the last nine, and one sequence is empty."""
    n_q, n, heads, kv_heads = CACHED[form]
    dim, page, first, behind = 64, 32, 5, 9
    m = -(-n // page)
    c = paro.KVCache.empty(1, m, kv_heads, page, dim, 2, m, dtype)
    lev = sh.levels(n, "blocks", n)
    k, v = sh.keys_and_values(lev, kv_heads, dim, 0, device="cuda")
    at = torch.arange(n, device="cuda")
    c.table[1] = torch.arange(m - 1, -1, -1, device="cuda").int()
    c.lengths[1] = n
    where = c.table[1].long()[at // page]
    c.k[0, where, :, at % page], c.v[0, where, :, at % page] = k.to(dtype), v.to(dtype)
    rows = first + n_q + behind
    q = sh.queries(rows, heads, dim, dtype, "cuda")
    y = torch.full_like(q, 3.0)
    cu = torch.tensor([first, first, first + n_q], device="cuda")
    slots = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    need = paro.paro_attention_prompt_cached_workspace_bytes(c, 2, rows, heads)
    ws = paro.make_workspace(need) if form == "cached parts" else None
    assert ws is None or need > 0
    paro.paro_attention_prompt_cached(c, 0, q, slots, cu, y, scale=sh.LOG2, workspace=ws)
    assert bool((y[:first] == 3).all()) and bool((y[first + n_q:] == 3).all())
    sh.check(y[first:first + n_q], lev, v)


# ---- the largest sizes ----

@pytest.mark.parametrize("dtype", TYPES)
def test_most_packed_rows(dtype):
    """2^21 query rows in 16384 sequences, 64 heads: q and y have 2^33 elements."""
    count, n, heads, dim = 16384, 128, 64, 64
    lev = sh.levels(n, "blocks", 1)
    k, v = (x.to(dtype).repeat(count, 1, 1) for x in sh.keys_and_values(lev, 1, dim, 0, device="cuda"))
    v[-n:] *= 0.5  # the last sequence has values of its own
    q = sh.queries(count * n, heads, dim, dtype, "cuda")
    y = torch.full_like(q, NAN)
    cu = torch.arange(count + 1, device="cuda") * n
    paro.paro_attention_prompt(q, k, v, cu, cu, y, scale=sh.LOG2)
    for s in (0, 1, 8191, 8192, count - 2, count - 1):
        sh.check(y[s * n:(s + 1) * n], lev, v[s * n:(s + 1) * n].float())
    same = y[:-n].view(count - 1, n * heads * dim)
    for part in same.split(1024):
        assert torch.equal(part, same[:1].expand(part.shape[0], -1))


@pytest.mark.parametrize("dtype", TYPES)
def test_longest_slot(dtype):
    """2^20 pages of 256 positions (the same four pages again and again), all keys alike: y is the mean of the values,
    with 2^28 keys and with 77 fewer."""
    pages, page, dim, heads, kv_heads = 1 << 20, 256, 64, 8, 2
    c = paro.KVCache.empty(1, 4, kv_heads, page, dim, 1, pages, dtype)
    c.v.copy_(torch.tensor([1.0, 2.0, 4.0, -3.0]).view(1, 4, 1, 1, 1).expand_as(c.v))
    c.table[0] = (torch.arange(pages, device="cuda") % 4).int()
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    dec = paro.make_workspace(paro.paro_attention_decode_workspace_bytes(c, 1, heads))
    chunk = paro.make_workspace(paro.paro_attention_prompt_cached_workspace_bytes(c, 1, 3, heads))
    for n in (pages * page, pages * page - 77):
        c.lengths[0] = n
        want = 1.0  # (1 + 2 + 4 - 3) / 4; 77 values of -3 fewer change it by under 2^-19
        for rows in (1, 3):
            q = randn((rows, heads, dim), dtype, rows)
            y = torch.full_like(q, NAN)
            if rows == 1:
                paro.paro_attention_decode(c, 0, q, slots, y, dec)
            else:
                paro.paro_attention_prompt_cached(c, 0, q, slots, offsets([rows]), y, workspace=chunk)
            # sums of up to 2^20 whole numbers a part, exact, then 2^8 parts; half a step of the type for y
            off = (y.double() - want).abs()
            assert float(off.max()) <= sh.HALF_STEP[dtype] + 2.0 ** -12, float(off.max())
