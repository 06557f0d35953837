"""Calls at the edges of what the attention entry points allow, on every form
of the kernels: views whose rows overlap."""
import pytest

from _attention import check_rows, default_scale, offsets, randn

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")

pytestmark = pytest.mark.gpu

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
