"""Host checks of the attention and cache entry points (no GPU): every refusal
returns its status before anything is launched, with a message."""
import ctypes

import pytest

paro = pytest.importorskip("rotation_int4_weight_amd")
from rotation_int4_weight_amd import _lib  # noqa: E402

NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5, 7
A = 1 << 40  # addresses that are checked, never used
STEP = 1 << 36


def cache(**kw):
    f = dict(layers=2, kv_heads=2, head_dim=128, page_size=16, num_pages=64, slots=4, max_pages=8, dt=0, k=A,
             v=A + STEP, refs=A + 2 * STEP, table=A + 3 * STEP, lengths=A + 4 * STEP)
    f.update(kw)
    return _lib.ParoKvCacheC(*[f[n] for n, _ in _lib.ParoKvCacheC._fields_])


def shape(**kw):
    f = dict(q_heads=8, kv_heads=2, head_dim=128, causal=1, scale=0.1, q_token=1024, q_head=128, k_token=256,
             k_head=128, v_token=256, v_head=128, y_token=1024, y_head=128)
    f.update(kw)
    return _lib.ParoAttentionShapeC(*[f[n] for n, _ in _lib.ParoAttentionShapeC._fields_])


Q, Y, K, V, LIST, CU, WS, OUT = (A + (5 + i) * STEP for i in range(8))
BIG = 1 << 34


def prompt(s=None, q=Q, k=K, v=V, dt=0, cu_q=CU, cu_k=CU, n=1, tq=0, tk=0, y=Y):
    return _lib.load().paro_attention_prompt(ctypes.byref(shape() if s is None else s), q, k, v, dt, cu_q, cu_k, n, tq,
                                             tk, y, None)


def cached(c=None, layer=0, s=None, q=Q, slots=LIST, cu=CU, n=1, tq=0, y=Y, ws=None, nb=0):
    return _lib.load().paro_attention_prompt_cached(ctypes.byref(c or cache()), layer, ctypes.byref(s or shape()), q,
                                                    slots, cu, n, tq, y, ws, nb, None)


def decode(c=None, layer=0, s=None, q=Q, slots=LIST, rows=0, y=Y, ws=WS, nb=BIG):
    return _lib.load().paro_attention_decode(ctypes.byref(c or cache()), layer, ctypes.byref(s or shape()), q, slots,
                                             rows, y, ws, nb, None)


def append(c=None, layer=0, k=K, kt=256, kh=128, v=V, vt=256, vh=128, slots=LIST, cu=CU, granted=None, n=1, tokens=0):
    return _lib.load().paro_kv_append(ctypes.byref(c or cache()), layer, k, kt, kh, v, vt, vh, slots, cu, granted, n,
                                      tokens, None)


def plan(name, c=None, a=LIST, b=CU, n=1, out=OUT, ws=WS, nb=BIG):
    return getattr(_lib.load(), name)(ctypes.byref(c or cache()), a, b, n, out, ws, nb, None)


def free(c=None, a=LIST, n=1):
    return _lib.load().paro_kv_free(ctypes.byref(c or cache()), a, n, None)


def compact(c=None, used=OUT, ws=WS, nb=BIG):
    return _lib.load().paro_kv_compact(ctypes.byref(c or cache()), used, ws, nb, None)


def test_nothing_to_do_is_ok():
    assert prompt() == 0 and prompt(tq=5, n=0) == 0 and cached() == 0 and decode() == 0 and append() == 0
    assert plan("paro_kv_reserve", n=0) == 0 and plan("paro_kv_fork", n=0) == 0 and free(n=0) == 0


SHAPES = [
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED), (dict(q_heads=7), SHAPE),
    (dict(q_heads=0), SHAPE), (dict(kv_heads=0), SHAPE), (dict(q_heads=512), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(q_token=4), SHAPE), (dict(q_head=-8), SHAPE), (dict(y_token=1 << 40), SHAPE), (dict(y_token=0), SHAPE),
    (dict(y_head=64), SHAPE), (dict(y_token=896), SHAPE),
]


@pytest.mark.parametrize("bad,status", SHAPES)
def test_shapes_are_refused(bad, status):
    assert prompt(shape(**bad), tq=9, tk=9) == status
    assert paro.paro_last_error()
    assert decode(s=shape(**bad), rows=9) == status
    assert cached(s=shape(**bad), tq=9) == status


def test_prompt_arguments():
    assert prompt(tq=9, tk=9, dt=2) == DTYPE
    assert prompt(tq=-1) == SHAPE and prompt(tk=-1) == SHAPE and prompt(n=-1) == SHAPE
    assert prompt(tq=(1 << 21) + 1) == UNSUPPORTED and prompt(n=65537) == UNSUPPORTED
    for name in ("q", "y", "k", "v", "cu_q", "cu_k"):
        assert prompt(tq=9, tk=9, **{name: None}) == NULL
    for name in ("q", "y", "k", "v"):
        assert prompt(tq=9, tk=9, **{name: Q + 8}) == ALIGN
    assert prompt(tq=9, tk=9, cu_q=CU + 4) == ALIGN
    for name in ("q", "k", "v", "cu_q"):
        assert prompt(tq=9, tk=9, **{name: Y + 16}) == SHAPE  # y overlaps an input
    assert prompt(shape(k_token=12), tq=9, tk=9) == SHAPE and prompt(shape(v_head=1), tq=9, tk=9) == SHAPE
    assert _lib.load().paro_attention_prompt(None, Q, K, V, 0, CU, CU, 1, 9, 9, Y, None) == NULL


CACHES = [
    (dict(head_dim=32), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=512), UNSUPPORTED), (dict(layers=0), SHAPE), (dict(kv_heads=257), SHAPE), (dict(num_pages=0), SHAPE),
    (dict(num_pages=(1 << 22) + 1), SHAPE), (dict(slots=0), SHAPE), (dict(slots=4097), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(max_pages=1 << 20, page_size=256), 0), (dict(max_pages=(1 << 20) + 1), SHAPE), (dict(dt=2), DTYPE),
    (dict(dt=-2 ** 31), DTYPE), (dict(refs=None), NULL), (dict(table=None), NULL), (dict(lengths=None), NULL),
    (dict(lengths=A + 2 * STEP + 4), SHAPE), (dict(refs=A + 2 * STEP + 2), ALIGN),
]


@pytest.mark.parametrize("bad,status", CACHES)
def test_caches_are_refused(bad, status):
    if bad.get("page_size") == 256:
        bad = dict(bad, max_pages=1 << 23)  # max_pages is checked first, then the positions
        status = SHAPE
    c = cache(**bad)
    assert free(c) == status and append(c) == status and compact(c) == status
    assert decode(c, rows=1) == status and cached(c, tq=1) == status
    assert plan("paro_kv_reserve", c) == status and plan("paro_kv_fork", c) == status
    assert _lib.load().paro_kv_workspace_bytes(ctypes.byref(c)) == 0
    assert _lib.load().paro_attention_decode_workspace_bytes(ctypes.byref(c), 4, 8) == 0


def test_cache_data_and_layers():
    for bad, status in ((dict(k=None), NULL), (dict(v=None), NULL), (dict(k=A + 8), ALIGN), (dict(v=A + 64), SHAPE)):
        c = cache(**bad)
        assert append(c) == status and compact(c) == status and plan("paro_kv_reserve", c) == status
        assert decode(c, rows=1) == status and cached(c, tq=1) == status
    for layer in (-1, 2):
        assert append(layer=layer) == SHAPE and decode(layer=layer) == SHAPE and cached(layer=layer) == SHAPE
    assert decode(s=shape(kv_heads=4), rows=1) == SHAPE and cached(s=shape(head_dim=64), tq=1) == SHAPE


def test_decode_and_cached_arguments():
    assert decode(rows=-1) == SHAPE and decode(rows=65537) == UNSUPPORTED and cached(tq=-1) == SHAPE
    for name in ("q", "y", "slots"):
        assert decode(rows=2, **{name: None}) == NULL and cached(tq=2, **{name: None}) == NULL
    assert cached(tq=2, cu=None) == NULL and cached(tq=2, cu=CU + 4) == ALIGN and decode(rows=2, slots=LIST + 2) == ALIGN
    assert decode(rows=2, ws=None) == WORKSPACE and decode(rows=2, nb=64) == WORKSPACE and decode(rows=2, ws=WS + 8) == ALIGN
    for at in (Y, Q, LIST, A, A + STEP, A + 3 * STEP):
        assert decode(rows=2, ws=at) == SHAPE  # the workspace overlaps something
    for at in (A, A + STEP, A + 3 * STEP, A + 4 * STEP):
        assert decode(rows=2, y=at) == SHAPE and cached(tq=2, y=at) == SHAPE
    assert decode(rows=2, y=LIST) == SHAPE and cached(tq=2, y=CU) == SHAPE


def test_cached_workspace():
    big = cache(max_pages=400, num_pages=800)
    need = lambda c, n, t, h: _lib.load().paro_attention_prompt_cached_workspace_bytes(ctypes.byref(c), n, t, h)  # noqa: E731
    assert need(big, 1, 4, 8) > 2 ** 21 and need(cache(), 1, 4, 8) == 0  # 128 positions: nothing to split
    assert need(big, 1, 5000, 8) == 0 and need(big, 200, 200, 8) == 0  # enough rows without
    assert need(big, 0, 4, 8) == 0 and need(big, 1, 0, 8) == 0 and need(big, 1, 4, 7) == 0
    assert need(big, -1, 4, 8) == 0 and need(big, 1, 1 << 30, 8) == 0 and need(big, 1 << 20, 4, 8) == 0
    few = dict(c=big, n=1, tq=4)
    n = need(big, 1, 4, 8)
    assert cached(**few, ws=WS, nb=n - 1) == WORKSPACE and cached(**few, ws=WS, nb=0) == WORKSPACE
    assert cached(**few, ws=WS + 8, nb=BIG) == ALIGN
    for at in (Q, Y, CU, LIST, A, A + STEP, A + 2 * STEP, A + 3 * STEP, A + 4 * STEP):
        assert cached(**few, ws=at, nb=BIG) == SHAPE


def test_append_arguments():
    assert append(n=-1) == SHAPE and append(tokens=-1) == SHAPE and append(n=65537) == UNSUPPORTED
    assert append(cu=None, n=3, tokens=2) == SHAPE
    for name in ("k", "v", "slots"):
        assert append(tokens=2, **{name: None}) == NULL
    assert append(tokens=2, k=K + 8) == ALIGN and append(tokens=2, cu=CU + 4) == ALIGN and append(tokens=2, kt=3) == SHAPE
    assert append(tokens=2, k=A + 64) == SHAPE and append(tokens=2, v=A + STEP + 64) == SHAPE
    assert append(tokens=1, granted=OUT + 2) == ALIGN


def test_bookkeeping_arguments():
    for name in ("paro_kv_reserve", "paro_kv_fork"):
        assert plan(name, n=-1) == SHAPE and plan(name, n=4097) == SHAPE
        assert plan(name, a=None) == NULL and plan(name, b=None) == NULL and plan(name, out=None) == NULL
        assert plan(name, ws=None) == WORKSPACE and plan(name, nb=8) == WORKSPACE and plan(name, ws=WS + 4) == ALIGN
        assert plan(name, a=LIST + 1) == ALIGN
        assert plan(name, out=LIST) == SHAPE and plan(name, out=CU) == SHAPE  # granted over an input
        for at in (A + 2 * STEP, A + 3 * STEP, A + 4 * STEP, WS):
            assert plan(name, out=at) == SHAPE and plan(name, a=at) == SHAPE
        assert plan(name, ws=A + 3 * STEP) == SHAPE
    assert free(n=-1) == SHAPE and free(n=4097) == SHAPE and free(a=None) == NULL and free(a=A + 2 * STEP) == SHAPE
    assert compact(used=None) == NULL and compact(ws=None) == WORKSPACE and compact(used=A + 4 * STEP) == SHAPE
    assert compact(ws=A) == SHAPE


def test_workspace_sizes():
    lib, c = _lib.load(), cache()
    need = lib.paro_attention_decode_workspace_bytes
    assert need(ctypes.byref(c), 0, 8) == 0 and need(ctypes.byref(c), 4, 7) == 0 and need(None, 4, 8) == 0
    assert need(ctypes.byref(c), 4, 8) > 0
    # behind the counter area that the linears' workspaces start with: 2^14 lines of 128 bytes
    assert need(ctypes.byref(c), 4, 8) >= 2 ** 21 and lib.paro_kv_workspace_bytes(ctypes.byref(c)) > 2 ** 21
    assert lib.paro_kv_workspace_bytes(ctypes.byref(c)) >= 4 * 64 and lib.paro_kv_workspace_bytes(None) == 0


def test_binding_refuses_host_tensors_and_mismatches():
    torch = pytest.importorskip("torch")
    f = torch.float16
    with pytest.raises(paro.ParoError):
        paro.KVCache(torch.zeros(1, 2, 1, 16, 64), torch.zeros(1, 2, 1, 16, 64), *(torch.zeros(1),) * 3)
    c = paro.KVCache.empty(1, 4, 2, 16, 64, 3, 2, f, device="cpu")
    assert c.c.page_size == 16 and c.c.slots == 3 and c.c.max_pages == 2 and c.c.num_pages == 4
    q = torch.zeros(3, 4, 64, dtype=f)
    k = torch.zeros(3, 2, 64, dtype=f)
    s = torch.zeros(3, dtype=torch.int32)
    cu = torch.zeros(4, dtype=torch.int64)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda: paro.paro_attention_prompt(q, k, k, cu, cu, q.clone()),
                 lambda: paro.paro_attention_prompt_cached(c, 0, q, s, cu, q.clone()),
                 lambda: paro.paro_attention_decode(c, 0, q, s, q.clone(), ws),
                 lambda: paro.paro_kv_append(c, 0, k, k, s), lambda: paro.paro_kv_free(c, s),
                 lambda: paro.paro_kv_reserve(c, s, s, s.clone(), ws), lambda: paro.paro_kv_compact(c, s[:1], ws)):
        with pytest.raises(paro.ParoError, match="device memory"):
            call()
    for call in (lambda: paro.paro_kv_append(c, 0, k.float(), k, s), lambda: paro.paro_kv_append(c, 0, k[:, :1], k, s),
                 lambda: paro.paro_kv_append(c, 0, k, k, s, cu[:3]), lambda: paro.paro_kv_free(c, s.long()),
                 lambda: paro.paro_kv_reserve(c, s, s[:2], s, ws), lambda: paro.paro_kv_fork(c, s, s, s[::2], ws),
                 lambda: paro.paro_attention_decode(c, 0, q, s, q[:2], ws)):
        with pytest.raises(paro.ParoError):
            call()


@pytest.mark.parametrize("scale,status", [(2.0 ** 127, 0), (-2.0 ** 127, 0), (0.0, 0), (2.0 ** 127 * 1.001, SHAPE),
                                          (-3e38, SHAPE), (float("inf"), SHAPE), (-float("inf"), SHAPE),
                                          (float("nan"), SHAPE)])
def test_scales_that_overflow_in_base_two_are_refused(scale, status):
    """2^127 log2(e) still fits fp32; no call here has rows, so none is launched."""
    s = shape(scale=scale)
    assert prompt(s) == status and cached(s=s) == status and decode(s=s) == status


def test_lists_inside_the_cache_are_refused():
    """Lists that a call would overwrite, or read while it writes them: over K, V or the tables."""
    inside = (A + 64, A + STEP + 64, A + 2 * STEP, A + 3 * STEP, A + 4 * STEP)
    for at in inside:
        for name in ("paro_kv_reserve", "paro_kv_fork"):
            assert plan(name, a=at) == SHAPE and plan(name, b=at) == SHAPE and plan(name, out=at) == SHAPE
        assert free(a=at) == SHAPE and compact(used=at) == SHAPE
        for name in ("slots", "cu", "granted"):
            assert append(tokens=2, **{name: at}) == SHAPE
        assert append(cu=None, n=2, tokens=2, slots=at) == SHAPE
    # a cache without data serves fork and free; its tables are checked all the same
    bare = cache(k=None, v=None)
    assert plan("paro_kv_fork", bare, a=A + 3 * STEP) == SHAPE and free(bare, a=A + 2 * STEP) == SHAPE
