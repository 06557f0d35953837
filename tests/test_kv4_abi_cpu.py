"""Host checks of the four-bit cache and of paro_kv_read (no GPU): every refusal returns its status before anything is
launched; the format's helper agrees with itself; the binding's checks."""
import ctypes

import pytest

from test_attention_abi_cpu import (A, ALIGN, BIG, CU, DTYPE, K, LIST, NULL, OUT, SHAPE, STEP, UNSUPPORTED, V, append, cache,
                                    cached, compact, decode, free, plan, shape)

paro = pytest.importorskip("rotation_int4_weight_amd")
torch = pytest.importorskip("torch")
import _kv4  # noqa: E402
from rotation_int4_weight_amd import _lib  # noqa: E402

KV4 = (paro.KV4_F16, paro.KV4_BF16)


def read(c=None, layer=0, k=K, kt=256, kh=128, v=V, vt=256, vh=128, out=0, slots=LIST, cu=CU, first=None, n=1, tokens=0):
    return _lib.load().paro_kv_read(ctypes.byref(c or cache()), layer, k, kt, kh, v, vt, vh, out, slots, cu, first, n,
                                    tokens, None)


@pytest.mark.parametrize("dt", KV4)
def test_the_calls_take_it(dt):
    c = cache(dt=dt)
    assert append(c) == 0 and decode(c) == 0 and free(c, n=0) == 0 and read(c, out=dt - 16) == 0 and read(c, out=2) == 0
    assert plan("paro_kv_reserve", c, n=0) == 0 and plan("paro_kv_fork", c, n=0) == 0
    lib = _lib.load()
    assert lib.paro_kv_workspace_bytes(ctypes.byref(c)) == lib.paro_kv_workspace_bytes(ctypes.byref(cache()))
    need = lib.paro_attention_decode_workspace_bytes
    assert need(ctypes.byref(c), 4, 8) > 2 ** 21 and need(ctypes.byref(c), 4, 7) == 0 and need(ctypes.byref(c), 0, 8) == 0
    assert need(ctypes.byref(c), 32768, 8) == need(ctypes.byref(c), 1, 8) and need(ctypes.byref(c), 32769, 8) == 0


@pytest.mark.parametrize("dt", KV4)
def test_refusals(dt):
    c = cache(dt=dt)
    assert cached(c, tq=2) == UNSUPPORTED and cached(c) == UNSUPPORTED and "paro_kv_read" in paro.paro_last_error()
    assert _lib.load().paro_attention_prompt_cached_workspace_bytes(
        ctypes.byref(cache(dt=dt, max_pages=400, num_pages=800)), 1, 4, 8) == 0
    for bad, status in ((dict(head_dim=96), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(k=None), NULL),
                        (dict(k=A + 8), ALIGN), (dict(refs=None), NULL)):
        b = cache(dt=dt, **bad)
        assert append(b) == status and compact(b) == status and decode(b, rows=1) == status and read(b) == status
    # the pool's bytes: 9/16 of one for each value, where the 16-bit cache has 2
    pool = 2 * 64 * 2 * 16 * 128 * 9 // 16
    assert append(cache(dt=dt, v=A + pool)) == 0 and append(cache(dt=dt, v=A + pool - 16)) == SHAPE
    assert decode(cache(dt=dt, v=A + pool), rows=1, y=A + pool - 16) == SHAPE
    for wrong in (3, 15, 18, 32):
        assert append(cache(dt=wrong)) == DTYPE and read(cache(dt=wrong)) == DTYPE
    # the rows' type is not one of its own
    assert _lib.load().paro_attention_prompt(ctypes.byref(shape()), K, K, V, dt, CU, CU, 1, 3, 3, OUT, None) == DTYPE


@pytest.mark.parametrize("dt", (0, 1) + KV4)
def test_read_arguments(dt):
    c, out = cache(dt=dt), dt & 15
    assert read(c, out=out) == 0 and read(c, out=out, tokens=2, k=None, v=None) == 0 and read(c, out=out, n=0, tokens=2) == 0
    go = lambda **kw: read(c, **{"out": out, "tokens": 2, **kw})  # noqa: E731
    assert go(out=1 - out) == DTYPE and go(out=16) == DTYPE and go(out=3) == DTYPE
    assert go(layer=2) == SHAPE and go(layer=-1) == SHAPE and go(n=-1) == SHAPE and go(tokens=-1) == SHAPE
    assert go(n=16385) == UNSUPPORTED and go(tokens=(1 << 21) + 1) == UNSUPPORTED and go(cu=None, n=3) == SHAPE
    assert go(slots=None) == NULL and go(k=K + 8) == ALIGN and go(v=V + 8) == ALIGN
    assert go(slots=LIST + 2) == ALIGN and go(cu=CU + 4) == ALIGN and go(first=OUT + 2) == ALIGN
    assert go(kt=12) == SHAPE and go(vh=-8) == SHAPE
    assert go(kt=128) == SHAPE and go(vh=64) == SHAPE and go(kt=0) == SHAPE  # rows or heads overlap
    for at in (A, A + STEP, A + 2 * STEP, A + 3 * STEP, A + 4 * STEP):
        assert go(k=at) == SHAPE and go(v=at) == SHAPE  # over the cache
    for at in (LIST, CU):
        assert go(k=at) == SHAPE and go(v=at) == SHAPE
    assert go(first=K) == SHAPE and go(first=V) == SHAPE
    size = 4 if out == 2 else 2
    assert go(v=K) == SHAPE and go(v=K + size * 128) == SHAPE and go(v=K + size * 256) == SHAPE
    # heads of K and V side by side in rows of one buffer are no overlap (here caught by nothing but that check)
    for gap, status in ((256, None), (248, SHAPE), (512, None), (776, SHAPE), (768, None)):
        rc = _lib.load().paro_kv_read(ctypes.byref(c), 0, K, 1024, 128, K + size * gap, 1024, 128, out, LIST, CU + 4, None,
                                      1, 2, None)
        assert rc == ALIGN  # (alignment comes first, so that nothing here is launched)
        if status:
            assert read(c, k=K, kt=1024, v=K + size * gap, vt=1024, out=out, tokens=2) == status


def test_binding():
    c = paro.KVCache.empty(1, 4, 2, 16, 128, 3, 2, torch.bfloat16, device="cpu", bits=4)
    assert c.bits == 4 and c.dtype == torch.bfloat16 and c.k.shape == (1, 4, 2, 16, 72) and c.k.dtype == torch.uint8
    assert c.c.dt == paro.KV4_BF16 and c.c.head_dim == 128 and c.c.page_size == 16
    wide = paro.KVCache.empty(1, 4, 2, 16, 128, 3, 2, torch.float16, device="cpu")
    assert wide.bits == 16 and wide.c.dt == paro.F16
    tables = (c.refs, c.table, c.lengths)
    with pytest.raises(paro.ParoError):  # the rows' type is needed
        paro.KVCache(c.k, c.v, *tables)
    with pytest.raises(paro.ParoError):
        paro.KVCache(c.k, c.v, *tables, dtype=torch.float32)
    with pytest.raises(paro.ParoError):
        paro.KVCache(c.k[..., :64].contiguous(), c.v[..., :64].contiguous(), *tables, dtype=torch.float16)
    with pytest.raises(paro.ParoError):
        paro.KVCache(wide.k, wide.v, *tables, dtype=torch.bfloat16)
    with pytest.raises(paro.ParoError):
        paro.KVCache.empty(1, 4, 2, 16, 128, 3, 2, torch.float16, device="cpu", bits=8)
    with pytest.raises(paro.ParoError):
        paro.KVCache.empty(1, 4, 2, 16, 96, 3, 2, torch.float16, device="cpu", bits=4)
    k = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    s, cu = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(paro.ParoError, match="device memory"):
        paro.paro_kv_read(c, 0, k, k.clone(), s)
    for call in (lambda: paro.paro_kv_read(c, 0, None, None, s), lambda: paro.paro_kv_read(c, 0, k.half(), None, s),
                 lambda: paro.paro_kv_read(c, 0, k, k.float(), s), lambda: paro.paro_kv_read(c, 0, k[:2], k, s),
                 lambda: paro.paro_kv_read(c, 0, k, k, s, cu[:3]), lambda: paro.paro_kv_read(c, 0, k, k, s, cu, first=cu),
                 lambda: paro.paro_kv_read(c, 0, k[:, :1], None, s), lambda: paro.paro_kv_append(c, 0, k.half(), k.half(), s)):
        with pytest.raises(paro.ParoError):
            call()


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("page,dim", [(16, 64), (32, 128)])
def test_the_format_of_the_tests(dtype, page, dim):
    """Every code has a place of its own, and packing and unpacking agree."""
    for key in (True, False):
        byte, bit = _kv4.places(page, dim, key)
        assert len(set(zip(byte.flatten().tolist(), bit.flatten().tolist()))) == page * dim
        assert int(byte.max()) == page * dim // 2 - 1 and set(bit.flatten().tolist()) == {0, 4}
        x = torch.randn((3, 2, page, dim), generator=torch.Generator().manual_seed(dim)).to(dtype)
        held = _kv4.values_of(_kv4.pages_of(x, key), dtype, key)
        assert torch.equal(held, _kv4.stands_for(*_kv4.quantise(x)))
    # worked words: channels 0..7 of a K row hold codes 0..7, channels 0..3 of a V row codes 1..4
    x = torch.zeros((1, 1, page, dim))
    x[0, 0, 0, :64] = torch.arange(64) % 16
    k = _kv4.pages_of(x.to(dtype), True)[0, 0].flatten()
    assert k[:4].tolist() == [0x20, 0x64, 0x31, 0x75]
    x[0, 0, 0, :5] = torch.tensor([1.0, 2.0, 3.0, 4.0, 0.0])
    v = _kv4.pages_of(x.to(dtype), False)[0, 0].flatten()
    assert v[:2].tolist() == [0x21, 0x43]
