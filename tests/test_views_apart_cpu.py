"""Outputs that are views apart of one buffer, rows or heads in turn, against the elements themselves (no GPU: every call
here is refused, those on views apart by a later check)."""
import ctypes
import random

import pytest

paro = pytest.importorskip("rotation_int4_weight_amd")
pytest.importorskip("torch")
from rotation_int4_weight_amd import _lib  # noqa: E402
from test_attention_abi_cpu import K, cache  # noqa: E402
from test_kv4_abi_cpu import read  # noqa: E402
from test_rotary_cpu import SHAPE, X, rotary, shape  # noqa: E402

SIZE = {0: 2, 1: 2, 2: 4}


def elements(at, rows, heads, dim, token, head):
    return {at + r * token + h * head + c for r in range(rows) for h in range(heads) for c in range(dim)}


def apart(rows, heads, token, head, dim):
    """Rows and heads lie apart from each other, the one inside the other."""
    return (heads == 1 or head >= dim) and (rows == 1 or token >= (heads - 1) * head + dim) or \
        (rows == 1 or token >= dim) and (heads == 1 or head >= (rows - 1) * token + dim)


def draws(seed, n):
    rng = random.Random(seed)
    while n:
        dim, rows, heads = 8 * rng.randint(1, 3), rng.randint(1, 5), rng.randint(1, 5)
        token, head = 8 * rng.randint(0, 24), 8 * rng.randint(0, 24)
        if apart(rows, heads, token, head, dim):
            n -= 1
            yield rows, heads, dim, token, head, 8 * rng.randint(-60, 60)


def test_rotary_tells_overlaps_from_views_apart():
    seen = set()
    for rows, heads, dim, token, head, delta in draws(1, 1500):
        dt = (rows + heads) % 3
        mine, other = elements(0, rows, heads, dim, token, head), elements(delta, rows, heads, dim, token, head)
        y = X + SIZE[dt] * delta
        # (freqs at y: what is refused when x and y are no overlap)
        assert rotary(shape(heads=heads, head_dim=dim, rot_dim=2, x_token=token, x_head=head, y_token=token, y_head=head),
                      dt=dt, tokens=rows, y=y, freqs=y) == SHAPE
        clash = delta != 0 and bool(mine & other)
        message = paro.paro_last_error()
        assert ("y overlaps x" in message) == clash, (rows, heads, dim, token, head, delta, message)
        assert clash or "freqs" in message
        seen.add((clash, delta != 0 and max(mine) >= min(other) and max(other) >= min(mine)))
    assert seen == {(True, True), (False, True), (False, False)}


def test_rotary_at_the_largest_strides():
    big = (1 << 40) - 8
    for delta, clash in ((8, False), (-8, False), (24, False), (32, True), (4 * big, True), (4 * big + 8, False),
                         (4 * big + 16, True), (-(1 << 20) * big, True), (8 - (1 << 20) * big, False)):
        s = shape(heads=3, head_dim=8, rot_dim=2, x_token=big, x_head=16, y_token=big, y_head=16)
        x = X if delta > 0 else 1 << 62  # (addresses are not below 0)
        y = x + 2 * delta
        assert rotary(s, x=x, tokens=1 << 21, y=y, freqs=y) == SHAPE
        assert ("y overlaps x" in paro.paro_last_error()) == clash, delta
    # other strides than x's: only behind one another
    assert rotary(shape(heads=2, head_dim=8, rot_dim=2, x_token=64, x_head=16, y_token=128, y_head=16), tokens=2,
                  y=X + 16, freqs=X + 16) == SHAPE and "y overlaps x" in paro.paro_last_error()
    # the strides of a single row or head do not matter
    for kw in (dict(heads=1, x_head=0, y_head=48, x_token=64, y_token=64), dict(heads=3, x_head=32, y_head=32, x_token=0, y_token=640)):
        n = 1 if kw["heads"] == 3 else 4
        assert rotary(shape(head_dim=16, rot_dim=2, **kw), tokens=n, y=X + 32, freqs=X + 32) == SHAPE
        assert "freqs" in paro.paro_last_error()


def test_read_tells_overlaps_from_views_apart():
    """K and V of one buffer; `first` at K is what is refused where they are no overlap."""
    seen = set()
    rng = random.Random(2)
    while len(seen) < 3 or rng.random() > 0.001:
        rows, heads, dim, dt = rng.randint(1, 4), rng.randint(1, 4), 64, rng.randint(0, 1)
        token, head, delta = (64 * rng.randint(0, 12) + 8 * rng.randint(-1, 1) for _ in range(3))
        delta *= rng.choice((-1, 1))
        if min(token, head) < 0 or not apart(rows, heads, token, head, dim):
            continue
        out = rng.choice((dt, 2))
        v = K + SIZE[out] * delta
        c = cache(dt=dt + 16 * rng.randint(0, 1), head_dim=dim, kv_heads=heads)
        assert read(c, k=K, kt=token, kh=head, v=v, vt=token, vh=head, out=out, n=1, tokens=rows, first=K) == SHAPE
        mine, other = elements(0, rows, heads, dim, token, head), elements(delta, rows, heads, dim, token, head)
        clash, message = bool(mine & other), paro.paro_last_error()
        assert ("k and v overlap" in message) == clash, (rows, heads, token, head, delta, message)
        assert clash or "first" in message
        seen.add((clash, max(mine) >= min(other) and max(other) >= min(mine)))


def test_read_of_a_single_row_or_head():
    """Their strides do not matter."""
    c = cache(kv_heads=2)
    assert read(c, k=K, kt=1024, kh=256, v=K + 2 * 128, vt=512, vh=256, tokens=1, first=K) == SHAPE
    assert "first" in paro.paro_last_error()
    assert read(c, k=K, kt=1024, kh=256, v=K + 2 * 128, vt=512, vh=256, tokens=2, first=K) == SHAPE
    assert "k and v overlap" in paro.paro_last_error()
    c = cache(kv_heads=1)
    assert read(c, k=K, kt=512, kh=0, v=K + 2 * 128, vt=512, vh=1024, tokens=3, first=K) == SHAPE
    assert "first" in paro.paro_last_error()
