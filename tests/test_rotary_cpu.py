"""Host side of the rotary positions (no GPU): refusals, and the frequencies against their formulas."""
import ctypes
import math

import pytest

paro = pytest.importorskip("rotation_int4_weight_amd")
from rotation_int4_weight_amd import _lib  # noqa: E402

torch = pytest.importorskip("torch")

NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED = 1, 2, 3, 4, 5
A, STEP = 1 << 40, 1 << 36  # addresses that are checked, never used
X, Y, POS, FREQ = (A + i * STEP for i in range(4))


def shape(**kw):
    f = dict(heads=4, head_dim=128, rot_dim=128, interleaved=0, inverse=0, magnitude=1.0, x_token=512, x_head=128,
             y_token=512, y_head=128)
    f.update(kw)
    return _lib.ParoRotaryShapeC(*[f[n] for n, _ in _lib.ParoRotaryShapeC._fields_])


def rotary(s=None, x=X, dt=0, pos=POS, freqs=FREQ, tokens=0, y=Y):
    return _lib.load().paro_rotary(ctypes.byref(s or shape()), x, dt, pos, freqs, tokens, y, None)


def test_nothing_to_do_is_ok():
    assert rotary() == 0 and rotary(dt=1) == 0 and rotary(dt=2) == 0 and rotary(x=None, y=None, pos=None) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(heads=0), SHAPE), (dict(heads=257), SHAPE), (dict(head_dim=0), UNSUPPORTED), (dict(head_dim=100), UNSUPPORTED),
    (dict(head_dim=520), UNSUPPORTED), (dict(rot_dim=0), SHAPE), (dict(rot_dim=127), SHAPE), (dict(rot_dim=130), SHAPE),
    (dict(magnitude=float("nan")), SHAPE), (dict(magnitude=float("inf")), SHAPE), (dict(x_token=4), SHAPE),
    (dict(x_head=-8), SHAPE), (dict(y_token=1 << 40), SHAPE), (dict(y_token=0), SHAPE), (dict(y_head=64), SHAPE),
    (dict(y_token=448), SHAPE)])
def test_shapes_are_refused(bad, status):
    assert rotary(shape(**bad), tokens=3) == status
    assert paro.paro_last_error()


def test_arguments():
    assert rotary(dt=3, tokens=3) == DTYPE and rotary(dt=16, tokens=3) == DTYPE and rotary(dt=-1, tokens=3) == DTYPE
    assert rotary(tokens=-1) == SHAPE and rotary(tokens=(1 << 21) + 1) == UNSUPPORTED
    for name in ("x", "y", "pos", "freqs"):
        assert rotary(tokens=3, **{name: None}) == NULL
    assert rotary(tokens=3, x=X + 8) == ALIGN and rotary(tokens=3, y=Y + 8) == ALIGN
    assert rotary(tokens=3, pos=POS + 2) == ALIGN and rotary(tokens=3, freqs=FREQ + 4) == ALIGN
    # y over an input: the same tensor only with the same strides
    assert rotary(tokens=3, y=X + 128) == SHAPE and rotary(tokens=3, y=POS) == SHAPE and rotary(tokens=3, y=FREQ) == SHAPE
    assert rotary(shape(x_token=1024), tokens=3, y=X) == SHAPE and rotary(shape(y_head=136, y_token=640), tokens=3, y=X) == SHAPE
    assert _lib.load().paro_rotary(None, X, 0, POS, FREQ, 3, Y, None) == NULL


def test_binding_refuses_host_tensors_and_mismatches():
    x = torch.zeros((3, 2, 64), dtype=torch.float16)
    pos, f = torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(paro.ParoError, match="device memory"):
        paro.paro_rotary(x, pos, f, x)
    for call in (lambda: paro.paro_rotary(x, pos[:2], f, x), lambda: paro.paro_rotary(x, pos.long(), f, x),
                 lambda: paro.paro_rotary(x, pos, f.float(), x), lambda: paro.paro_rotary(x, pos, f, x[:2]),
                 lambda: paro.paro_rotary(x, pos, f, x.float()), lambda: paro.paro_rotary(x.double(), pos, f, x.double()),
                 lambda: paro.paro_rotary(x.transpose(1, 2), pos, f, x)):
        with pytest.raises(paro.ParoError):
            call()


def freqs(rot, **kw):
    f, m = paro.paro_rotary_frequencies(rot, device="cpu", **kw)
    return f.tolist(), m


def near(got, want):
    return len(got) == len(want) and all(abs(a - b) <= 1e-13 * abs(b) for a, b in zip(got, want))


@pytest.mark.parametrize("rot", [2, 6, 64, 128, 510])
def test_frequencies(rot):
    base, n = 500000.0, rot // 2
    plain = [base ** (-2 * i / rot) for i in range(n)]
    assert near(freqs(rot, base=base)[0], plain) and freqs(rot)[1] == 1.0
    f, m = freqs(rot, base=base, kind="linear", factor=4.0)
    assert near(f, [x / 4 for x in plain]) and m == 1.0
    if rot >= 4:
        f, _ = freqs(rot, base=base, kind="base", factor=8.0)
        assert f[0] == 1.0 and abs(f[-1] - plain[-1] / 8) <= 1e-12 * plain[-1]
    # by the turns over the trained context
    context, low, high, factor = 8192.0, 1.0, 4.0, 8.0
    want = []
    for x in plain:
        turns = context * x / (2 * math.pi)
        if turns >= high:
            want.append(x)
        elif turns <= low:
            want.append(x / factor)
        else:
            k = (turns - low) / (high - low)
            want.append(k * x + (1 - k) * x / factor)
    assert near(freqs(rot, base=base, kind="bands", context=context, factor=factor)[0], want)
    # by the index: the pairs that make 32 turns and one, and a line between
    first = max(0, math.floor(rot * math.log(context / (32 * 2 * math.pi)) / (2 * math.log(base))))
    last = min(rot - 1, math.ceil(rot * math.log(context / (2 * math.pi)) / (2 * math.log(base))))
    want = []
    for i, x in enumerate(plain):
        r = 0.0 if i <= first else 1.0 if i >= last else (i - first) / (last - first)
        want.append(x * (1 - r) + x / factor * r)
    f, m = freqs(rot, base=base, kind="ramp", context=context, factor=factor)
    assert near(f, want) and m == pytest.approx(0.1 * math.log(8.0) + 1, rel=1e-7)


def test_frequencies_are_refused():
    c = lambda **kw: _lib.ParoRotaryScalingC(*[dict(dict(kind=0, base=1e4, factor=2.0, context=4096.0, low=1.0, high=4.0), **kw)[n]  # noqa: E731
                                               for n, _ in _lib.ParoRotaryScalingC._fields_])
    out = (ctypes.c_double * 256)()
    call = lambda rot=64, **kw: _lib.load().paro_rotary_frequencies(ctypes.byref(c(**kw)), rot, out, None)  # noqa: E731
    assert call() == 0 and call(rot=512) == 0
    for rot in (0, -2, 63, 514):
        assert call(rot=rot) == SHAPE
    assert call(rot=2, kind=2) == SHAPE and call(rot=2, kind=1) == 0
    assert call(kind=5) == UNSUPPORTED and call(kind=-1) == UNSUPPORTED
    nan, inf = float("nan"), float("inf")
    for bad in (dict(base=1.0), dict(base=nan), dict(base=inf), dict(kind=1, factor=0.5), dict(kind=1, factor=nan),
                dict(kind=3, context=0.0), dict(kind=3, low=0.0), dict(kind=3, high=1.0), dict(kind=4, high=inf),
                dict(kind=4, context=nan)):
        assert call(**bad) == SHAPE, bad
    assert call(factor=nan) == 0 and call(kind=1, context=nan) == 0  # not used
    lib = _lib.load()
    assert lib.paro_rotary_frequencies(None, 64, out, None) == NULL
    assert lib.paro_rotary_frequencies(ctypes.byref(c()), 64, None, None) == NULL
    with pytest.raises(paro.ParoError):
        paro.paro_rotary_frequencies(64, kind="other", device="cpu")
