"""Rotary positions through the C-ABI against the definition in 64 bits: layouts, parts of the head, types, strides,
far positions, in place, the gradient."""
import pytest

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0, torch.float32: 0.0}
TYPES = (torch.float16, torch.bfloat16, torch.float32)


def definition(x, positions, freqs, interleaved, inverse=False, magnitude=1.0):
    """y and the size of its terms, more where angles are so large that 64 bits round them, in 64 bits."""
    x, rot = x.double().cpu(), 2 * freqs.numel()
    angle = positions.cpu().double()[:, None, None] * freqs.cpu().double()
    cos, sin = angle.cos() * magnitude, angle.sin() * (-magnitude if inverse else magnitude)
    y, size = x.clone(), torch.zeros_like(x)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    size[..., a] = size[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(magnitude) * (1 + 2.0 ** -29 * angle.abs())
    return y, size


def check(got, x, positions, freqs, interleaved, inverse=False, magnitude=1.0):
    """Sine and cosine within 2^-22 (an angle within half a quarter turn rounded to 2^-26 of one, a function within two
    units, the magnitude), products and sum rounded in fp32, one rounding of the output."""
    y, size = definition(x, positions, freqs, interleaved, inverse, magnitude)
    # (2^-22 * 2^-29 of the angle: one rounding of it on either side, 2^-53 each, with room for the reduction's)
    limit = HALF_STEP[got.dtype] * y.abs() + size * (2.0 ** -22 + 2 * 2.0 ** -24) * 1.01 + TINY[got.dtype]
    off = (got.double().cpu() - y).abs()
    assert bool((off <= limit).all()), f"off by {float(off.max()):.3e} ({int((off > limit).sum())} values)"
    rot = 2 * freqs.numel()
    assert torch.equal(got[..., rot:], x[..., rot:])


def randn(shape, dtype, seed):
    return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(dtype)


def ints(n, seed, low=0, high=5000):
    return torch.randint(low, high, (n,), generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()


def frequencies(rot, **kw):
    return paro.paro_rotary_frequencies(rot, **kw)[0]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(8, 2), (8, 8), (64, 64), (64, 32), (80, 20), (80, 22), (96, 48), (128, 128),
                                     (128, 126), (256, 64), (512, 512), (512, 6), (64, 24), (128, 56), (72, 36)])
def test_sizes(dtype, interleaved, dim, rot):
    for tokens, heads in ((1, 1), (5, 3), (67, 2), (300, 1)):
        x, pos = randn((tokens, heads, dim), dtype, dim + rot), ints(tokens, rot)
        y = torch.full_like(x, float("nan"))
        f = frequencies(rot, base=1000.0)
        paro.paro_rotary(x, pos, f, y, interleaved=interleaved)
        check(y, x, pos, f, interleaved)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_heads_and_tokens(dtype):
    for tokens, heads, dim, rot in ((1, 256, 8, 2), (3, 256, 128, 128), (2000, 40, 128, 128), (4099, 9, 64, 64),
                                    (1, 256, 512, 6)):
        x, pos = randn((tokens, heads, dim), dtype, tokens), ints(tokens, heads)
        y, f = torch.full_like(x, float("nan")), frequencies(rot)
        paro.paro_rotary(x, pos, f, y, magnitude=1.25)
        check(y, x, pos, f, False, magnitude=1.25)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved):
    """Angles that 32 bits would lose: positions up to 2^31 - 1, turning by one radian each; in fp32 and whole turns."""
    pos = torch.tensor([0, 1, -1, 1 << 20, (1 << 20) + 1, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31, 123456789],
                       dtype=torch.int32, device="cuda")
    for kind in ("none", "linear", "base", "bands", "ramp"):
        f, m = paro.paro_rotary_frequencies(64, base=500000.0, kind=kind, factor=8.0, context=8192.0)
        x = randn((len(pos), 3, 64), torch.float32, 5)
        y = torch.empty_like(x)
        paro.paro_rotary(x, pos, f, y, interleaved=interleaved, magnitude=m)
        check(y, x, pos, f, interleaved, magnitude=m)


def test_quarter_turns():
    """Whole quarters: sine and cosine are 0 and 1, in every quadrant and direction."""
    f = torch.full((4,), torch.pi / 2, dtype=torch.float64, device="cuda")
    pos = torch.arange(-9, 10, dtype=torch.int32, device="cuda")
    x = randn((19, 2, 8), torch.float32, 8)
    for inverse in (False, True):
        y = torch.empty_like(x)
        paro.paro_rotary(x, pos, f, y, inverse=inverse)
        check(y, x, pos, f, False, inverse)
        a, b = x[..., :4], x[..., 4:]
        for i, p in enumerate(pos.tolist()):
            q = (-p if inverse else p) % 4
            want = [(a, b), (-b, a), (-a, -b), (b, -a)][q]
            off = (y[i] - torch.cat([w[i] for w in want], -1)).abs().max()
            assert float(off) <= 1e-6


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_views_and_in_place(dtype, interleaved):
    tokens, dim = 70, 64
    fused = randn((tokens, 12, dim), dtype, 3)  # 6 q, 2 k, 4 others
    before = fused.clone()
    pos, f = ints(tokens, 3), frequencies(48)
    x = fused[:, 1:9]
    # into a (heads, tokens, dim) tensor, with a gap behind each row that stays
    out = torch.full((8, tokens + 2, dim + 8), 7.0, dtype=dtype, device="cuda")
    y = out.transpose(0, 1)[:tokens, :, :dim]
    paro.paro_rotary(x, pos, f, y, interleaved=interleaved)
    check(y, x, pos, f, interleaved)
    assert bool((out[:, tokens:] == 7).all()) and bool((out[..., dim:] == 7).all())
    # in place: the same values, and the heads beside stay
    paro.paro_rotary(x, pos, f, x, interleaved=interleaved)
    assert torch.equal(fused[:, 1:9], y) and torch.equal(fused[:, 0], before[:, 0]) and torch.equal(fused[:, 9:], before[:, 9:])
    # one row for all tokens, one head for all heads
    one = randn((1, 1, dim), dtype, 4).expand(tokens, 3, dim)
    z = torch.empty((tokens, 3, dim), dtype=dtype, device="cuda")
    paro.paro_rotary(one, pos, f, z, interleaved=interleaved)
    check(z, one, pos, f, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 26])
def test_inverse_is_the_gradient(interleaved, rot):
    tokens, heads, dim = 9, 2, 64
    pos = ints(tokens, 2, high=100000)
    f, m = paro.paro_rotary_frequencies(rot, kind="ramp", factor=4.0, context=4096.0)
    x, g = randn((tokens, heads, dim), torch.float32, 1), randn((tokens, heads, dim), torch.float32, 2)
    gx = torch.empty_like(g)
    paro.paro_rotary(g, pos, f, gx, interleaved=interleaved, inverse=True, magnitude=m)
    # the formula's
    check(gx, g, pos, f, interleaved, inverse=True, magnitude=m)
    # autograd's of the definition
    leaf = x.double().cpu().requires_grad_()
    y, _ = definition(leaf, pos, f, interleaved, magnitude=m)
    y.backward(g.double().cpu())
    off = (gx.double().cpu() - leaf.grad).abs()
    assert float(off.max()) <= 2.0 ** -21 * float(g.abs().max()) * 2 * m
    # differences of the loss <y, g>: it is linear in x, so a step of any size gives the slope
    def loss(x):
        y = torch.empty_like(x)
        paro.paro_rotary(x, pos, f, y, interleaved=interleaved, magnitude=m)
        return float((y.double() * g.double()).sum())
    for t, h, c in ((0, 0, 0), (3, 1, 1), (5, 0, rot - 1), (8, 1, dim - 1)):
        up, down = x.clone(), x.clone()
        up[t, h, c] += 4.0
        down[t, h, c] -= 4.0
        # 2^-21 for each of the few outputs that change, against a step of 8
        size = 3 * float(g.abs().max()) * (float(x.abs().max()) + 4) * 2.0 ** -21 * 4 / 8
        assert abs((loss(up) - loss(down)) / 8 - float(gx[t, h, c])) <= size + 2.0 ** -21 * 8
    # and back: turned by t, then by -t, with 1 / m^2
    if m != 1.0:
        back = torch.empty_like(x)
        y = torch.empty_like(x)
        paro.paro_rotary(x, pos, f, y, interleaved=interleaved, magnitude=m)
        paro.paro_rotary(y, pos, f, back, interleaved=interleaved, inverse=True, magnitude=1 / m ** 1)
        off = (back[..., :rot] - x[..., :rot]).abs().max()
        assert float(off) <= 2.0 ** -19 * float(x.abs().max())


def test_values_that_are_not_finite_stay_in_their_pair():
    x = randn((3, 2, 64), torch.bfloat16, 1)
    x[1, 0, 5] = float("nan")
    x[2, 1, 40] = float("inf")
    pos, f = ints(3, 1), frequencies(64)
    y = torch.empty_like(x)
    paro.paro_rotary(x, pos, f, y)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 0, [5, 37]] = True
    want[2, 1, [8, 40]] = True
    assert torch.equal(bad, want)


def test_streams_and_graphs():
    x = [randn((50, 6, 128), torch.bfloat16, i) for i in range(2)]
    pos = [ints(50, i) for i in range(2)]
    f = frequencies(128)
    want = []
    for a, p in zip(x, pos):
        y = torch.empty_like(a)
        paro.paro_rotary(a, p, f, y)
        want.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.empty_like(a) for a in x]
    for s, a, p, y in zip(streams, x, pos, got):
        paro.paro_rotary(a, p, f, y, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    a, p, y = x[0].clone(), pos[0].clone(), torch.empty_like(x[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        paro.paro_rotary(a, p, f, y)
    for i in (0, 1, 0, 1):
        a.copy_(x[i])
        p.copy_(pos[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])


def test_the_largest_offsets():
    """Elements past 2^32: a row far behind in a long buffer."""
    dim, tokens = 64, 3
    step = 3 << 29
    flat = torch.zeros(2 * step + 2 * dim, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((tokens, 2, dim), (step, dim, 1))
    x.copy_(randn((tokens, 2, dim), torch.bfloat16, 1))
    pos, f = ints(tokens, 1), frequencies(dim)
    y = torch.empty((tokens, 2, dim), dtype=torch.bfloat16, device="cuda")
    paro.paro_rotary(x, pos, f, y)
    check(y, x, pos, f, False)
    paro.paro_rotary(x, pos, f, x)
    assert torch.equal(x, y)
