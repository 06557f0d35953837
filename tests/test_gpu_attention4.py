"""Decode attention over the cache in four bits through the C-ABI, against attention in 64 bits over the values that
the cache's bytes stand for."""
import pytest

from _attention import offsets

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")
import _kv4  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = (torch.float16, torch.bfloat16)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rows(shape, dtype, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def decode(c, q, slots, scale=None, layer=0, ws=None, y=None):
    y = torch.full_like(q, float("nan")) if y is None else y
    ws = paro.make_workspace(paro.paro_attention_decode_workspace_bytes(c, q.shape[0], q.shape[1])) if ws is None else ws
    paro.paro_attention_decode(c, layer, q, slots, y, ws, scale=scale)
    return y


def check(c, q, slots, y, scale=None, layer=0):
    scale = _kv4.default_scale(q.shape[2]) if scale is None else scale
    known = {}
    for r, s in enumerate(slots):
        if not 0 <= s < c.c.slots or int(c.lengths[s]) == 0:
            assert bool((y[r] == 0).all())
            continue
        if s not in known:
            known[s] = _kv4.held_rows(c, layer, s)
        _kv4.check_decode(y[r], q[r], *known[s], scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_lengths(dtype, dim, page):
    """Every length around a block, a step, a workgroup's unit and the whole rows' limit; behind the end lie pairs of
    NaN and codes of 15."""
    lengths = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 160, 255, 257, 383, 384, 385, 513, 700, 1100]
    c = _kv4.fill(paro, lengths, page, 2, dim, dtype, page + dim, layers=2)
    slots = list(range(len(lengths)))[::-1] + [-1, len(lengths), 7, 7]
    q = rows((len(slots), 6, dim), dtype, 3)
    y = decode(c, q, ints(slots), layer=1)
    check(c, q, slots, y, layer=1)
    # again: the same bits
    assert torch.equal(y.view(torch.int16), decode(c, q, ints(slots), layer=1).view(torch.int16))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (3, 2), (2, 3), (2, 5), (2, 7), (1, 8), (1, 9), (1, 16), (2, 17),
                                            (1, 40), (8, 4), (5, 1), (1, 256), (256, 1)])
def test_heads(dtype, kv_heads, group):
    lengths = [300, 45]
    for dim in (64, 128):
        c = _kv4.fill(paro, lengths, 32, kv_heads, dim, dtype, group)
        q = rows((2, kv_heads * group, dim), dtype, 1)
        check(c, q, [1, 0], decode(c, q, ints([1, 0])))


@pytest.mark.parametrize("rows_", [1, 2, 5, 40, 70, 300])
def test_rows_share_the_card(rows_):
    """Few rows are split over workgroups and joined, many are not; rows beside each other have very different lengths."""
    lengths = [1 + (i * 1237 + 5) % 3000 for i in range(8)]
    c = _kv4.fill(paro, lengths, 16, 4, 128, torch.bfloat16, 9)
    slots = [(3 * i) % 8 for i in range(rows_)]
    q = rows((rows_, 8, 128), torch.bfloat16, rows_)
    y = decode(c, q, ints(slots))
    check(c, q[:24], slots[:24], y[:24])
    # a repeated call gives the same bits
    assert torch.equal(y.view(torch.int16), decode(c, q, ints(slots)).view(torch.int16))


@pytest.mark.parametrize("rows_,most", [(30, 400), (64, 700), (65, 900), (200, 500), (300, 900), (300, 2500), (1024, 1500),
                                        (600, 130), (1500, 100), (4096, 60), (4097, 300)])
def test_many_rows(rows_, most):
    """Every row of calls whose outputs are cut, have a workgroup each, and have a wave each; one row is far the
    longest where rows are many, some are empty and some name no slot."""
    lengths = [most] + [(i * 1237 + 5) % (most // 4) for i in range(12)] + [0]
    c = _kv4.fill(paro, lengths, 16, 2, 64, torch.float16, 9)
    slots = [(5 * i + 1) % 15 - 1 if rows_ <= 64 or i % 97 else 0 for i in range(rows_)]
    q = rows((rows_, 6, 64), torch.float16, rows_)
    y = decode(c, q, ints(slots))
    check(c, q, slots, y)
    assert torch.equal(y.view(torch.int16), decode(c, q, ints(slots)).view(torch.int16))


def test_the_most_rows():
    c = _kv4.fill(paro, [70, 0, 300, 5], 16, 1, 64, torch.bfloat16, 3)
    q, slots = rows((8, 2, 64), torch.bfloat16, 1), [0, 3, 1, 2, -1, 2, 4, 0]
    y = decode(c, q.repeat(4096, 1, 1), ints(slots).repeat(4096)).view(4096, 8, 2, 64)
    check(c, q, slots, y[0])
    assert torch.equal(y.view(torch.int16), y[:1].expand(4096, 8, 2, 64).contiguous().view(torch.int16))


@pytest.mark.parametrize("dtype", TYPES)
def test_a_long_row(dtype):
    c = _kv4.fill(paro, [20011, 3], 64, 1, 128, dtype, 2)
    q = rows((2, 4, 128), dtype, 4)
    y = decode(c, q, ints([0, 1]))
    check(c, q, [0, 1], y)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 2.0, 1e-30])
def test_scales(dtype, scale):
    c = _kv4.fill(paro, [90, 500], 16, 2, 64, dtype, 2)
    q = rows((2, 4, 64), dtype, 4)
    check(c, q, [0, 1], decode(c, q, ints([0, 1]), scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k_scale,v_scale,q_scale", [
    (1e-3, 1e-3, 1.0), (30.0, 1.0, 0.02), (1.0, 2000.0, 1.0), (1.0, 1e-6, 1.0), (1e-4, 1.0, 6000.0), (0.0, 1.0, 1.0),
    (1.0, 0.0, 1.0)])
def test_sizes_of_values(dtype, k_scale, v_scale, q_scale):
    for dim in (64, 128):
        c = _kv4.fill(paro, [33, 600], 16, 2, dim, dtype, 2, k_scale=k_scale, v_scale=v_scale)
        q = rows((2, 4, dim), dtype, 4, q_scale)
        check(c, q, [0, 1], decode(c, q, ints([0, 1])))


def pairs_view(c, t):
    """The pairs of a cache's K or V: (layers, pages, heads, page, dim / 64, 2) in the rows' type, a view."""
    page, dim = c.c.page_size, c.c.head_dim
    return t.flatten(3)[..., page * dim // 2:].view(c.dtype).unflatten(-1, (page, dim // 64, 2))


def test_bfloat16_values_far_outside_fp16():
    """Scales, lows and queries that fp16 could not hold: 2^100 and 2^-100, finite results."""
    for exponent in (100, 60, -60, -100):
        for dim in (64, 128):
            c = _kv4.fill(paro, [33, 600], 16, 2, dim, torch.bfloat16, 2)
            q = rows((2, 4, dim), torch.bfloat16, 4)
            kp, vp = pairs_view(c, c.k), pairs_view(c, c.v)
            kp.copy_((kp.float() * 2.0 ** -exponent).to(c.dtype))
            vp.copy_((vp.float() * 2.0 ** exponent).to(c.dtype))
            q = (q.float() * 2.0 ** exponent).to(torch.bfloat16)
            y = decode(c, q, ints([0, 1]))
            assert bool(torch.isfinite(y).all())
            check(c, q, [0, 1], y)


def test_one_key_with_a_scale_far_over_the_others():
    """Weights are relative to the largest scale so far, which comes early, late, or never."""
    for dtype in TYPES:
        for at in (0, 70, 599):
            for factor in (1000.0, 2.0 ** -12):
                c = _kv4.fill(paro, [600], 16, 1, 128, dtype, 2)
                page, p = int(c.table[0, at // 16]), at % 16
                vp = pairs_view(c, c.v)
                vp[0, page, 0, p, 1] = (vp[0, page, 0, p, 1].float() * factor).to(dtype)
                q = rows((1, 4, 128), dtype, 4)
                check(c, q, [0], decode(c, q, ints([0])))


def test_scores_below_the_range_of_fp32_weigh_nothing():
    """Keys whose products leave fp32 downwards fill whole steps, the first ones and others, of some waves."""
    c = _kv4.fill(paro, [300], 16, 1, 64, torch.bfloat16, 2)
    kp = pairs_view(c, c.k)
    for p in [*range(64), *range(160, 192), 250]:
        kp[0, int(c.table[0, p // 16]), 0, p % 16, 0, 0] = 0.0
        kp[0, int(c.table[0, p // 16]), 0, p % 16, 0, 1] = -3e38
    q = rows((1, 3, 64), torch.bfloat16, 4).abs() + 100.0
    kept = [p for p in range(300) if p not in {*range(64), *range(160, 192), 250}]
    k, v = _kv4.held_rows(c, 0, 0)
    y = decode(c, q, ints([0]), scale=0.01)
    _kv4.check_decode(y[0], q[0], k[kept], v[kept], 0.01)


def test_queries_of_one_large_channel():
    for dtype in TYPES:
        c = _kv4.fill(paro, [200], 16, 1, 128, dtype, 2, k_scale=0.01)
        q = rows((1, 2, 128), dtype, 4, 1e-3)
        q[0, 0, 77] = 60000.0
        q[0, 1, 2] = -3000.0
        check(c, q, [0], decode(c, q, ints([0]), scale=1e-4), scale=1e-4)


def test_largest_fp16_values_stay_finite():
    c = _kv4.fill(paro, [257], 16, 1, 64, torch.float16, 2)
    vp = pairs_view(c, c.v)
    vp[..., 0] = 0
    vp[..., 1] = 65504.0
    q = rows((1, 3, 64), torch.float16, 4)
    y = decode(c, q, ints([0]))
    assert bool((y == 65504.0).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_groups_that_are_not_finite(dtype):
    """A NaN pair of V: that group of 64 channels of every query head, and nothing else; of K: the whole row."""
    c = _kv4.fill(paro, [300, 300], 16, 2, 128, dtype, 2)
    q = rows((2, 6, 128), dtype, 4)
    good = decode(c, q, ints([0, 1]))
    vp = pairs_view(c, c.v)
    keep = vp.clone()
    vp[0, int(c.table[0, 5]), 1, 3, 0] = float("nan")
    y = decode(c, q, ints([0, 1]))
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, 3:, :64] = True
    assert torch.equal(y.isnan(), bad) and torch.equal(y[~bad], good[~bad])
    vp.copy_(keep)
    pairs_view(c, c.k)[0, int(c.table[1, 5]), 0, 3, 1] = float("nan")
    y = decode(c, q, ints([0, 1]))
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1, :3] = True
    assert torch.equal(y.isnan(), bad) and torch.equal(y[~bad], good[~bad])
    q[0, 2, 9] = float("nan")
    y = decode(c, q, ints([0, 1]))
    bad[0, 2] = True
    assert torch.equal(y.isnan(), bad) and torch.equal(y[~bad], good[~bad])


def test_strided_queries_and_outputs():
    dtype, dim = torch.bfloat16, 128
    c = _kv4.fill(paro, [100, 40, 7], 16, 2, dim, dtype, 2)
    fused = rows((3, 12, dim), dtype, 4)
    q = fused[:, 1:9]
    out = torch.full((8, 5, dim + 8), 7.0, dtype=dtype, device="cuda")
    y = out.transpose(0, 1)[1:4, :, :dim]
    decode(c, q, ints([2, 0, 1]), y=y)
    check(c, q, [2, 0, 1], y)
    assert bool((out[:, [0, 4]] == 7).all()) and bool((out[..., dim:] == 7).all())


def test_an_invalid_state_reads_inside_the_cache():
    """Tables of nonsense, lengths past the end: wrong numbers or none, no access out of bounds, rows beside unharmed."""
    c = _kv4.fill(paro, [100, 64, 40], 16, 2, 64, torch.float16, 2)
    q = rows((3, 4, 64), torch.float16, 4)
    good = decode(c, q, ints([0, 1, 2]))
    c.table[1, :] = ints([-5, 10 ** 6, 3, -1] * 10)[:c.table.shape[1]]
    c.lengths[2] = 10 ** 9
    c.lengths[1] = 64
    y = decode(c, q, ints([0, 1, 2]))
    torch.cuda.synchronize()
    assert torch.equal(y[0], good[0])
    c.lengths[2] = -4
    assert bool((decode(c, q, ints([0, 1, 2]))[2] == 0).all())


def test_workspaces_streams_and_graphs():
    """Two streams with a workspace each; a captured call replayed with new lengths and queries; one workspace that the
    16-bit form used before."""
    dtype, dim = torch.bfloat16, 128
    lengths = [900, 1500, 31, 700]
    c = _kv4.fill(paro, lengths, 16, 2, dim, dtype, 2)
    qs = [rows((4, 8, dim), dtype, i) for i in range(3)]
    need = paro.paro_attention_decode_workspace_bytes(c, 4, 8)
    slots = ints([0, 1, 2, 3])
    want = [decode(c, q, slots) for q in qs]
    torch.cuda.synchronize()
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [paro.make_workspace(need) for _ in range(2)]
    got = [[torch.empty_like(q) for q in qs] for _ in range(2)]
    for i, q in enumerate(qs):
        for s, w, y in zip(streams, spaces, got):
            paro.paro_attention_decode(c, 0, q, slots, y[i], w, stream=s)
    torch.cuda.synchronize()
    for y in got:
        assert all(torch.equal(a, b) for a, b in zip(y, want))
    assert not spaces[0][:1 << 21].any()  # the counter area is left zero
    q, y = qs[0].clone(), torch.empty_like(qs[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        paro.paro_attention_decode(c, 0, q, slots, y, spaces[0])
    for i in (0, 1, 2, 0, 1):
        q.copy_(qs[i])
        c.lengths.copy_(ints(lengths if i else [5, 0, 31, 699]))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, decode(c, q, slots, ws=spaces[1])) and (i == 0 or torch.equal(y, want[i]))


def test_the_largest_offsets():
    """Pages past 2^32 bytes of a pool, and a table that names them."""
    dtype, dim, page, heads = torch.float16, 128, 256, 8
    block = heads * page * dim * 9 // 16
    pages = (1 << 32) // block + 40
    c = paro.KVCache.empty(1, pages, heads, page, dim, 1, 4, dtype, bits=4)
    table = ints([[pages - 1, 3, pages - 7, -1]])
    c.table.copy_(table)
    c.lengths.copy_(ints([700]))
    k, v = rows((700, heads, dim), dtype, 1), rows((700, heads, dim), dtype, 2)
    paro.paro_kv_append(c, 0, k, v, ints([0]), offsets([700]))
    held = _kv4.held_rows(c, 0, 0)
    assert torch.equal(held[0], _kv4.stands_for(*_kv4.quantise(k.cpu())))
    assert torch.equal(held[1], _kv4.stands_for(*_kv4.quantise(v.cpu())))
    q = rows((1, 32, dim), dtype, 3)
    check(c, q, [0], decode(c, q, ints([0])))
    got = torch.empty((700, heads, dim), device="cuda")
    paro.paro_kv_read(c, 0, got, None, ints([0]), offsets([700]))
    assert bool(((got.cpu().double() - held[0]).abs() <= 2.0 ** -24 * held[0].abs()).all())
