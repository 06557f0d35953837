"""The cache in four bits through the C-ABI: rows quantised as they are written, read back, copied by the page calls,
against the documented format and rules."""
import random

import pytest

from _attention import filled_cache, offsets

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")
import _kv4  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = (torch.float16, torch.bfloat16)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rows(shape, dtype, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def empty_cache(lengths, page, kv_heads, dim, dtype, layers=2, spare=3, bits=4, seed=0):
    """A cache whose slots have these lengths and pages in random order; every byte of the pages is 0xA5."""
    counts = [-(-n // page) for n in lengths]
    c = paro.KVCache.empty(layers, sum(counts) + spare, kv_heads, page, dim, len(lengths), max(counts + [0]) + 2, dtype,
                           bits=bits)
    for t in (c.k, c.v):
        t.view(torch.uint8).fill_(0xA5)
    order = list(range(sum(counts) + spare))
    random.Random(seed).shuffle(order)
    table, refs = torch.full(c.table.shape, -1, dtype=torch.int32), torch.zeros(len(order), dtype=torch.int32)
    for i, n in enumerate(counts):
        for j in range(n):
            table[i, j] = order.pop()
            refs[table[i, j]] = 1
    c.table.copy_(table)
    c.refs.copy_(refs)
    c.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
    return c


def written(c, layer, slot, first, x, key, into):
    """Writes rows x (n, heads, dim) at positions first.. of a slot into `into`, the pool's bytes on the host."""
    page, dim, heads = c.c.page_size, c.c.head_dim, c.c.kv_heads
    codes, scale, low = _kv4.quantise(x)
    byte, bit = _kv4.places(page, dim, key)
    pairs = torch.stack([scale, low], -1).contiguous().view(torch.uint8).flatten(2)
    table = c.table.cpu()
    for j in range(x.shape[0]):
        where, p = int(table[slot, (first + j) // page]), (first + j) % page
        flat = into[layer, where].view(heads, -1)
        out = torch.zeros((heads, page * dim // 2), dtype=torch.int64)
        out.index_add_(1, byte[p], codes[j] << bit[p])
        mine = byte[p].unique()
        flat[:, mine] = out[:, mine].to(torch.uint8)
        at = page * dim // 2 + p * dim // 16
        flat[:, at:at + dim // 16] = pairs[j]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page,kv_heads,dim", [(16, 1, 64), (16, 3, 128), (64, 2, 64), (128, 8, 128), (256, 1, 128)])
def test_append_writes_the_format_and_nothing_else(dtype, page, kv_heads, dim):
    prefix, new = [0, 5, 0, 31, 100, 7], [1, 40, 0, 1, 33, 20]
    c = empty_cache([a + b for a, b in zip(prefix, new)], page, kv_heads, dim, dtype)
    total = sum(new)
    # views of a fused buffer, with rows before and behind those of the entries
    fused = rows((total + 5, 2 * kv_heads + 1, dim), dtype, page)
    dev = fused.cuda()
    k, v = dev[:, :kv_heads], dev[:, kv_heads + 1:]
    cu = offsets(new) + 2
    want = [c.k.cpu().clone(), c.v.cpu().clone()]
    for i, (p, n) in enumerate(zip(prefix, new)):
        at = int(cu[i])
        for t, x, key in ((want[0], fused[:, :kv_heads], True), (want[1], fused[:, kv_heads + 1:], False)):
            written(c, 1, i, p, x[at:at + n], key, t)
    paro.paro_kv_append(c, 1, k, v, ints(range(6)), cu)
    assert torch.equal(c.k.cpu(), want[0]) and torch.equal(c.v.cpu(), want[1])


@pytest.mark.parametrize("dtype", TYPES)
def test_append_one_row_each_skips_what_does_not_belong(dtype):
    c = empty_cache([40, 17, 0, 3], 16, 2, 128, dtype)
    c.table[1, 1] = 9999  # no such page: position 16 of slot 1
    x, y = rows((8, 2, 128), dtype, 1), rows((8, 2, 128), dtype, 2)
    slots = [3, 1, 0, 3, -1, 4, 2, 0]
    granted = [1, 1, 0, 1, 1, 1, 1, 1]
    want = [c.k.cpu().clone(), c.v.cpu().clone()]
    written(c, 0, 3, 2, x[0:1], True, want[0])
    written(c, 0, 3, 2, y[0:1], False, want[1])
    paro.paro_kv_append(c, 0, x.cuda(), y.cuda(), ints(slots), granted=ints(granted))
    assert torch.equal(c.k.cpu(), want[0]) and torch.equal(c.v.cpu(), want[1])


def borders(dtype):
    """Rows of one group at the quantiser's borders."""
    big = torch.finfo(dtype).max
    least = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps  # the least subnormal
    g = torch.Generator().manual_seed(3)
    out = [torch.zeros(64), torch.full((64,), -3.5), torch.full((64,), big), torch.linspace(-big, big, 64),
           torch.linspace(-big, 0, 64), torch.tensor([-0.0, 0.0] * 32)]
    for unit in (1.0, 0.25, 0.625, 3.0, 1.875):  # ties: multiples of half a step over 0..15
        for low in (0.0, -4.0, 1.0, -7.5):
            t = low + unit * torch.arange(64).remainder(31) / 2
            t[31] = low + 15 * unit
            out.append(t)
    for n in range(1, 40, 3):  # ranges of a few of the least steps: scales that are subnormal or round to zero
        out.append(least * torch.arange(64).remainder(n + 1))
        out.append(least * (torch.arange(64).remainder(n + 1) - 200.0))
    for e in range(-14, 15, 4):  # one value of another size
        t = torch.randn(64, generator=g)
        t[17] = 2.0 ** e
        out.append(t)
        out.append(t * 2.0 ** -10)
    for bad in (float("nan"), float("inf"), -float("inf")):
        t = torch.randn(64, generator=g)
        t[33] = bad
        out.append(t)
    t = torch.full((64,), float("inf"))
    out += [t, -t, t * 0]
    if dtype == torch.bfloat16:
        out += [torch.linspace(1, 2, 64) * 2.0 ** e for e in (-130, -126, -100, 60, 120, 126)]
        t = torch.linspace(-1, 1, 64)
        t[5] = 2.0 ** 100
        out.append(t)
    while len(out) % 4:
        out.append(torch.randn(64, generator=g))
    return torch.stack(out).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_quantiser_at_its_borders(dtype, dim):
    x = borders(dtype).view(-1, 2, dim)  # (rows, heads, dim): neighbouring groups differ
    n = x.shape[0]
    c = empty_cache([n], 16, 2, dim, dtype, layers=1)
    want = [c.k.cpu().clone(), c.v.cpu().clone()]
    written(c, 0, 0, 0, x, True, want[0])
    written(c, 0, 0, 0, x.flip(0), False, want[1])
    paro.paro_kv_append(c, 0, x.cuda(), x.flip(0).cuda(), ints([0]), offsets([n]))
    k, v = torch.empty((n, 2, dim), device="cuda"), torch.empty((n, 2, dim), device="cuda")
    paro.paro_kv_read(c, 0, k, v, ints([0]), offsets([n]))
    for got, rows_of, t, key in ((k, x, c.k, True), (v, x.flip(0), c.v, False)):
        codes, scale, low = _kv4.quantise(rows_of)
        # (a lowest value of zero may carry either sign)
        held = _kv4.held_rows(c, 0, 0)[0 if key else 1]
        exact = _kv4.stands_for(codes, scale, low)
        same = (held == exact) | (held.isnan() & exact.isnan())
        assert bool(same.all()), (held[~same][:4], exact[~same][:4])
        read = got.cpu().double()
        near = (read - exact).abs() <= 2.0 ** -24 * exact.abs() + 2.0 ** -150
        assert bool((near | (read.isnan() & exact.isnan())).all())
        finite = torch.isfinite(rows_of.float().unflatten(-1, (-1, 64))).all(-1)
        assert torch.equal(exact.isnan().unflatten(-1, (-1, 64)).all(-1), ~finite)
        assert torch.equal(exact.isnan().unflatten(-1, (-1, 64)).any(-1), ~finite)


@pytest.mark.parametrize("dtype", TYPES)
def test_held_values_are_near(dtype):
    """Within half a step of what was written, a step being a fifteenth of the group's range, and the rounding of the
    scale: 15 steps of it, relative half a step of the type."""
    x = rows((200, 4, 128), dtype, 5)
    c = empty_cache([200], 32, 4, 128, dtype, layers=1)
    paro.paro_kv_append(c, 0, x.cuda(), x.cuda(), ints([0]), offsets([200]))
    k, v = torch.empty((200, 4, 128), device="cuda"), torch.empty((200, 4, 128), device="cuda")
    paro.paro_kv_read(c, 0, k, v, ints([0]), offsets([200]))
    g = x.unflatten(-1, (-1, 64)).double()
    span = (g.amax(-1) - g.amin(-1))[..., None]
    u = _kv4.HALF_STEP[dtype]
    for got in (k, v):
        off = (got.cpu().double().unflatten(-1, (-1, 64)) - g).abs()
        # half a step of the rounded scale, or past the fifteenth code where the scale was rounded down
        assert bool((off <= span / 30 * (1 + u) + span * u + 2.0 ** -23 * g.abs()).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page,kv_heads,dim", [(16, 2, 64), (32, 8, 128), (256, 1, 128)])
def test_read(dtype, page, kv_heads, dim):
    lengths = [70, 0, 1, 257, 16]
    c = _kv4.fill(paro, lengths, page, kv_heads, dim, dtype, page + dim, layers=2)
    held = [_kv4.held_rows(c, 1, s) for s in range(5)]
    for out in (dtype, torch.float32):
        u = _kv4.HALF_STEP[out] if out != torch.float32 else 0.0

        def check(got, want):
            limit = (u + 2.0 ** -23) * want.abs() + (2.0 ** -25 if out == torch.float16 else 0)
            assert bool(((got.cpu().double() - want).abs() <= limit).all())

        # everything, into views with other heads beside; rows outside the entries stay
        cu = offsets(lengths) + 1
        n = int(cu[-1]) + 2
        buf = torch.full((n, 2 * kv_heads + 1, dim), 7.0, dtype=out, device="cuda")
        k, v = buf[:, :kv_heads], buf[:, kv_heads + 1:]
        paro.paro_kv_read(c, 1, k, v, ints(range(5)), cu)
        for s in range(5):
            check(k[cu[s]:cu[s + 1]], held[s][0])
            check(v[cu[s]:cu[s + 1]], held[s][1])
        assert bool((buf[0] == 7).all()) and bool((buf[int(cu[-1]):] == 7).all()) and bool((buf[:, kv_heads] == 7).all())
        # the newest ones, one per slot, K or V alone, slots twice and foreign ones
        k = torch.full((6, kv_heads, dim), 7.0, dtype=out, device="cuda")
        v = k.clone()
        slots = [3, 0, 3, 1, -1, 5]
        paro.paro_kv_read(c, 1, k, None, ints(slots))
        paro.paro_kv_read(c, 1, None, v, ints(slots))
        for got, i in ((k, 0), (v, 1)):
            for r, s in enumerate(slots):
                check(got[r], held[s][i][-1] if s in (0, 3) else torch.zeros(kv_heads, dim))
        # from given positions on, past the ends
        first, counts, slots = [60, -3, 0, 250, 5, 2 ** 31 - 1], [20, 6, 3, 7, 0, 2], [0, 0, 2, 3, 3, 4]
        cu = offsets(counts)
        k, v = (torch.full((int(cu[-1]), kv_heads, dim), 7.0, dtype=out, device="cuda") for _ in range(2))
        paro.paro_kv_read(c, 1, k, v, ints(slots), cu, first=ints(first))
        for got, i in ((k, 0), (v, 1)):
            r = 0
            for f, m, s in zip(first, counts, slots):
                for p in range(f, f + m):
                    check(got[r], held[s][i][p] if 0 <= p < lengths[s] else torch.zeros(kv_heads, dim))
                    r += 1


@pytest.mark.parametrize("dtype", TYPES)
def test_read_of_a_16_bit_cache_copies(dtype):
    lengths = [70, 0, 33]
    c = filled_cache(paro, lengths, 16, 2, 64, dtype, 4, layers=2)
    c.k[1, int(c.table[0, 1]), 0, 3, 5] = float("nan")
    cu = offsets([75, 2, 33])
    k, v = (torch.empty((110, 2, 64), dtype=dtype, device="cuda") for _ in range(2))
    paro.paro_kv_read(c, 1, k, v, ints([0, 1, 2]), cu)
    wide = [torch.empty((110, 2, 64), device="cuda") for _ in range(2)]
    paro.paro_kv_read(c, 1, *wide, ints([0, 1, 2]), cu)
    from _attention import cached_rows
    for i, (got, w) in enumerate(zip((k, v), wide)):
        a, b = cached_rows(c, 1, 0)[i], cached_rows(c, 1, 2)[i]
        want = torch.cat([torch.zeros_like(a[:5]), a, torch.zeros_like(a[:2]), b])
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        assert torch.equal(w.view(torch.int32)[5:], want.float().view(torch.int32)[5:])


@pytest.mark.parametrize("dtype,dim", [(torch.float16, 64), (torch.bfloat16, 128)])
def test_page_calls_carry_the_bytes(dtype, dim):
    """Fork, copy on write, free and compaction: what each slot reads back is what was written to it."""
    rng, page, kv_heads = random.Random(dim), 16, 3
    c = paro.KVCache.empty(2, 40, kv_heads, page, dim, 6, 12, dtype, bits=4)
    for t in (c.k, c.v):
        t.fill_(0xFF)
    ws = paro.make_workspace(paro.paro_kv_workspace_bytes(c))
    held = {s: [torch.zeros((0, kv_heads, dim), dtype=dtype)] * 4 for s in range(6)}  # K, V of layer 0, of layer 1
    out = ints([0] * 6)

    def grow(counts, seed):
        slots = [s for s, n in counts.items() if n]
        paro.paro_kv_reserve(c, ints(slots), ints([counts[s] for s in slots]), out[:len(slots)], ws)
        assert out[:len(slots)].tolist() == [1] * len(slots)
        new = [counts[s] for s in slots]
        x = [rows((sum(new), kv_heads, dim), dtype, seed + i) for i in range(4)]
        for layer in range(2):
            paro.paro_kv_append(c, layer, x[2 * layer].cuda(), x[2 * layer + 1].cuda(), ints(slots), offsets(new))
        at = 0
        for s, n in zip(slots, new):
            held[s] = [torch.cat([a, b[at:at + n]]) for a, b in zip(held[s], x)]
            at += n

    def check():
        for s, want in held.items():
            n = want[0].shape[0]
            assert int(c.lengths[s]) == n
            if not n:
                continue
            for layer in range(2):
                k, v = (torch.empty((n, kv_heads, dim), device="cuda") for _ in range(2))
                paro.paro_kv_read(c, layer, k, v, ints([s]), offsets([n]))
                for got, x in ((k, want[2 * layer]), (v, want[2 * layer + 1])):
                    exact = _kv4.stands_for(*_kv4.quantise(x))
                    assert bool(((got.cpu().double() - exact).abs() <= 2.0 ** -24 * exact.abs()).all()), (s, layer)

    grow({0: 37, 2: 16, 4: 1}, 100)
    check()
    paro.paro_kv_fork(c, ints([0, 0, 2]), ints([1, 3, 5]), out[:3], ws)
    assert out[:3].tolist() == [1, 1, 1]
    held[1] = held[3] = held[0]
    held[5] = held[2]
    check()
    for i in range(6):
        grow({s: rng.choice([0, 1, 1, 2, 5]) for s in range(6)}, 200 + 10 * i)
    check()
    paro.paro_kv_free(c, ints([0, 4]))
    for s in (0, 4):
        held[s] = [torch.zeros((0, kv_heads, dim), dtype=dtype)] * 4
    used = ints([0])
    paro.paro_kv_compact(c, used, ws)
    assert int((c.refs > 0).sum()) == int(used) and not c.refs[int(used):].any()
    check()
    grow({0: 20, 1: 3, 4: 17}, 400)
    check()


def test_captured_writes_and_reads():
    """A graph of an append and a read, replayed with new rows, positions and eager work between."""
    c = empty_cache([64, 64, 64], 16, 2, 128, torch.bfloat16, layers=1)
    slots, cu = ints([2, 0]), offsets([1, 3])
    x = rows((4, 2, 128), torch.bfloat16, 0).cuda()
    y = x.clone()
    k, v = (torch.empty((4, 2, 128), device="cuda") for _ in range(2))
    paro.paro_kv_append(c, 0, x, y, slots, cu)  # (warm)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        paro.paro_kv_append(c, 0, x, y, slots, cu)
        paro.paro_kv_read(c, 0, k, v, slots, cu)
    for i in range(5):
        c.lengths.copy_(ints([20 + i, 9, 40 - 3 * i]))
        a, b = rows((4, 2, 128), torch.bfloat16, 10 + i), rows((4, 2, 128), torch.bfloat16, 20 + i)
        x.copy_(a)
        y.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        for got, want in ((k, a), (v, b)):
            exact = _kv4.stands_for(*_kv4.quantise(want))
            assert bool(((got.cpu().double() - exact).abs() <= 2.0 ** -24 * exact.abs()).all())
        held = _kv4.held_rows(c, 0, 0)[0][-3:]
        assert torch.equal(held, _kv4.stands_for(*_kv4.quantise(a))[1:])
