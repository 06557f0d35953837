"""The cache's pages through the C-ABI against a plain model on the host:
reserve (copy on write), fork, free, compact and append, one by one and in
random chains, with repeated, foreign and refused entries."""
import random

import pytest

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")

pytestmark = pytest.mark.gpu


class Model:
    """The documented rules, one entry and one page at a time; data: {(page): stamp} as a tensor per page."""

    def __init__(self, pages, page, slots, max_pages, layers=1):
        self.page, self.max_pages = page, max_pages
        self.refs = [0] * pages
        self.table = [[-1] * max_pages for _ in range(slots)]
        self.lengths = [0] * slots

    def held(self, n):
        return -(-n // self.page)

    def reserve(self, slots, grow):
        """Returns granted and the (source, target) copies."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        before = list(self.refs)
        seen, total, granted, copies = set(), 0, [], []
        for s, g in zip(slots, grow):
            if not 0 <= s < len(self.lengths) or s in seen:
                granted.append(0)
                continue
            seen.add(s)
            n = self.lengths[s]
            if g < 0 or n + g > self.max_pages * self.page:
                granted.append(0)
                continue
            have = self.held(n)
            last = self.table[s][have - 1] if n % self.page else -1
            cow = g > 0 and last >= 0 and before[last] > 1
            need = self.held(n + g) - have + cow
            total += need
            if need and total > len(free):
                granted.append(0)
                continue
            granted.append(1)
            mine = free[total - need:total]
            if cow:
                copies.append((last, mine[0]))
                self.refs[last] -= 1
            for i, p in enumerate(mine):
                self.table[s][have - cow + i] = p
                self.refs[p] = 1
            self.lengths[s] = n + g
        return granted, copies

    def fork(self, parents, children):
        lengths = list(self.lengths)
        seen, granted = set(), []
        for a, c in zip(parents, children):
            first = c not in seen
            seen.add(c)
            good = all(0 <= x < len(lengths) for x in (a, c)) and a != c and first and lengths[c] == 0
            granted.append(int(good))
            if good:
                self.lengths[c] = lengths[a]
                for j in range(self.held(lengths[a])):
                    self.table[c][j] = self.table[a][j]
                    self.refs[self.table[a][j]] += 1
        return granted

    def free(self, slots):
        for s in set(slots):
            if 0 <= s < len(self.lengths):
                for j in range(self.held(self.lengths[s])):
                    self.refs[self.table[s][j]] -= 1
                    self.table[s][j] = -1
                self.lengths[s] = 0

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        holes = [p for p in range(used) if self.refs[p] == 0]
        moves = list(zip([p for p in range(used, len(self.refs)) if self.refs[p] > 0], holes))
        to = dict(moves)
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return used, moves


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Pair:
    """A cache and its model, moved together."""

    def __init__(self, pages, page, slots, max_pages, layers=1, kv_heads=2, dim=64, dtype=torch.float16):
        self.m = Model(pages, page, slots, max_pages)
        self.c = paro.KVCache.empty(layers, pages, kv_heads, page, dim, slots, max_pages, dtype)
        g = torch.Generator(device="cuda").manual_seed(pages)
        self.c.k.copy_(torch.randn(self.c.k.shape, device="cuda", generator=g))
        self.c.v.copy_(torch.randn(self.c.v.shape, device="cuda", generator=g))
        self.k, self.v = self.c.k.clone(), self.c.v.clone()
        self.ws = torch.randint(0, 255, (paro.paro_kv_workspace_bytes(self.c),), dtype=torch.uint8, device="cuda")

    def copies(self, moves):
        if moves:
            a, b = (torch.tensor(x, device="cuda") for x in zip(*moves))
            self.k[:, b], self.v[:, b] = self.k[:, a], self.v[:, a]

    def reserve(self, slots, grow):
        got = torch.full((len(slots),), 77, dtype=torch.int32, device="cuda")
        paro.paro_kv_reserve(self.c, ints(slots), ints(grow), got, self.ws)
        granted, moves = self.m.reserve(slots, grow)
        self.copies(moves)
        assert got.tolist() == granted
        self.same()
        return granted

    def fork(self, parents, children):
        got = torch.full((len(parents),), 77, dtype=torch.int32, device="cuda")
        paro.paro_kv_fork(self.c, ints(parents), ints(children), got, self.ws)
        granted = self.m.fork(parents, children)
        assert got.tolist() == granted
        self.same()
        return granted

    def free(self, slots):
        paro.paro_kv_free(self.c, ints(slots))
        self.m.free(slots)
        self.same()

    def compact(self):
        used = ints([-1])
        paro.paro_kv_compact(self.c, used, self.ws)
        n, moves = self.m.compact()
        self.copies(moves)
        assert used.tolist() == [n]
        self.same()

    def same(self):
        assert self.c.refs.tolist() == self.m.refs
        assert self.c.lengths.tolist() == self.m.lengths
        assert self.c.table.tolist() == self.m.table
        assert torch.equal(self.c.k, self.k) and torch.equal(self.c.v, self.v)


def test_reserve_grows_in_order_and_refuses():
    p = Pair(20, 16, 6, 8)
    assert p.reserve([0, 1, 2], [1, 16, 17]) == [1, 1, 1]
    assert p.reserve([2, 0, 2, -1, 6, 1, 3], [15, 0, 5, 3, 3, -2, 129]) == [1, 1, 0, 0, 0, 0, 0]
    assert p.reserve([0], [15]) == [1]  # fills its page: no new one
    # 20 - 1 - 1 - 2 = 16 pages are free, and 8 + 7 + 1 are asked for
    assert p.reserve([3, 4, 5, 0], [128, 112, 1, 0]) == [1, 1, 1, 1]
    # none is left: who needs none is still granted
    assert p.reserve([5, 0, 1], [1, 1, 0]) == [1, 0, 1]
    assert p.reserve([5], [15]) == [0]
    p.free([4, 4, 9, -3])
    assert p.reserve([5, 5], [15, 1]) == [1, 0]


def test_fork_shares_and_reserve_copies_on_write():
    p = Pair(40, 16, 8, 6, layers=3, kv_heads=3, dim=128, dtype=torch.bfloat16)
    p.reserve([0, 1], [37, 32])
    assert p.fork([0, 0, 1, 0, 0, 7, 2], [2, 3, 4, 2, 0, 5, 6]) == [1, 1, 1, 0, 0, 1, 1]
    # 0, 2 and 3 share a page that is not full: each that grows gets a copy; 1 and 4 end at a page's end
    assert p.reserve([2, 4, 1], [1, 3, 1]) == [1, 1, 1]
    assert p.reserve([0, 3], [1, 1]) == [1, 1]
    p.free([0, 2])
    p.free([1, 3, 4])
    assert sum(p.m.refs) == 0


def test_fork_of_a_child_of_the_same_call_and_of_taken_slots():
    p = Pair(10, 16, 5, 4)
    p.reserve([0], [20])
    assert p.fork([0, 1, 3], [1, 2, 0]) == [1, 1, 0]
    assert p.m.lengths == [20, 20, 0, 0, 0]


def test_all_holders_copy_and_the_page_is_free_again():
    p = Pair(9, 32, 4, 2)
    p.reserve([0], [40])
    p.fork([0, 0], [1, 2])
    assert p.reserve([0, 1, 2], [1, 1, 1]) == [1, 1, 1]
    assert p.m.refs[1] == 0


def test_copy_on_write_refused_when_no_page_is_left():
    p = Pair(2, 16, 3, 4)
    p.reserve([0], [20])
    p.fork([0], [1])
    assert p.reserve([1, 0], [1, 1]) == [0, 0]
    p.free([0])
    assert p.reserve([1], [1]) == [1]


@pytest.mark.parametrize("pages,slots", [(3, 2), (64, 64), (1000, 40), (17000, 300)])
def test_compact(pages, slots):
    rng = random.Random(pages)
    p = Pair(pages, 16, slots, max(2, 2 * pages // slots), kv_heads=1)
    p.compact()
    for _ in range(3):
        p.reserve(list(range(slots)), [rng.randint(0, 16 * max(1, pages // slots)) for _ in range(slots)])
        p.free(rng.sample(range(slots), slots // 2 + 1))
    held = [s for s in range(slots) if p.m.lengths[s]]
    empty = [s for s in range(slots) if not p.m.lengths[s]]
    p.fork([rng.choice(held) if held else 0 for _ in empty[:5]], empty[:5])
    p.compact()
    p.compact()  # nothing left to move


def test_scan_finds_the_last_pages():
    """Free pages lie behind several steps of the page scan."""
    p = Pair(40000, 16, 4, 40000, kv_heads=1)
    p.reserve([0], [16 * 39990])
    assert p.reserve([1, 2], [16 * 9, 17]) == [1, 0]
    assert p.reserve([3], [1]) == [1]
    p.free([0])
    p.compact()


def test_many_slots():
    p = Pair(5000, 16, 4096, 4, kv_heads=1)
    rng = random.Random(1)
    order = rng.sample(range(4096), 4096)
    p.reserve(order, [rng.randint(0, 40) for _ in order])
    p.free(order[:2000])
    full = [s for s in range(4096) if p.m.lengths[s]]
    empty = [s for s in range(4096) if not p.m.lengths[s]]
    p.fork([rng.choice(full) for _ in empty], empty)
    p.reserve(rng.sample(range(4096), 4096), [rng.randint(0, 5) for _ in range(4096)])


@pytest.mark.parametrize("seed", range(4))
def test_random_chains(seed):
    rng = random.Random(seed)
    slots, pages = rng.randint(3, 12), rng.randint(10, 60)
    p = Pair(pages, rng.choice([16, 32]), slots, rng.randint(2, 8), layers=rng.randint(1, 2))
    for _ in range(25):
        what, n = rng.choice(["reserve", "reserve", "fork", "free", "compact"]), rng.randint(1, slots)
        ids = [rng.randint(-1, slots) for _ in range(n)]
        if what == "reserve":
            p.reserve(ids, [rng.randint(-1, 40) for _ in ids])
        elif what == "fork":
            p.fork(ids, [rng.randint(0, slots - 1) for _ in ids])
        elif what == "free":
            p.free(ids[:2])
        else:
            p.compact()


# ---- append ----

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("page,kv_heads,dim", [(16, 8, 128), (32, 1, 64), (256, 3, 128), (64, 5, 64)])
def test_append(page, kv_heads, dim, dtype):
    p = Pair(120, page, 7, 30, layers=2, kv_heads=kv_heads, dim=dim, dtype=dtype)
    p.reserve([0, 1, 2, 4], [3, 100, 16, 200])
    p.reserve([4, 1, 3], [9, 70, 1])
    counts, slots = [9, 70, 0, 1], [4, 1, 2, 3]
    cu = torch.tensor([0, 9, 79, 79, 80], dtype=torch.int64, device="cuda")
    rows = torch.randn((80, 2 * kv_heads, dim), device="cuda").to(dtype)
    k, v = rows[:, :kv_heads], rows[:, kv_heads:]  # strided
    paro.paro_kv_append(p.c, 1, k, v, ints(slots), cu)
    r = 0
    for s, n in zip(slots, counts):
        for i in range(n):
            pos = p.m.lengths[s] - n + i
            where = p.m.table[s][pos // page]
            p.k[1, where, :, pos % page], p.v[1, where, :, pos % page] = k[r], v[r]
            r += 1
    p.same()
    # one row each, without offsets; repeated, foreign and empty slots are skipped
    k, v = (torch.randn((6, kv_heads, dim), device="cuda").to(dtype) for _ in range(2))
    slots = [3, 0, 3, -1, 7, 5]
    paro.paro_kv_append(p.c, 0, k, v, ints(slots))
    for r in (0, 1):
        pos = p.m.lengths[slots[r]] - 1
        where = p.m.table[slots[r]][pos // page]
        p.k[0, where, :, pos % page], p.v[0, where, :, pos % page] = k[r], v[r]
    p.same()


def test_append_skips_what_reserve_refused():
    """Three slots, two of which share a page, and one free page left: the refused entries' rows go nowhere."""
    c = paro.KVCache.empty(1, 3, 1, 16, 64, 4, 4, torch.float16)
    ws = torch.empty(paro.paro_kv_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    got = ints([-1, -1, -1])
    paro.paro_kv_reserve(c, ints([0, 2]), ints([10, 16]), got[:2], ws)
    paro.paro_kv_fork(c, ints([0]), ints([1]), got[:1], ws)
    c.k.normal_()
    c.v.normal_()
    k0, v0 = c.k.clone(), c.v.clone()
    rows = torch.randn((5, 1, 64), device="cuda").half()
    # slot 2 takes the last free page; slot 0's copy and slot 9 are refused
    slots, cu = ints([2, 0, 9]), torch.tensor([0, 2, 4, 5], dtype=torch.int64, device="cuda")
    paro.paro_kv_reserve(c, slots, ints([2, 2, 1]), got, ws)
    paro.paro_kv_append(c, 0, rows, -rows, slots, cu, granted=got)
    assert got.tolist() == [1, 0, 0] and c.lengths.tolist() == [10, 10, 18, 0]
    page = int(c.table[2, 1])
    assert torch.equal(c.k[0, page, 0, :2], rows[:2, 0]) and torch.equal(c.v[0, page, 0, :2], -rows[:2, 0])
    k0[0, page, 0, :2], v0[0, page, 0, :2] = rows[:2, 0], -rows[:2, 0]
    assert torch.equal(c.k, k0) and torch.equal(c.v, v0)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 300, 4096])
def test_append_finds_its_sequence(n):
    """Offsets with many empty sequences: each row lands in its own slot."""
    rng = random.Random(n)
    p = Pair(4500, 16, n, 2, kv_heads=1)
    counts = [rng.choice([0, 0, 1, 2]) for _ in range(n)]
    counts[-1] = 3
    p.reserve(list(range(n)), counts)
    cu = [0]
    for x in counts:
        cu.append(cu[-1] + x)
    order = list(range(n))
    k, v = (torch.randn((cu[-1], 1, 64), device="cuda").half() for _ in range(2))
    paro.paro_kv_append(p.c, 0, k, v, ints(order), torch.tensor(cu, dtype=torch.int64, device="cuda"))
    where = torch.tensor([p.m.table[s][0] for s in range(n) for _ in range(counts[s])], device="cuda")
    at = torch.tensor([i for s in range(n) for i in range(counts[s])], device="cuda")
    p.k[0, where, :, at], p.v[0, where, :, at] = k, v
    p.same()


@pytest.mark.parametrize("cu", [[-7, 3, 2, 50], [5, 0, 20], [0, 100, 100], [9, 9, 9], [-50, -40, 0]])
def test_append_malformed_offsets_stay_in_bounds(cu):
    p = Pair(12, 16, 3, 3)
    p.reserve([0, 1, 2], [20, 5, 33])
    held = set(x for row in p.m.table for x in row if x >= 0)
    k = torch.ones((12, 2, 64), dtype=torch.float16, device="cuda")
    paro.paro_kv_append(p.c, 0, k, k, ints([0, 1, 2][:len(cu) - 1]),
                        torch.tensor(cu, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    free = [x for x in range(12) if x not in held]
    assert torch.equal(p.c.k[:, free], p.k[:, free]) and p.c.table.tolist() == p.m.table


def test_offsets_past_32_bits():
    """A pool of over 4 GiB elements for K: the last pages are written, copied and moved."""
    pages = 36000
    c = paro.KVCache(torch.empty((2, pages, 8, 64, 128), dtype=torch.float16, device="cuda"),
                     torch.empty((2, pages, 8, 64, 128), dtype=torch.float16, device="cuda"),
                     torch.zeros(pages, dtype=torch.int32, device="cuda"),
                     torch.full((2, pages), -1, dtype=torch.int32, device="cuda"),
                     torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert c.k.numel() > 2 ** 32
    c.table[0, 0], c.refs[pages - 1] = pages - 1, 1
    c.lengths[0] = 5
    rows = torch.randn((2, 5, 8, 128), device="cuda").half()
    cu = torch.tensor([0, 5], dtype=torch.int64, device="cuda")
    for layer in range(2):
        paro.paro_kv_append(c, layer, rows[layer], -rows[layer], ints([0]), cu)
    for _ in range(2):
        for layer in range(2):
            page = int(c.table[0, 0])
            assert torch.equal(c.k[layer, page, :, :5].transpose(0, 1), rows[layer])
            assert torch.equal(c.v[layer, page, :, :5].transpose(0, 1), -rows[layer])
            q = torch.randn((1, 8, 128), device="cuda").half()
            y = torch.empty_like(q)
            paro.paro_attention_decode(c, layer, q, ints([0]), y, paro.make_workspace(
                paro.paro_attention_decode_workspace_bytes(c, 1, 8)))
            z = torch.empty_like(q)
            paro.paro_attention_prompt_cached(c, layer, q, ints([0]), torch.tensor([0, 1], device="cuda"), z)
            s = (q[0].double()[:, None] * rows[layer].double().transpose(0, 1)).sum(-1) / 128 ** 0.5
            want = -(torch.softmax(s, -1)[:, :, None] * rows[layer].double().transpose(0, 1)).sum(1)
            vmax = float(rows.abs().max())
            for got in (y, z):
                # weights and output in half steps of fp16 (2^-11), as in the attention tests' bound
                assert float((got[0].double() - want).abs().max()) <= 4 * 2.0 ** -11 * vmax
        used = ints([0])
        paro.paro_kv_compact(c, used, torch.empty(paro.paro_kv_workspace_bytes(c), dtype=torch.uint8, device="cuda"))
        assert used.tolist() == [1] and int(c.table[0, 0]) == 0


def test_most_pages_and_slots():
    """2^22 pages over 4096 slots: the last free ones are found, and 2048 holes are filled from the end."""
    pages, slots, width = 1 << 22, 4096, 1024
    c = paro.KVCache.empty(1, pages, 1, 16, 64, slots, width, torch.float16)
    index = torch.arange(pages, dtype=torch.int32, device="cuda")
    for x, salt in ((c.k, 0), (c.v, 1)):  # page p's first four bytes say p
        x.view(torch.int32)[0, :, 0, 0, 0] = index ^ salt
    c.table.copy_(index.view(slots, width))
    c.table[-1, -5:] = -1
    c.refs.fill_(1)
    c.refs[-5:] = 0
    c.lengths.fill_(width * 16)
    c.lengths[-1] = (width - 5) * 16 - 3
    ws = torch.empty(paro.paro_kv_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    got = ints([-1] * 3)
    paro.paro_kv_reserve(c, ints([0, slots - 1, 5]), ints([1, 3 + 33, 0]), got, ws)  # slot 0 is full
    assert got.tolist() == [0, 1, 1] and c.table[-1, -6:].tolist() == [pages - 6, pages - 5, pages - 4, pages - 3, -1, -1]
    assert c.refs[-5:].tolist() == [1, 1, 1, 0, 0]
    paro.paro_kv_free(c, ints([0, 7, 0]))
    used = ints([0])
    paro.paro_kv_compact(c, used, ws)
    n = pages - 2 - 2 * width
    assert used.tolist() == [n] and bool((c.refs[:n] == 1).all()) and not c.refs[n:].any()
    want = index.view(slots, width).clone()
    want[-1, -2:] = -1
    holes = torch.cat([torch.arange(width), 7 * width + torch.arange(width)]).int().cuda()
    moving = want >= n  # in ascending order, as the table is
    want[moving] = holes
    want[0] = want[7] = -1
    assert torch.equal(c.table, want)
    stamp = index[:n].clone()
    stamp[holes.long()] = torch.arange(n, n + 2 * width, dtype=torch.int32, device="cuda")
    for x, salt in ((c.k, 0), (c.v, 1)):
        assert torch.equal(x.view(torch.int32)[0, :n, 0, 0, 0], stamp ^ salt)
