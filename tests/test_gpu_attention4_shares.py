"""Decode attention over the cache in four bits counts every key once, in every form of its kernel: outputs cut between
workgroups and joined, a workgroup for each, a wave for each, more rows than are looked up; one and several tiles of 1 to
16 heads; the inputs of _shares4.py."""
import pytest

import _shares as sh
import _shares4 as s4

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]
GROUPS = [1, 4, 7, 8, 16, 17, 40]


def cache(lengths, page, kv_heads, dim, dtype, extra=2):
    """A cache whose slots have room for `lengths`, in pages of random order; 0xFF everywhere."""
    counts = [-(-n // page) for n in lengths]
    c = paro.KVCache.empty(1, sum(counts) + 3, kv_heads, page, dim, len(lengths), max(counts) + extra, dtype, bits=4)
    c.k.fill_(0xFF)
    c.v.fill_(0xFF)
    order, at = torch.randperm(sum(counts) + 3, generator=torch.Generator().manual_seed(page)).int().cuda(), 0
    for i, m in enumerate(counts):
        c.table[i, :m] = order[at:at + m]
        c.refs[order[at:at + m].long()] = 1
        at += m
    c.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
    return c


def decode(lengths, slots, heads, kv_heads, dim, page, dtype, pattern, form, many, centred=True, sign=1.0, passes=None):
    c = cache(lengths, page, kv_heads, dim, dtype)
    mine = [lengths[s] if s >= 0 else 0 for s in slots]
    assert s4.form(mine, heads, kv_heads, c.c.max_pages * page) == (form, many)
    levs = [sh.levels(n, pattern, n + i) for i, n in enumerate(lengths)]
    rows = len(slots)
    q = sh.queries(rows, heads, dim, dtype, "cuda")
    at = torch.tensor(slots, dtype=torch.int32, device="cuda")
    ws = paro.make_workspace(paro.paro_attention_decode_workspace_bytes(c, rows, heads))
    for p in range(passes or sh.windows(max(lengths), dim)):
        values = []
        for s, lev in enumerate(levs):
            n = lengths[s]
            (kc, kp), (vc, vp), v = s4.rows_of(lev, kv_heads, dim, p, sign, centred, "cuda")
            if n:
                where = c.table[s, :-(-n // page)].long()
                c.k[0, where] = s4.pages(kc, kp, page, dtype, True)
                c.v[0, where] = s4.pages(vc, vp, page, dtype, False)
            values.append(v)
        y = torch.full_like(q, float("nan"))
        paro.paro_attention_decode(c, 0, q, at, y, ws, scale=sign * sh.LOG2)
        for s, lev in enumerate(levs):
            got = y[at == s]
            if lengths[s] == 0:
                assert bool((got == 0).all())
            elif got.shape[0]:
                s4.check(got, lev, values[s], centred)
        assert bool((y[at < 0] == 0).all())
    torch.cuda.synchronize()
    assert not ws[:1 << 21].any()  # the counters are left zero


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", GROUPS)
def test_cut_outputs(group, dim, dtype):
    """Few rows: outputs are cut between workgroups and their parts joined."""
    for pattern in ("blocks", "rising", "falling", "first", "last"):
        decode([3000, 1, 1100], [1, 0, 2], 2 * group, 2, dim, 16, dtype, pattern, "cut", False)
    decode([2500], [0], group, 1, dim, 64, dtype, "blocks", "cut", False, sign=-1.0)
    decode([1800], [0], group, 1, dim, 256, dtype, "blocks", "cut", False, centred=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv_heads,dim", [(32, 8, 128), (16, 1, 128), (40, 1, 64), (4, 1, 128)])
def test_a_long_row_alone(heads, kv_heads, dim, dtype):
    """Up to 512 parts of an output."""
    for n in (9000, 33000, 70001):
        decode([n], [0], heads, kv_heads, dim, 64, dtype, "blocks", "cut", False, passes=3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", GROUPS)
def test_a_workgroup_for_each_output(group, dim, dtype):
    for pattern in ("blocks", "rising", "falling", "first", "last"):
        decode([640, 513, 512, 129, 1, 0], [3, 0, 1, -1, 4, 2, 5], 2 * group, 2, dim, 32, dtype, pattern, "output", False)
    decode([600, 30], [0, 1], 2 * group, 2, dim, 16, dtype, "blocks", "output", False, sign=-1.0)
    decode([600, 30], [0, 1], 2 * group, 2, dim, 16, dtype, "blocks", "output", False, centred=False)


SHORT = [250, 128, 129, 200, 33, 1, 97, 0]  # their rows are dealt out to waves
UNEVEN = [2900, 128, 40, 300, 1, 0, 77, 513]  # one row is far the longest


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", GROUPS)
def test_a_wave_for_each_output(group, dim, dtype):
    slots = [(5 * i + 1) % 9 - 1 for i in range(900)]
    for pattern in ("blocks", "rising", "last"):
        decode(SHORT, slots, 2 * group, 2, dim, 16, dtype, pattern, "wave", True)
    decode(SHORT, slots, 2 * group, 2, dim, 64, dtype, "falling", "wave", True, sign=-1.0)
    decode(SHORT, slots, 2 * group, 2, dim, 16, dtype, "blocks", "wave", True, centred=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", GROUPS)
def test_many_outputs_cut(group, dim, dtype):
    """More outputs than workgroups with one row far the longest: cut, in the kernel for many outputs."""
    slots = [0 if i in (7, 130) else (5 * i + 1) % 8 or 1 for i in range(300)]
    for pattern in ("blocks", "rising", "last"):
        decode(UNEVEN, slots, 2 * group, 2, dim, 16, dtype, pattern, "cut", True)
    decode(UNEVEN, slots, 2 * group, 2, dim, 64, dtype, "falling", "cut", True, sign=-1.0, passes=1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,group", [(64, 1), (128, 4), (128, 7), (128, 17), (64, 16)])
def test_more_rows_than_are_looked_up(dim, group, dtype):
    slots = [(5 * i + 1) % 9 - 1 for i in range(4097)]
    decode(SHORT, slots, group, 1, dim, 16, dtype, "blocks", "rows", True)


@pytest.mark.parametrize("dtype", TYPES)
def test_shapes_of_a_model(dtype):
    """32 query heads over 8 of 128 channels: rows that are cut, whole, dealt to waves."""
    decode([777], [0], 32, 8, 128, 16, dtype, "blocks", "cut", False)
    decode([512, 400, 33], [0, 1, 2] * 10, 32, 8, 128, 16, dtype, "blocks", "output", False)
    decode([4096, 2000, 700, 90], [0, 1, 2, 3] * 8, 32, 8, 128, 16, dtype, "blocks", "cut", False, passes=2)
    decode([300, 200, 90, 12], [0, 1, 2, 3] * 75, 32, 8, 128, 16, dtype, "blocks", "wave", True)
    decode([1000, 200, 90, 700], [0, 1, 2, 3] * 75, 32, 8, 128, 16, dtype, "blocks", "cut", True)
