"""Decode attention over the cache in four bits where values' scales differ from key to key, from head to head and from
group to group: what a key adds counts by its weight, however large or small the others' scales are."""
import pytest

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")
import _kv4  # noqa: E402
import _kv4_bounds  # noqa: E402
from test_gpu_attention4 import TYPES, decode, ints, pairs_view, rows  # noqa: E402

pytestmark = pytest.mark.gpu

HEADS = [(1, 4), (1, 7), (2, 16), (1, 17)]  # key-value heads, query heads of each


def check(c, q, y, scale=None):
    assert bool(torch.isfinite(y).all())
    scale = _kv4.default_scale(q.shape[2]) if scale is None else scale
    for r in range(q.shape[0]):
        _kv4_bounds.check(y[r], q[r], *_kv4_bounds.held(c, 0, r), scale)


def at(c, slot, p):
    return int(c.table[slot, p // c.c.page_size]), p % c.c.page_size


def set_key(c, slot, p, low):
    """K of position p in all channels."""
    page, r = at(c, slot, p)
    kp = pairs_view(c, c.k)
    kp[0, page, :, r, :, 0] = 0.0
    kp[0, page, :, r, :, 1] = low


def grow_values(c, slot, p, exponent, group=slice(None)):
    page, r = at(c, slot, p)
    vp = pairs_view(c, c.v)
    vp[0, page, :, r, group] = (vp[0, page, :, r, group].float() * 2.0 ** exponent).to(c.dtype)


@pytest.mark.parametrize("kv_heads,group", HEADS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [100, 600, 5000])
def test_a_huge_scale_without_weight(n, dim, kv_heads, group):
    """One key has values 2^40 times the others' and no weight at all: first, late, last."""
    for p in (0, 1, 70, n // 2, n - 1):
        c = _kv4.fill(paro, [n], 16, kv_heads, dim, torch.bfloat16, 2)
        set_key(c, 0, p, -300.0)
        grow_values(c, 0, p, 40)
        q = rows((1, kv_heads * group, dim), torch.bfloat16, 4).abs()
        check(c, q, decode(c, q, ints([0])))


@pytest.mark.parametrize("kv_heads,group", HEADS)
@pytest.mark.parametrize("dim", [64, 128])
def test_a_huge_scale_with_the_weight_of_some_heads(dim, kv_heads, group):
    """Every other head puts all weight on the key with the huge scale, the others none."""
    for p in (0, 70, 599):
        c = _kv4.fill(paro, [600], 32, kv_heads, dim, torch.bfloat16, 2)
        set_key(c, 0, p, -300.0)
        grow_values(c, 0, p, 40)
        q = rows((1, kv_heads * group, dim), torch.bfloat16, 4).abs()
        q[:, ::2] *= -1
        check(c, q, decode(c, q, ints([0])))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [600, 5000])
def test_scales_before_the_scores_rise(dim, n):
    """The first keys of every wave have huge scales and are then left behind by later keys with far higher scores."""
    c = _kv4.fill(paro, [n], 16, 1, dim, torch.bfloat16, 2)
    for p in range(0, n, 16):
        if p // 128 % 2 == 0:
            set_key(c, 0, p, -3.0)
            grow_values(c, 0, p, 60)
    q = rows((1, 5, dim), torch.bfloat16, 4).abs() * 4.0
    check(c, q, decode(c, q, ints([0])))


@pytest.mark.parametrize("dtype", TYPES)
def test_one_group_of_channels_is_far_larger(dtype):
    """Channels 64 and up are 2^10 (fp16) or 2^50 (bf16) times the others: each group keeps its own precision."""
    c = _kv4.fill(paro, [300, 1], 16, 2, 128, dtype, 2, v_scale=1.0 if dtype == torch.bfloat16 else 2.0 ** -6)
    vp = pairs_view(c, c.v)
    vp[..., 1, :] = (vp[..., 1, :].float() * 2.0 ** (50 if dtype == torch.bfloat16 else 10)).to(dtype)
    q = rows((2, 6, 128), dtype, 4)
    check(c, q, decode(c, q, ints([0, 1])))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [600, 1000])
def test_constant_values_before_tiny_ones(dim, n):
    """The first keys' groups are constant (their scale is 0), the later ones' values are of size 2^-60."""
    for first in (1, 32, 128, 500):
        c = _kv4.fill(paro, [n], 16, 2, dim, torch.bfloat16, 2, v_scale=2.0 ** -60)
        vp = pairs_view(c, c.v)
        for p in range(first):
            page, r = at(c, 0, p)
            vp[0, page, :, r] = 0.0
        q = rows((1, 8, dim), torch.bfloat16, 4)
        check(c, q, decode(c, q, ints([0])))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,falling", [(400, False), (400, True), (3000, False), (3000, True)])
def test_scales_and_scores_against_each_other(dim, n, falling):
    """Scores go one way and scales the other, so that weight times scale stays alike over many orders of each."""
    c = _kv4.fill(paro, [n], 16, 1, dim, torch.bfloat16, 2)
    for p in range(n):
        level = p * 40 // n if falling else 40 - p * 40 // n
        set_key(c, 0, p, -level / 8.0)
        grow_values(c, 0, p, level)
    # a score falls by log 2 a level
    q = torch.full((1, 4, dim), 1.0, dtype=torch.bfloat16, device="cuda")
    check(c, q, decode(c, q, ints([0]), scale=0.6931471805599453 * 8 / dim), scale=0.6931471805599453 * 8 / dim)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 7, 8, 16, 17, 40])
def test_ordinary_values(group, dim, dtype):
    """Rows cut between workgroups, a workgroup for each output, a wave for each, one long row: within the bound that
    weights what each key can add."""
    for lengths, slots, kv_heads in (([3000, 700], [0, 1], 2), ([600, 33], [1, 0], 2), ([250, 128, 129, 33], [0, 1, 2, 3] * 200, 2),
                                     ([2600, 90, 300], [0] + [1, 2] * 150, 2), ([20011], [0], 1)):
        c = _kv4.fill(paro, lengths, 16, kv_heads, dim, dtype, group)
        q = rows((len(slots), kv_heads * group, dim), dtype, 5, 1.5)
        y = decode(c, q, ints(slots))
        for r in {0, 1, len(slots) // 2, len(slots) - 1} & set(range(len(slots))):
            _kv4_bounds.check(y[r], q[r], *_kv4_bounds.held(c, 0, slots[r]), _kv4.default_scale(dim))
