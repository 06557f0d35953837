"""The check of _shares.py on the host: right outputs pass, and each kind of mistake that a kernel could make with its
keys (planted here in the definition) does not."""
import pytest

torch = pytest.importorskip("torch")

import _shares as sh  # noqa: E402

LENGTHS = [33, 384, 777, 9001]


def outputs(lev, v, n_q, dtype, group, counts):
    """What a kernel that counts key j of row i counts[i, j] times would give."""
    w = (2.0 ** lev.double())[None] * counts
    y = torch.einsum("ij,jhd->ihd", w, v.double()) / w.sum(1)[:, None, None]
    return y.repeat_interleave(group, 1).to(dtype)


def seen_by(n, n_q):
    return (torch.arange(n)[None] <= torch.arange(n_q)[:, None] + n - n_q).double()


def passes(got, lev, v):
    try:
        sh.check(got, lev, v)
    except AssertionError:
        return False
    return True


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("pattern", sh.PATTERNS)
def test_every_lost_doubled_or_foreign_key_is_noticed(pattern, dtype):
    dim, kv_heads, group = 64, 2, 3
    for n in LENGTHS:
        lev = sh.levels(n, pattern, n)
        n_q = min(n, 3)
        values = [sh.keys_and_values(lev, kv_heads, dim, p)[1] for p in range(sh.windows(n, dim))]
        clean = seen_by(n, n_q)
        assert all(passes(outputs(lev, v, n_q, dtype, group, clean), lev, v) for v in values)
        # one key, at every kind of edge, and runs of keys: a step, a tile, a page, a part
        runs = [(j, j + 1) for j in sorted({0, 1, 15, 16, 31, 32, n // 2, n - 4, n - 3, n - 1} & set(range(n)))]
        runs += [(a, min(n, a + m)) for m in (16, 32, 64, 128, 256) for a in (0, n // 2) if n > m + a]
        for a, b in runs:
            for times in (0.0, 2.0):
                counts = clean.clone()
                counts[:, a:b] *= times
                if float(counts.sum(1).min()) == 0:
                    continue
                assert not all(passes(outputs(lev, v, n_q, dtype, group, counts), lev, v) for v in values), (n, a, times)
        if n_q > 1:  # a key that the first row may not see
            counts = clean.clone()
            counts[0, n - n_q + 1] = 1.0
            assert not all(passes(outputs(lev, v, n_q, dtype, group, counts), lev, v) for v in values), n


def test_a_shifted_value_row_is_noticed():
    """Weights of one key with the values of its neighbour, within a block of equal levels too."""
    for pattern in ("flat", "rising", "blocks"):
        lev = sh.levels(500, pattern, 1)
        v = sh.keys_and_values(lev, 1, 64, 0)[1]
        moved = v.clone()
        moved[200:232] = v[201:233]
        got = outputs(lev, moved, 1, torch.bfloat16, 1, torch.ones(1, 500, dtype=torch.float64))
        assert not passes(got, lev, v)


@pytest.mark.parametrize("n,kv_heads,dim", [(1, 1, 64), (9001, 2, 64), (5000, 1, 128)])
def test_windows_cover_every_key_once(n, kv_heads, dim):
    lev = sh.levels(n, "blocks", 3)
    hits = sum((sh.keys_and_values(lev, kv_heads, dim, p)[1] != 0).sum((1, 2)) for p in range(sh.windows(n, dim)))
    assert bool((hits == kv_heads).all())
