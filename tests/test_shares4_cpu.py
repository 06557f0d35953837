"""The checks of the four-bit decode tests notice what they are there for (no GPU): outputs that lack a key, count one
twice, lack a step, a part or everything are refused, the right ones are not."""
import pytest

torch = pytest.importorskip("torch")
import _kv4  # noqa: E402
import _kv4_bounds  # noqa: E402
import _shares as sh  # noqa: E402
import _shares4 as s4  # noqa: E402

TYPES = (torch.float16, torch.bfloat16)


class Outputs:
    """What a kernel gives that counts some keys more or less often than once: (1, kv_heads, dim)."""

    def __init__(self, lev, v, dtype):
        self.w, self.dtype = 2.0 ** lev.double(), dtype
        self.terms = self.w[:, None, None] * v.double()
        self.sums = self.terms.sum(0), self.w.sum()

    def __call__(self, keys=slice(0, 0), more=0):
        y = (self.sums[0] + more * self.terms[keys].sum(0)) / (self.sums[1] + more * self.w[keys].sum())
        return y.to(self.dtype)[None]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pattern", sh.PATTERNS)
@pytest.mark.parametrize("n,dim,centred", [(33, 64, True), (513, 128, True), (1100, 64, False), (3000, 128, True),
                                           (20011, 128, True)])
def test_a_lost_or_doubled_key_is_noticed(n, dim, centred, pattern, dtype):
    lev = sh.levels(n, pattern, n)
    total, noticed = torch.zeros(n, dtype=torch.long), set()
    for which in range(sh.windows(n, dim)):
        _, _, v = s4.rows_of(lev, 1, dim, which, centred=centred)
        seen = (v > 0).any(-1)[:, 0]
        total += seen
        out, right = Outputs(lev, v, dtype), s4.expected(lev, v, 1, dtype, centred)
        assert not s4.wrong(out(), *right).any()
        assert s4.wrong(torch.zeros_like(out()), *right).any()
        keys = torch.nonzero(seen).flatten().tolist()
        for j in {keys[0], keys[-1], keys[len(keys) // 2], keys[len(keys) // 3]}:
            for more in (-1, 1):
                assert s4.wrong(out([j], more), *right).any(), (j, more)
        for length in (32, 128, 384):  # a wave's step, a workgroup's, a part
            for first in range(0, n, max(length, n // 5 // length * length)):
                # (a window's own keys may lack as much as the sum of the weights does: 3 of a channel's 16 beside one of
                # 4096 in 24106; another window's do not)
                if length < n and s4.wrong(out(slice(first, first + length), -1), *right).any():
                    noticed.add((length, first))
    assert bool((total == 1).all())  # one head's windows cover every key once
    assert noticed == {(length, first) for length in (32, 128, 384) if length < n
                       for first in range(0, n, max(length, n // 5 // length * length))}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [600, 3000, 20011])
def test_the_bound_of_random_rows_refuses_lost_shares(n, dtype):
    g = torch.Generator().manual_seed(n)
    k, v = (_kv4.quantise(torch.randn((n, 1, 128), generator=g).to(dtype)) for _ in range(2))
    q = torch.randn((4, 128), generator=g).to(dtype)
    held = [(x[0].double(), x[1].double(), x[2].double()) for x in (k, v)]
    y, limit = _kv4_bounds.attention(q, *held, _kv4.default_scale(128))
    assert not _kv4_bounds.wrong(y.to(dtype), y, limit).any()
    assert _kv4_bounds.wrong(torch.zeros_like(y), y, limit).any()
    assert _kv4_bounds.wrong(_kv4.stands_for(*v)[:, 0].mean(0).expand_as(y), y, limit).any()
    assert _kv4_bounds.wrong(_kv4_bounds.attention(q, *held, 0.9 * _kv4.default_scale(128))[0], y, limit).any()
    for kept in (slice(0, n // 2), slice(n // 2, n), slice(384, n), slice(0, n - 384)):
        less = [tuple(x[kept] for x in t) for t in held]
        assert _kv4_bounds.wrong(_kv4_bounds.attention(q, *less, _kv4.default_scale(128))[0], y, limit).any(), kept


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_what_the_pages_hold(sign, dtype):
    """The bytes stand for the levels and values, whichever way they are written."""
    lev = sh.levels(50, "blocks", 3)
    for dim, centred in ((64, True), (128, False)):
        (kc, kp), (vc, vp), v = s4.rows_of(lev, 2, dim, 0, sign, centred)
        k = _kv4.values_of(s4.pages(kc, kp, 16, dtype, True), dtype, True).transpose(1, 2).flatten(0, 1)
        assert torch.equal(k[:50, :, 0], (sign * lev.double())[:, None].expand(50, 2)) and bool(k[50:].isnan().all())
        got = _kv4.values_of(s4.pages(vc, vp, 16, dtype, False), dtype, False).transpose(1, 2).flatten(0, 1)
        assert torch.equal(got[:50], v.double())


def test_forms():
    assert s4.form([777], 32, 8, 1024) == ("cut", False) and s4.form([500], 32, 8, 1024) == ("output", False)
    assert s4.form([100] * 300, 32, 8, 128) == ("wave", True) and s4.form([9] * 4097, 2, 1, 16) == ("rows", True)
    assert s4.form([3000] + [90] * 299, 32, 8, 4096) == ("cut", True)
