"""Outputs that are views apart of one buffer: rows or heads in turn with the inputs, or with each other."""
import pytest

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")
from test_gpu_rotary import TYPES, check, frequencies, ints, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_between_views_of_one_buffer(dtype, interleaved):
    """Heads beside each other in a row, heads in turn, rows in turn; what lies between keeps its bytes."""
    n, dim, rot = 131, 64, 48
    f, pos = frequencies(rot), ints(n, 1)
    whole = randn((n, 10, dim), dtype, 1)
    turns = randn((n, 5, 2, dim), dtype, 2)
    rows = randn((n, 2, 5, dim), dtype, 3)
    for t, x, y in ((whole, lambda t: t[:, 1:5], lambda t: t[:, 5:9]), (whole, lambda t: t[:, 6:10], lambda t: t[:, 1:5]),
                    (turns, lambda t: t[:, :, 0], lambda t: t[:, :, 1]), (rows, lambda t: t[:, 1], lambda t: t[:, 0])):
        t, before = t.clone(), t.clone()
        paro.paro_rotary(x(t), pos, f, y(t), interleaved=interleaved)
        check(y(t), x(before), pos, f, interleaved)
        y(before).copy_(y(t))
        assert torch.equal(t, before)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_read_into_heads_and_rows_in_turn(dtype, bits):
    """K's and V's heads in turn, rows in turn, heads side by side; every element outside keeps its value."""
    heads, dim, lengths = 3, 64, [37, 5]
    c = paro.KVCache.empty(1, 6, heads, 16, dim, 2, 4, dtype, bits=bits)
    c.table.copy_(torch.tensor([[4, 0, 2, -1], [5, -1, -1, -1]], dtype=torch.int32))
    c.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
    cu, slots = torch.tensor([0, 37, 42], device="cuda"), torch.arange(2, dtype=torch.int32, device="cuda")
    n = sum(lengths)
    paro.paro_kv_append(c, 0, randn((n, heads, dim), dtype, 1), randn((n, heads, dim), dtype, 2), slots, cu)
    k, v = (torch.empty((n, heads, dim), dtype=dtype, device="cuda") for _ in range(2))
    paro.paro_kv_read(c, 0, k, v, slots, cu)
    for shape, mine, other in (((n, heads, 2, dim), lambda t: t[:, :, 0], lambda t: t[:, :, 1]),
                               ((n, heads, 3, dim), lambda t: t[:, :, 2], lambda t: t[:, :, 0]),
                               ((n, 2, heads, dim), lambda t: t[:, 0], lambda t: t[:, 1]),
                               ((n, 9, dim), lambda t: t[:, 5:8], lambda t: t[:, 1:4])):
        got, want = torch.full(shape, 7.0, dtype=dtype, device="cuda"), torch.full(shape, 7.0, dtype=dtype, device="cuda")
        mine(want).copy_(k)
        other(want).copy_(v)
        paro.paro_kv_read(c, 0, mine(got), other(got), slots, cu)
        assert torch.equal(got, want)
