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
