"""Decode attention over the 16-bit cache whose rows end in many parts: each part is joined once, with few and with many
of them in flight."""
import pytest

torch = pytest.importorskip("torch")
pytest.importorskip("rotation_int4_weight_amd")
from test_gpu_attention_shares import TYPES, decode  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 1), (8, 1), (16, 1), (40, 1), (32, 8)])
@pytest.mark.parametrize("n", [1100, 9000, 33000])
def test_every_part_is_joined_once(n, heads, kv_heads, dim, dtype):
    """A row alone: 9, 71 and (of one key-value head) 256 parts."""
    for pattern in ("blocks", "rising", "last"):
        decode([n], heads, kv_heads, dim, 64, dtype, pattern, passes=2)
