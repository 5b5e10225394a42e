"""GPU: rows that are not cut up (xfer_attn_paged), in counts of rows, kv heads
and groups of query heads that do not divide evenly among the eight dies:
every (row, head) is computed once, and nothing past the output is written."""
import pytest

from tests.test_gpu_attn_paged import World, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (3, 3), (40, 40), (28, 28), (66, 2), (99, 3), (132, 4)])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 17])
@pytest.mark.parametrize("d,kind", [(64, "e4m3"), (128, "bf16")])
def test_rows_and_heads_of_every_count(rows, hq, hkv, d, kind):
    w = World([1 + (29 * i + 7 * hq) % 70 for i in range(rows)], hq, hkv, d, 16, kind, seed=rows + hq)
    assert w.workspace()[1] == 0
    run(w)
