"""GPU: several new tokens of one request as rows of their own, with the same
pages and increasing lengths (drafted positions): each row sees the tokens up
to its own and none of those that the later rows see."""
import pytest
import torch

from tests.test_gpu_attn_paged import World, run

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def drafted(lens, positions, hq, hkv, d, kind, **kw):
    """A World of one row for each of the last `positions` tokens of every request."""
    w = World(lens, hq, hkv, d, 16, kind, **kw)
    g = torch.Generator().manual_seed(sum(lens))
    rows = [(r, n - positions + 1 + i) for r, n in enumerate(lens) for i in range(positions)]
    assert min(n for _, n in rows) > 0
    width = w.table.shape[1]
    table = torch.full((len(rows), width + 1), 0x7FFFFFFF, dtype=torch.int32, device=DEV)
    table[:, :width] = w.table[[r for r, _ in rows]]
    whole = w.at
    w.table, w.rows, w.lens = table[:, :width], len(rows), [n for _, n in rows]
    w.dlens = torch.tensor(w.lens, dtype=torch.int32).to(DEV)
    assert w.window == 0
    w.at = [(whole[r][0][:n], whole[r][1][:n]) for r, n in rows]
    w.q = (torch.randn((len(rows), hq, d), generator=g) * 1.5).to(torch.bfloat16)
    w.dq = w.q.to(DEV)
    return w


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("positions", [2, 4, 5])
@pytest.mark.parametrize("lens,max_len", [([17, 33, 5, 130], None), ([900, 300, 1025], None), ([4100, 20, 9000], None),
                                          ([700, 1600], 60000)])
def test_positions_of_one_request(lens, max_len, positions, kind):
    run(drafted(lens, positions, 8, 4, 128, kind, order="tokens", max_len=max_len, seed=51), calls=2)
