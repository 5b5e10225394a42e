"""GPU: every variant of the store kernel (head_dim, kind of cache, rotation
order; one head a lane, four, or four past the caches).  The first two against
the formulas in 64 bits, the third by the bits of calls that take the second."""
import numpy as np
import pytest
import torch

from bf16_wire_all_amd import decode
from tests.gpu_util import say
from tests.test_gpu_rope_store import World

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens", [9, 1100])
def test_few_and_many_workgroups(tokens, d, kind, pairs):
    say("rope_store", tokens, d, kind, pairs)
    w = World(tokens, 1, 1, d, 16, kind, "heads", True, d // 2, pairs, seed=d + tokens)
    before, fused = w.pool.cpu().clone(), w.fused.cpu().clone()
    q_out = torch.empty(w.q.shape, dtype=torch.bfloat16, device=DEV)
    w.call(q_out)
    w.check(q_out, before, fused)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_past_the_caches(d, kind, pairs):
    hq, hkv = 40, 8
    t = (128 << 20) // (4 * (hq + 2 * hkv) * d) + 100
    say("rope_store past the caches", t, d, kind, pairs)
    w = World(t, hq, hkv, d, 16, kind, "tokens", True, d, pairs, seed=d)
    whole = torch.empty(w.q.shape, dtype=torch.bfloat16, device=DEV)
    before = w.pool.clone()
    w.call(whole)
    after = w.pool.clone()
    w.pool.copy_(before)
    cs, pos, slots = torch.from_numpy(w.cs).to(DEV), w.pos.to(DEV), w.slots.to(DEV)
    halves = torch.empty_like(whole)
    for r in (slice(0, t // 2), slice(t // 2, t)):
        decode.qkv_rope_store(w.cache, w.q[r], w.nk[r], w.nv[r], pos[r], cs, slots[r], halves[r], w.wq, w.wk,
                              interleaved=pairs)
    torch.cuda.synchronize()
    assert torch.equal(whole.view(torch.int16), halves.view(torch.int16))
    assert torch.equal(w.pool, after) and not torch.equal(before, after)


def test_a_position_outside_the_table_stores_neither_key_nor_value():
    w = World(6, 2, 1, 64, 4, "bf16", "tokens", True, 64, False, seed=6)
    w.slots = torch.arange(6)
    w.pos[1], w.pos[4] = -1, 500
    before = w.pool.cpu().clone()
    w.call(torch.zeros(w.q.shape, dtype=torch.bfloat16, device=DEV))
    torch.cuda.synchronize()
    bad, good = np.array([1, 4]), np.array([0, 2, 3, 5])
    for now, at in ((w.k, 0), (w.v, 1)):
        now, was = now.cpu().reshape(-1, 1, 64), before[:, at].reshape(-1, 1, 64)
        assert torch.equal(now[bad], was[bad])
        assert not any(torch.equal(now[i], was[i]) for i in good)
