"""GPU: a slot that the cache does not have gives a record of zeros, whatever the heads' scales are."""
import numpy as np
import pytest
import torch

from bf16_wire_all_amd import decode
from tests import wire_reference as wire
from tests.gpu_util import say
from tests.test_gpu_kv_wire import DEV, Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("heads,d", [(8, 128), (6, 64), (3, 256), (1, 64)])
def test_a_missing_slot_under_any_head_scale_is_zeros(bits, heads, d):
    c = Cache(3, 16, heads, d, "e4m3", "heads", seed=6)
    odd = np.array([np.inf, -np.inf, np.nan, -1.7, -0.0, 3e38, 1e-40, 0.5], np.float32)
    for i, (mine, theirs) in enumerate(((c.ks, c.c.tensors[2]), (c.vs, c.c.tensors[3]))):
        mine.copy_(torch.from_numpy(np.resize(np.roll(odd, 3 * i), heads)))
        theirs.copy_(mine)
    slots = torch.tensor([-1, 5, 48, 1 << 40, 47, -(1 << 62), 0])
    rec = torch.full((7, decode.kv_record_bytes(c.c, bits)), 0xA5, dtype=torch.uint8, device=DEV)
    say("missing", bits, heads, d)
    decode.kv_quantize(c.c, slots.to(DEV), rec, bits)
    got = rec.cpu().numpy()
    there = ((slots >= 0) & (slots < 48)).numpy()
    assert not got[~there].any()
    with np.errstate(all="ignore"):
        v = c.values()[slots.numpy()[there]].reshape(there.sum(), -1)
    assert np.array_equal(got[there], wire.records(v, bits))
