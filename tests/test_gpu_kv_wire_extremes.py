"""GPU: restoring into an E4M3 cache, every element that is no NaN below every
scale byte and head scale: a lane's sixteen elements have no NaN among them, so
all of them go the way of ordinary numbers."""
import numpy as np
import pytest
import torch

from bf16_wire_all_amd import decode
from tests import wire_reference as wire
from tests.gpu_util import say
from tests.test_gpu_kv_wire import DEV, Cache, head_scales

pytestmark = pytest.mark.gpu


def numbers():
    """The 254 codes of numbers, and two of them again."""
    codes = np.arange(256, dtype=np.uint8)
    return np.where((codes & 0x7F) == 0x7F, codes - 1, codes).astype(np.uint8)


def more_scales():
    """Those of the other test, and ones about the ends of what is taken by reciprocals."""
    ends = [m * 2.0 ** e for e in (-61, -60, -59, 59, 60, 61) for m in (1.0, 1.0 + 2.0 ** -23, 1.5, 1.75, 1.875, 2.0 - 2.0 ** -23)]
    s = np.concatenate([head_scales().reshape(-1), np.array(ends), [3.0, 0.7, 5.5, 1e-9]])
    return s.astype(np.float32).reshape(2, -1)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_every_number_over_every_scale_byte_by_head_scales(d):
    """Bit for bit what the quotient in binary32 rounds to."""
    scales = more_scales()
    heads, parts = scales.shape[1], 256 // d
    n, tokens = 2 * heads * d, 256 * parts                       # token: scale byte, and which of the codes
    codes = np.tile(numbers().reshape(1, parts, 1, d), (256, 1, 2 * heads, 1)).reshape(tokens, n)
    rec = np.concatenate([codes, np.repeat(np.repeat(np.arange(256, dtype=np.uint8), parts)[:, None], n // 32, 1)], 1)
    rec = np.pad(rec, ((0, 0), (0, -rec.shape[1] % 16)))
    c = Cache(tokens, 1, heads, d, "e4m3", "tokens", seed=4)
    for mine, theirs, v in ((c.ks, c.c.tensors[2], scales[0]), (c.vs, c.c.tensors[3], scales[1])):
        mine.copy_(torch.from_numpy(v))
        theirs.copy_(mine)
    say("numbers by head scales", d)
    decode.kv_restore(torch.from_numpy(rec).to(DEV), 8, c.c, torch.arange(tokens, device=DEV))
    with np.errstate(all="ignore"):
        q = wire.values(rec, n, 8).reshape(tokens, 2, heads, d).astype(np.float32) / scales[None, :, :, None]
    assert q.dtype == np.float32
    nan = np.isnan(q)
    want = wire.nearest(np.clip(np.where(nan, 0, q), -448, 448).astype(np.float64), 8)
    got = c.rows().numpy()
    assert np.array_equal(got[~nan], want[~nan])
    assert ((got[nan] & 0x7F) == 0x7F).all() and nan.any()
