"""The wire's calls on the CPU: every documented refusal, the records' sizes,
and the reference's own rounding against plain arithmetic.  No call here
reaches a launch: each either fails a host check or is empty work."""
import numpy as np
import pytest

import bf16_wire_all_amd as x
from bf16_wire_all_amd import decode
from tests import wire_reference as wire
from tests.test_decode_cpu import BAD_CACHES, K, KN, V, cache

S0 = 0
R, SLOTS = KN, KN + (1 << 30)


def quantize(c=None, slots=SLOTS, tokens=10, bits=8, records=R, ld=544):
    return decode.kv_quantize_raw(c or cache(), slots, tokens, bits, records, ld, stream=S0)


def restore(c=None, slots=SLOTS, tokens=10, bits=8, records=R, ld=544):
    return decode.kv_restore_raw(records, ld, tokens, bits, c or cache(), slots, stream=S0)


@pytest.mark.parametrize("call", [quantize, restore])
@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused(call, kw, status):
    assert call(cache(**kw)) == status


@pytest.mark.parametrize("call", [quantize, restore])
@pytest.mark.parametrize("kw", [dict(bits=0), dict(bits=5), dict(bits=16), dict(bits=-8), dict(slots=0), dict(slots=SLOTS + 4),
                                dict(records=0), dict(records=R + 8), dict(ld=520), dict(ld=512), dict(ld=0),
                                dict(ld=1 << 47), dict(ld=(1 << 64) - 16), dict(records=K), dict(records=V + 64),
                                dict(records=K - 544 * 9 - 16)])
def test_bad_arguments_are_refused(call, kw):
    assert call(**kw) == x.E_INVAL


def test_bits_are_checked_before_empty_work_and_pointers_are_not():
    for call in (quantize, restore):
        assert call(tokens=0, slots=0, records=0, ld=0) == x.OK
        assert call(tokens=0, bits=7) == x.E_INVAL


def test_an_output_over_an_input_is_refused():
    c = cache(kind=decode.KV_E4M3, k_scale=R + 544 * 9 + 524, v_scale=SLOTS + 4096)
    assert quantize(c) == x.E_INVAL                      # a scale in the last record
    assert quantize(slots=R + 544 * 9 + 520) == x.E_INVAL
    assert quantize(slots=R + 544 * 3 - 8) == x.E_INVAL
    # restoring writes the cache: nothing that is read may lie there
    assert restore(slots=K + 64) == x.E_INVAL
    assert restore(cache(kind=decode.KV_E4M3, v_scale=V + 128)) == x.E_INVAL


def test_restore_refuses_caches_whose_slots_share_bytes():
    assert restore(cache(token_stride=128)) == x.E_OVERLAP
    assert restore(cache(v=K + 256)) == x.E_OVERLAP
    assert restore(cache(head_stride=0)) == x.E_OVERLAP
    assert quantize(cache(head_stride=0), tokens=0) == x.OK


def test_too_large_is_refused():
    assert quantize(cache(kv_heads=1 << 23, head_stride=0), tokens=1) == x.E_UNSUPPORTED     # the record
    assert quantize(cache(kv_heads=1 << 31, head_stride=0, head_dim=256), tokens=1) == x.E_UNSUPPORTED
    assert quantize(cache(kv_heads=1 << 16, head_stride=0), tokens=(1 << 24) // (1 << 11) + 1, ld=1 << 25) == x.E_UNSUPPORTED


def record_bytes(c, bits):
    import ctypes
    return decode.lib().xfer_kv_record_bytes(ctypes.byref(c), bits)


def test_record_bytes():
    for heads in (1, 2, 3, 8):
        for d in (64, 128, 256):
            for bits in (8, 4):
                c = cache(kv_heads=heads, head_dim=d, head_stride=1024, token_stride=1024 * 8, page_stride=1 << 20)
                assert record_bytes(c, bits) == wire.records(np.zeros((1, 2 * heads * d)), bits).shape[1]
    assert record_bytes(cache(), 7) == 0
    assert record_bytes(cache(kind=3), 8) == 0
    assert record_bytes(cache(kv_heads=1 << 23, head_stride=0), 8) == 0


def test_the_reference_rounds_as_torch_does():
    import torch
    v = torch.linspace(-448, 448, 200001, dtype=torch.float64).float()
    got = wire.nearest(v.double().numpy(), 8)
    assert np.array_equal(got, v.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    halves = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, -0.0])
    assert list(wire.nearest(halves, 4)) == [0, 2, 2, 4, 4, 6, 6, 8, 14, 8]
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    with np.errstate(invalid="ignore"):
        f = bits.float().numpy().astype(np.float64)
    ok = ~np.isnan(f)
    assert np.array_equal(wire.bf16_bits(f)[ok], np.arange(65536, dtype=np.uint16)[ok])


def test_the_reference_s_scale_is_the_smallest_that_fits():
    for bits, top in ((8, 448.0), (4, 6.0)):
        for e in (-127, -120, -1, 0, 5, 118):
            for f, want in ((1.0, e), (1 + 2.0 ** -7, e + 1), (0.5, e - 1)):
                b = np.zeros((1, 32))
                b[0, 7] = -top * f * 2.0 ** e
                assert wire.scale_byte(b, bits)[0] == max(want, -127) + 127
