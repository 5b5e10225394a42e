"""GPU: what the decode-step binding takes for which format.  Tensors of another
type of the same size, and shards on another device, are refused before the
call; a single row may be of any width."""
import numpy as np
import pytest
import torch

from bf16_wire_all_amd import decode
from tests import decode_reference as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
R, HQ, HKV, D, PAGE = 2, 4, 2, 64, 16


def ones(shape, dtype):
    return torch.ones(shape, device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float32, torch.bool])
def test_caches_of_other_types_are_refused(dtype):
    bad = torch.zeros((3, PAGE, HKV, D), device=DEV).to(dtype)
    with pytest.raises(ValueError):
        decode.kv_cache(bad, bad.clone())


def test_keys_and_values_of_different_types_are_refused():
    k = torch.zeros((3, PAGE, HKV, D), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        decode.kv_cache(k, k.to(torch.float16))


def test_scales_of_other_types_are_refused():
    k = torch.zeros((3, PAGE, HKV, D), dtype=torch.uint8, device=DEV)
    decode.kv_cache(k, k.clone(), ones(HKV, torch.float32))
    for at in (0, 1):
        scales = [None, None]
        scales[at] = ones(HKV, torch.int32)
        with pytest.raises(ValueError):
            decode.kv_cache(k, k.clone(), *scales)


def cache():
    k = torch.zeros((3, PAGE, HKV, D), dtype=torch.bfloat16, device=DEV)
    return decode.kv_cache(k, k.clone())


ATTN = {"q": [torch.float16], "table": [torch.float32, torch.int64], "lens": [torch.float32, torch.int64],
        "out": [torch.float16, torch.int32, torch.float64]}


@pytest.mark.parametrize("name,dtype", [(n, t) for n, ts in ATTN.items() for t in ts])
def test_attention_refuses_other_types(name, dtype):
    args = {"q": ones((R, HQ, D), torch.bfloat16), "table": torch.zeros((R, 1), dtype=torch.int32, device=DEV),
            "lens": ones(R, torch.int32), "out": ones((R, HQ, D), torch.bfloat16)}
    c = cache()
    decode.attn_paged(c, args["q"], args["table"], args["lens"], PAGE, 1.0, args["out"])
    args[name] = args[name].to(dtype)
    before = args["out"].clone()
    with pytest.raises(ValueError):
        decode.attn_paged(c, args["q"], args["table"], args["lens"], PAGE, 1.0, args["out"])
    torch.cuda.synchronize()
    assert torch.equal(args["out"], before)


STORE = {"q": [torch.float16], "k": [torch.float16], "v": [torch.float16], "q_out": [torch.float16],
         "positions": [torch.float32, torch.int64], "cos_sin": [torch.int32, torch.float64],
         "slots": [torch.float64, torch.int32], "q_weight": [torch.float16], "k_weight": [torch.float16]}


@pytest.mark.parametrize("name,dtype", [(n, t) for n, ts in STORE.items() for t in ts])
def test_the_store_refuses_other_types(name, dtype):
    args = {"q": ones((R, HQ, D), torch.bfloat16), "k": ones((R, HKV, D), torch.bfloat16),
            "v": ones((R, HKV, D), torch.bfloat16), "positions": torch.zeros(R, dtype=torch.int32, device=DEV),
            "cos_sin": ones((9, D), torch.float32), "slots": torch.arange(R, device=DEV),
            "q_out": ones((R, HQ, D), torch.bfloat16), "q_weight": ones(D, torch.bfloat16),
            "k_weight": ones(D, torch.bfloat16)}
    c = cache()
    decode.qkv_rope_store(c, **args)
    args[name] = args[name].to(dtype)
    before = c.tensors[0].clone()
    with pytest.raises(ValueError):
        decode.qkv_rope_store(c, **args)
    torch.cuda.synchronize()
    assert torch.equal(c.tensors[0], before)


def draw(l0, l1, rows, u=None):
    n0, n1 = l0.shape[1], l1.shape[1]
    s = decode.shard(l0, n0, 0), decode.shard(l1, n1, n0)
    out = torch.full((rows, 2), 9, dtype=torch.int32, device=DEV)
    ws = torch.empty(decode.sample_workspace_bytes(rows, n0, n1), dtype=torch.uint8, device=DEV)
    params = torch.from_numpy(np.array([(1.0, 0, 1.0, 0.0)] * rows, decode.SAMPLE_PARAMS).view(np.uint8).copy()).to(DEV)
    return (*s, params, torch.full((rows,), 0.5, device=DEV) if u is None else u, out, ws)


def test_logits_and_numbers_of_other_types_are_refused():
    x = torch.zeros((R, 64), device=DEV)
    for dtype in (torch.float16, torch.float32):
        with pytest.raises(ValueError):
            decode.shard(x.to(dtype), 64, 0)
    b = x.to(torch.bfloat16)
    decode.sample_merge(*draw(b, b, R))
    with pytest.raises(ValueError):
        decode.sample_merge(*draw(b, b, R, u=ones(R, torch.int32)))


def test_patterns_as_whole_numbers_are_taken():
    """BF16 as int16 or uint16, E4M3 as bytes: the same bits as the float types."""
    g = torch.Generator().manual_seed(3)
    k, v, q = (torch.randn(s, generator=g).to(torch.bfloat16).to(DEV) for s in ((3, PAGE, HKV, D),) * 2 + ((R, HQ, D),))
    table, lens = torch.tensor([[2], [0]], dtype=torch.int32, device=DEV), torch.tensor([9, 16], dtype=torch.int32, device=DEV)
    outs = []
    for dtype in (torch.bfloat16, torch.int16, torch.uint16):
        out = torch.zeros((R, HQ, D), dtype=torch.bfloat16, device=DEV)
        decode.attn_paged(decode.kv_cache(k.view(dtype), v.view(dtype)), q.view(dtype), table, lens, PAGE, 0.125,
                          out.view(dtype))
        outs.append(out)
    k8, v8 = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
    for dtype in (torch.float8_e4m3fn, torch.uint8, torch.int8):
        out = torch.zeros((R, HQ, D), dtype=torch.bfloat16, device=DEV)
        decode.attn_paged(decode.kv_cache(k8.view(dtype), v8.view(dtype)), q, table, lens, PAGE, 0.125, out)
        outs.append(out)
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs[:3]) and all(torch.equal(o, outs[3]) for o in outs[3:])
    assert bool(torch.isfinite(outs[0].float()).all()) and not torch.equal(outs[0], outs[3])


def test_shards_on_another_device_are_refused():
    b = torch.zeros((R, 64), dtype=torch.bfloat16, device=DEV)
    args = draw(b, b, R)
    for s in args[:2]:
        here = s.device
        s.device = here + 1                                # as a shard of another GPU's tensor has it
        with pytest.raises(ValueError):
            decode.sample_merge(*args)
        s.device = here
    decode.sample_merge(*args)
    torch.cuda.synchronize()
    assert bool((args[4][:, 1] != 9).all())


@pytest.mark.parametrize("n0,n1", [(1, 1), (1001, 500), (40003, 20001), (7, 32770)])
def test_one_row_of_any_width(n0, n1):
    """A single row has no distance to a next one that could be odd."""
    say("sample, one row", n0, n1)
    g = torch.Generator().manual_seed(n0)
    l0, l1 = (torch.randn((1, n), generator=g).to(torch.bfloat16) for n in (n0, n1))
    args = draw(l0.to(DEV), l1.to(DEV), 1)
    decode.sample_merge(*args)
    torch.cuda.synchronize()
    got = args[4].cpu().numpy().view(decode.SAMPLED)[0, 0]
    x = torch.cat([l0, l1], 1)[0].double().numpy()
    idx, prob, margin = ref.sample(x, np.arange(n0 + n1), 1.0, 0, 1.0, 0.0, 0.5)
    assert margin > 1e-12 and got["idx"] == idx and abs(got["prob"] - prob) <= 2.0 ** -23 * prob
