"""GPU: a cache's slots as records of 8 or 4 bits (xfer_kv_quantize) and back
(xfer_kv_restore) against the formulas in 64 bits.  Elements and scales of the
records are compared bit for bit, and so is what comes back into a BF16 cache;
an E4M3 cache divides in binary32 first, so there a value may be half a step
off.  Every byte outside the named slots and records has to stay."""
import numpy as np
import pytest
import torch

import bf16_wire_all_amd as x
from bf16_wire_all_amd import decode
from tests import wire_reference as wire
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


class Cache:
    """A cache full of marks or given bits; the pool holds keys and values in turn."""

    def __init__(self, n_pages, page, heads, d, kind, order, seed=1, finite=True):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.heads, self.d, self.page, self.n_slots = kind, heads, d, page, n_pages * page
        shape = (n_pages, 2) + ((page, heads, d) if order == "tokens" else (heads, page, d))
        if kind == "bf16":
            spread = torch.randn(shape, generator=g) * 2.0 ** torch.randint(-6, 7, shape[:-1] + (1,), generator=g)
            pool = spread.to(torch.bfloat16).view(torch.int16)
        else:
            pool = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
            if finite:
                pool = torch.where((pool & 0x7F) == 0x7F, 0x3A, pool)
        self.pool = pool.to(DEV)
        self.order = order
        self.ks = self.vs = None
        if kind == "e4m3":
            self.ks, self.vs = (torch.rand(heads, generator=g) + 0.3 for _ in range(2))
        self.c = decode.kv_cache(*self.views(self.pool), *(None if s is None else s.to(DEV) for s in (self.ks, self.vs)))

    def views(self, pool):
        k, v = pool[:, 0], pool[:, 1]
        return (k, v) if self.order == "tokens" else (k.transpose(1, 2), v.transpose(1, 2))

    def rows(self, pool=None):
        """Bit patterns [slots, 2, heads, d] on the CPU."""
        k, v = self.views((self.pool if pool is None else pool).cpu())
        return torch.stack([t.reshape(-1, self.heads, self.d) for t in (k, v)], 1)

    def values(self):
        bits = self.rows()
        if self.kind == "bf16":
            return bits.contiguous().view(torch.bfloat16).double().numpy()
        f = bits.contiguous().view(torch.float8_e4m3fn).float()
        return (f * torch.stack([self.ks, self.vs])[None, :, :, None]).double().numpy()   # a product in binary32


def slots_of(n, n_slots, seed, bad=()):
    s = torch.randperm(n_slots, generator=torch.Generator().manual_seed(seed))[:n]
    for i, value in bad:
        if i < n:
            s[i] = value
    return s


def in_range(slots, n):
    return ((slots >= 0) & (slots < n)).numpy()


BAD = [(3, -1), (7, 1 << 40), (8, -(1 << 62)), (11, 10 ** 9)]
SHAPES = [(1, 1, 128, 16, "heads"), (37, 8, 128, 16, "heads"), (50, 3, 64, 32, "tokens"), (13, 2, 256, 1, "tokens"),
          (1, 1, 64, 1, "heads"), (300, 5, 128, 64, "tokens"), (129, 1, 256, 128, "heads"), (1025, 1, 64, 8, "tokens")]


@pytest.mark.parametrize("tokens,heads,d,page,order", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("bits", [8, 4])
def test_quantize(tokens, heads, d, page, order, kind, bits):
    say("quantize", tokens, heads, d, page, order, kind, bits)
    c = Cache(-(-tokens // page) + 3, page, heads, d, kind, order, seed=tokens + d)
    slots = slots_of(tokens, c.n_slots, 5, BAD)
    need = decode.kv_record_bytes(c.c, bits)
    gap = 32
    buf = torch.full((tokens, need + gap), 0xA5, dtype=torch.uint8, device=DEV)
    before = c.pool.clone()
    decode.kv_quantize(c.c, slots.to(DEV), buf[:, :need], bits)
    got = buf.cpu().numpy()
    there = in_range(slots, c.n_slots)
    v = c.values()[np.where(there, slots.numpy(), 0)].reshape(tokens, -1)
    v[~there] = 0.0
    assert np.array_equal(got[:, :need], wire.records(v, bits))
    assert (got[:, need:] == 0xA5).all()
    assert torch.equal(c.pool, before)


@pytest.mark.parametrize("tokens,heads,d,page,order", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("bits", [8, 4])
def test_restore(tokens, heads, d, page, order, kind, bits):
    say("restore", tokens, heads, d, page, order, kind, bits)
    g = torch.Generator().manual_seed(tokens * 3 + d)
    c = Cache(-(-tokens // page) + 3, page, heads, d, kind, order, seed=9)
    n, need = 2 * heads * d, decode.kv_record_bytes(c.c, bits)
    records = torch.randint(0, 256, (tokens, need + 16), generator=g, dtype=torch.uint8)
    records[:, n * bits // 8:n * bits // 8 + n // 32] = torch.randint(115, 128, (tokens, n // 32), generator=g).to(torch.uint8)
    slots = slots_of(tokens, c.n_slots, 6, BAD)
    before = c.rows()
    sent = records.to(DEV)
    decode.kv_restore(sent[:, :need], bits, c.c, slots.to(DEV))
    assert torch.equal(sent.cpu(), records)
    there = in_range(slots, c.n_slots)
    check_restored(c, before, slots.numpy()[there], wire.values(records.numpy(), n, bits)[there])


def check_restored(c, before, slots, v):
    got, n = c.rows(), len(slots)
    v = v.reshape(n, 2, c.heads, c.d)
    others = np.setdiff1d(np.arange(c.n_slots), slots)
    assert torch.equal(got[others], before[others])
    got = got[torch.from_numpy(slots)]
    if c.kind == "bf16":
        bits, want = got.numpy().view(np.uint16), wire.bf16_bits(v)
        nan = np.isnan(v)
        assert np.array_equal(bits[~nan], want[~nan])
        assert ((bits[nan] & 0x7FFF) > 0x7F80).all()
        return
    # a quotient in binary32, off by 2^-24 of itself, then half a step of E4M3
    exact = np.clip(v / torch.stack([c.ks, c.vs]).double().numpy()[None, :, :, None], -448, 448)
    value = got.contiguous().view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(value), np.isnan(exact))
    ok = ~np.isnan(exact)
    tol = 2.0 ** -24 * np.abs(exact[ok]) * (1 + 2.0 ** -4) + np.maximum(2.0 ** -4 * np.abs(exact[ok]), 2.0 ** -10)
    assert (np.abs(value[ok] - exact[ok]) <= tol).all()


TOPS = [0x0000, 0x0001, 0x007F, 0x0080, 0x0100, 0x0460, 0x0461, 0x3F00, 0x40C0, 0x40C1, 0x43DF, 0x43E0, 0x43E1, 0x43E8, 0x43FF,
        0x7F60, 0x7F61, 0x7F7F]


@pytest.mark.parametrize("bits", [8, 4])
def test_every_pattern_below_every_kind_of_largest_one(bits):
    """All finite BF16 numbers, 31 of them in a block below its largest."""
    rows = []
    for top in TOPS:
        mags = np.arange(top + 1, dtype=np.uint16)
        if len(mags) > 3000:   # all of the highest two thousand, some of the rest
            mags = np.concatenate([mags[::37], mags[-2000:]])
        both = np.concatenate([mags, mags | 0x8000])
        both = np.pad(both, (0, -len(both) % 31)).reshape(-1, 31)
        rows.append(np.concatenate([both, np.full((len(both), 1), top | (0x8000 if top % 2 else 0), np.uint16)], 1))
    blocks = np.concatenate(rows)
    blocks = np.pad(blocks, ((0, -len(blocks) % 8), (0, 0)))
    p = blocks.reshape(-1, 1, 2, 128)                                    # one head, pages of one token
    pool = torch.from_numpy(p.astype(np.uint16).view(np.int16).copy()).to(DEV)
    cache = decode.kv_cache(pool[:, :, 0:1], pool[:, :, 1:2])
    slots = torch.arange(len(p), device=DEV)
    rec = torch.zeros((len(p), decode.kv_record_bytes(cache, bits)), dtype=torch.uint8, device=DEV)
    say("patterns", bits, len(p))
    decode.kv_quantize(cache, slots, rec, bits)
    v = torch.from_numpy(p.view(np.int16).copy()).view(torch.bfloat16).double().numpy().reshape(len(p), -1)
    want = wire.records(v, bits)
    assert np.array_equal(rec.cpu().numpy(), want)
    # and back: exactly what the records stand for, which quantises to the same values
    back = torch.zeros_like(pool)
    to = decode.kv_cache(back[:, :, 0:1], back[:, :, 1:2])
    decode.kv_restore(rec, bits, to, slots)
    stood = wire.values(want, 256, bits)
    assert np.array_equal(back.cpu().numpy().view(np.uint16).reshape(len(p), -1), wire.bf16_bits(stood))
    # what rounds up to 2^128 is past BF16, and comes back infinite
    kept = (np.abs(stood) < 2.0 ** 128).reshape(-1, 32).all(1)
    assert not kept.all() and np.abs(v.reshape(-1, 32)[~kept]).max(1).min() >= 1.75 * 2.0 ** 127
    held = stood.reshape(-1, 32)[kept]
    assert np.array_equal(wire.bf16_bits(held).astype(np.uint32) << 16, held.astype(np.float32).view(np.uint32))
    again = torch.zeros_like(rec)
    decode.kv_quantize(to, slots, again, bits)
    assert np.array_equal(wire.values(again.cpu().numpy(), 256, bits).reshape(-1, 32)[kept], held)


@pytest.mark.parametrize("bits", [8, 4])
def test_a_block_that_is_not_finite_becomes_nan_alone(bits):
    c = Cache(4, 4, 2, 64, "bf16", "tokens")
    bits_of = {"nan": 0x7FC1, "-nan": 0xFF81, "inf": 0x7F80, "-inf": 0xFF80}
    for i, b in enumerate(bits_of.values()):
        c.views(c.pool)[i % 2][i, 1, i % 2, 40 * (i // 2) + 3] = int(np.uint16(b).view(np.int16))
    slots = torch.arange(c.n_slots, device=DEV)
    rec = torch.zeros((c.n_slots, decode.kv_record_bytes(c.c, bits)), dtype=torch.uint8, device=DEV)
    say("not finite", bits)
    decode.kv_quantize(c.c, slots, rec, bits)
    v = c.values().reshape(c.n_slots, -1)
    want = wire.records(v, bits)
    assert (want == 255).sum() >= 4
    assert np.array_equal(rec.cpu().numpy(), want)
    before = c.rows()
    decode.kv_restore(rec, bits, c.c, slots)
    stood = wire.values(want, 256, bits)
    assert np.isnan(stood).sum() == 32 * 4
    check_restored(c, before, np.arange(c.n_slots), stood)


def test_nan_of_an_e4m3_cache_and_of_its_scale():
    c = Cache(2, 8, 2, 64, "e4m3", "heads", finite=False)
    slots = torch.arange(c.n_slots, device=DEV)
    rec = torch.zeros((c.n_slots, decode.kv_record_bytes(c.c, 8)), dtype=torch.uint8, device=DEV)
    decode.kv_quantize(c.c, slots, rec, 8)
    want = wire.records(c.values().reshape(c.n_slots, -1), 8)
    assert (want[:, 256:264] == 255).any() and np.array_equal(rec.cpu().numpy(), want)
    c.c.tensors[2][1] = float("inf")
    c.ks[1] = float("inf")
    decode.kv_quantize(c.c, slots, rec, 8)
    assert np.array_equal(rec.cpu().numpy(), wire.records(c.values().reshape(c.n_slots, -1), 8))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_any_bytes_are_valid_records(bits, kind):
    """Every element code below every scale byte."""
    codes = np.tile(np.arange(256, dtype=np.uint8), 256).reshape(256, 256)
    n = 256 if bits == 8 else 512
    d = n // 2
    rec = np.concatenate([codes, np.repeat(np.arange(256, dtype=np.uint8)[:, None], n // 32, 1)], 1)
    rec = np.pad(rec, ((0, 0), (0, -rec.shape[1] % 16)), constant_values=0xEE)
    c = Cache(256, 1, 1, d, kind, "tokens", seed=4)
    before = c.rows()
    say("any bytes", bits, kind)
    decode.kv_restore(torch.from_numpy(rec).to(DEV), bits, c.c, torch.arange(256, device=DEV))
    check_restored(c, before, np.arange(256), wire.values(rec, n, bits))


def head_scales():
    """Ordinary ones, those whose quotients are halfway between E4M3 numbers but for binary32's rounding, and extremes."""
    rng = np.random.default_rng(8)
    halfway = [a / b for a in (8, 11, 13, 15) for b in (17, 21, 25, 27, 31)]
    powers = [2.0 ** e for e in (-149, -127, -126, -61, -60, -59, 0, 59, 60, 61, 127)]
    rest = [0.0, -0.0, -1.7, float("inf"), float("-inf"), float("nan"), 3.4e38, 1e-40, 1.0 - 2.0 ** -24, 1.0 + 2.0 ** -23]
    s = np.concatenate([halfway, powers, rest, rng.uniform(1e-3, 1e3, 96 - 41)]).astype(np.float32)
    return s.reshape(2, 48)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d", [64, 256])
def test_every_element_over_every_scale_byte_by_head_scales(bits, d):
    """Bit for bit what the quotient in binary32 rounds to."""
    scales = head_scales()
    heads = scales.shape[1]
    n, codes_of = 2 * heads * d, d * bits // 8
    codes = np.tile((np.arange(256 * codes_of) * (1 if bits == 8 else 37) % 256).astype(np.uint8).reshape(256, 1, codes_of),
                    (1, 2 * heads, 1)).reshape(256, -1)
    rec = np.concatenate([codes, np.repeat(np.arange(256, dtype=np.uint8)[:, None], n // 32, 1)], 1)
    rec = np.pad(rec, ((0, 0), (0, -rec.shape[1] % 16)))
    c = Cache(256, 1, heads, d, "e4m3", "tokens", seed=4)
    for mine, theirs, v in ((c.ks, c.c.tensors[2], scales[0]), (c.vs, c.c.tensors[3], scales[1])):
        mine.copy_(torch.from_numpy(v))
        theirs.copy_(mine)
    say("head scales", bits, d)
    decode.kv_restore(torch.from_numpy(rec).to(DEV), bits, c.c, torch.arange(256, device=DEV))
    with np.errstate(all="ignore"):
        q = wire.values(rec, n, bits).reshape(256, 2, heads, d).astype(np.float32) / scales[None, :, :, None]
    assert q.dtype == np.float32
    nan = np.isnan(q)
    want = wire.nearest(np.clip(np.where(nan, 0, q), -448, 448).astype(np.float64), 8)
    got = c.rows().numpy()
    assert np.array_equal(got[~nan], want[~nan])
    assert ((got[nan] & 0x7F) == 0x7F).all() and nan.any()


def test_a_slot_may_be_read_any_number_of_times_and_records_lie_far_apart():
    c = Cache(3, 16, 2, 128, "bf16", "heads")
    slots = torch.tensor([5, 5, 47, 5, 0], device=DEV)
    need = decode.kv_record_bytes(c.c, 8)
    buf = torch.zeros(4 * (1 << 30) + need, dtype=torch.uint8, device=DEV)      # records 1 GiB apart: offsets past 32 bits
    rec = buf.as_strided((5, need), (1 << 30, 1))
    say("records far apart")
    decode.kv_quantize(c.c, slots, rec, 8)
    want = wire.records(c.values()[slots.cpu().numpy()].reshape(5, -1), 8)
    assert np.array_equal(rec.cpu().numpy(), want)
    before = c.rows()
    to = torch.tensor([1, 2, 3, 40, 41], device=DEV)
    decode.kv_restore(rec, 8, c.c, to)
    check_restored(c, before, to.cpu().numpy(), wire.values(want, 512, 8))


def test_slots_past_4_gib_of_a_cache():
    page = 16 * 8 * 128 * 2
    n_pages = (5 << 30) // (2 * page)
    pool = torch.zeros((n_pages, 2, 8, 16, 128), dtype=torch.bfloat16, device=DEV)
    k, v = pool[:, 0].transpose(1, 2), pool[:, 1].transpose(1, 2)
    k[n_pages - 1, 9] = torch.randn((8, 128), device=DEV).to(torch.bfloat16)
    v[n_pages - 1, 9] = torch.randn((8, 128), device=DEV).to(torch.bfloat16)
    cache = decode.kv_cache(k, v)
    rec = torch.zeros((1, decode.kv_record_bytes(cache, 8)), dtype=torch.uint8, device=DEV)
    say("far slots")
    decode.kv_quantize(cache, torch.tensor([(n_pages - 1) * 16 + 9], device=DEV), rec, 8)
    src = torch.stack([k[n_pages - 1, 9], v[n_pages - 1, 9]]).cpu().double().numpy().reshape(1, -1)
    assert np.array_equal(rec.cpu().numpy(), wire.records(src, 8))
    decode.kv_restore(rec, 8, cache, torch.tensor([(n_pages - 2) * 16 + 3], device=DEV))
    got = torch.stack([k[n_pages - 2, 3], v[n_pages - 2, 3]]).cpu().view(torch.int16).numpy().view(np.uint16).reshape(1, -1)
    assert np.array_equal(got, wire.bf16_bits(wire.values(wire.records(src, 8), 2048, 8)))
    assert int((pool[:n_pages - 2] != 0).sum()) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_large_calls_take_the_path_past_the_caches(kind):
    """More bytes than the caches hold, the same bits as in pieces that they do hold."""
    tokens = 40000 if kind == "bf16" else 70000
    c = Cache(-(-tokens // 64), 64, 8, 128, kind, "heads", seed=3)
    slots = slots_of(tokens, c.n_slots, 8).to(DEV)
    for bits in (8, 4):
        need = decode.kv_record_bytes(c.c, bits)
        whole, pieces = (torch.zeros((tokens, need), dtype=torch.uint8, device=DEV) for _ in range(2))
        say("large", kind, bits)
        decode.kv_quantize(c.c, slots, whole, bits)
        for i in range(0, tokens, 9999):
            decode.kv_quantize(c.c, slots[i:i + 9999], pieces[i:i + 9999], bits)
        assert torch.equal(whole, pieces)
        pool = c.pool.clone()
        decode.kv_restore(whole, bits, c.c, slots)
        once, c.pool[:] = c.pool.clone(), pool
        for i in range(0, tokens, 9999):
            decode.kv_restore(whole[i:i + 9999], bits, c.c, slots[i:i + 9999])
        assert torch.equal(once, c.pool) and not torch.equal(pool, c.pool)
        c.pool[:] = pool


def test_another_stream_and_a_captured_graph():
    c, to = Cache(8, 16, 4, 128, "bf16", "heads"), Cache(8, 16, 4, 128, "e4m3", "tokens", seed=2)
    slots, to_slots = slots_of(90, c.n_slots, 1).to(DEV), slots_of(90, c.n_slots, 2).to(DEV)
    rec = torch.zeros((90, decode.kv_record_bytes(c.c, 4)), dtype=torch.uint8, device=DEV)

    def step():
        decode.kv_quantize(c.c, slots, rec, 4)
        decode.kv_restore(rec, 4, to.c, to_slots)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        c.pool.copy_(torch.randn(c.pool.shape, device=DEV).to(torch.bfloat16).view(torch.int16))
        step()
        want = rec.clone(), to.pool.clone()
        rec.zero_(), to.pool.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        there = to.rows()[to_slots.cpu()]
        assert torch.equal(rec, want[0]) and torch.equal(there, to.rows(want[1])[to_slots.cpu()])
        to.pool.copy_(want[1])


def test_the_binding_refuses_what_it_cannot_read():
    c = Cache(2, 16, 2, 128, "bf16", "heads")
    need = decode.kv_record_bytes(c.c, 8)
    slots, rec = torch.arange(4, device=DEV), torch.zeros((4, need), dtype=torch.uint8, device=DEV)
    for bad in (dict(slots=slots.int()), dict(slots=slots.cpu()), dict(slots=slots[:3]), dict(records=rec[:, :-16]),
                dict(records=rec.half()), dict(records=rec.cpu()), dict(records=rec.t())):
        a = {"slots": slots, "records": rec, **bad}
        with pytest.raises(ValueError):
            decode.kv_quantize(c.c, a["slots"], a["records"], 8)
        with pytest.raises(ValueError):
            decode.kv_restore(a["records"], 8, c.c, a["slots"])
    with pytest.raises(x.XferError):
        decode.kv_quantize(c.c, slots, rec, 5)
    with pytest.raises(x.XferError):
        decode.kv_quantize(c.c, slots, torch.zeros((4, need + 8), dtype=torch.uint8, device=DEV), 8)
