"""GPU: norms, rotation and the cache's rows (xfer_qkv_rope_store) against the
formulas in 64 bits, with every cache byte outside the named slots and every
byte around q_out compared with what was there before."""
import numpy as np
import pytest
import torch

import bf16_wire_all_amd as x
from bf16_wire_all_amd import decode
from tests import decode_reference as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def table(max_pos, rot_dim, seed=3):
    a = np.arange(max_pos)[:, None] * 1e4 ** (-np.arange(0, rot_dim, 2) / rot_dim)[None, :] + seed
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def bf16(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


class World:
    """Inputs of one call, on the CPU and on the GPU."""

    def __init__(self, tokens, hq, hkv, d, page, kind, order, norm, rot, pairs, seed=1, max_pos=500, extra=3):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.d, self.hq, self.hkv, self.page, self.rot, self.pairs = kind, d, hq, hkv, page, rot, pairs
        n_pages = -(-tokens // page) + extra
        shape = (n_pages, page, hkv, d) if order == "tokens" else (n_pages, hkv, page, d)
        # the cache starts full of marks, one buffer for keys and values in turn
        two = torch.randint(0, 256, (n_pages, 2) + shape[1:] + ((2,) if kind == "bf16" else ()), generator=g,
                            dtype=torch.uint8)
        two = two.view(torch.int16).squeeze(-1) if kind == "bf16" else two
        self.pool = two.to(DEV)
        self.order = order
        k, v = self.k, self.v = self.views(self.pool)
        self.ks = self.vs = None
        if kind == "e4m3":
            self.ks = (torch.rand(hkv, generator=g) + 0.01).to(DEV)
            self.vs = (torch.rand(hkv, generator=g) + 0.5).to(DEV)
        self.cache = decode.kv_cache(k, v, self.ks, self.vs)
        self.fused = bf16((tokens, (hq + 2 * hkv) * d), g, 2.0).to(DEV)
        f = self.fused
        self.q = f[:, :hq * d].view(tokens, hq, d)
        self.nk = f[:, hq * d:(hq + hkv) * d].view(tokens, hkv, d)
        self.nv = f[:, (hq + hkv) * d:].view(tokens, hkv, d)
        self.wq = (bf16((d,), g, 0.3) + 1).to(DEV) if norm else None
        self.wk = (bf16((d,), g, 0.3) + 1).to(DEV) if norm else None
        self.cs = table(max_pos, rot) if rot else None
        self.pos = torch.randint(0, max_pos, (tokens,), generator=g, dtype=torch.int32)
        if tokens > 1:
            self.pos[0], self.pos[-1] = 0, max_pos - 1
        self.slots = torch.randperm(n_pages * page, generator=g)[:tokens]
        if tokens > 2:
            self.slots[1] = -1
            self.slots[2] = n_pages * page  # past the cache: not stored

    def views(self, pool):
        """Keys and values of a pool as [page, token, head, dim]."""
        k, v = pool[:, 0], pool[:, 1]
        return (k.transpose(1, 2), v.transpose(1, 2)) if self.order == "heads" else (k, v)

    def call(self, q_out, stream=None):
        dcs = None if self.cs is None else torch.from_numpy(self.cs).to(DEV)
        decode.qkv_rope_store(self.cache, self.q, self.nk, self.nv, None if dcs is None else self.pos.to(DEV), dcs,
                              self.slots.to(DEV), q_out, self.wq, self.wk, eps=1e-6, interleaved=self.pairs,
                              stream=stream)

    def check(self, q_out, before, fused):
        torch.cuda.synchronize()
        d, hq, hkv = self.d, self.hq, self.hkv
        f = fused.float().numpy().astype(np.float64)
        t = f.shape[0]
        parts = (f[:, :hq * d].reshape(t, hq, d), f[:, hq * d:(hq + hkv) * d].reshape(t, hkv, d),
                 f[:, (hq + hkv) * d:].reshape(t, hkv, d))
        w = [None if a is None else a.cpu().float().numpy() for a in (self.wq, self.wk)]
        cs = self.cs if self.rot else np.zeros((1, 0), np.float32)
        pos = self.pos.numpy() if self.rot else np.zeros(t, int)
        yq, mq = ref.rope_heads(parts[0], w[0], 1e-6, cs, pos, self.rot, self.pairs)
        yk, mk = ref.rope_heads(parts[1], w[1], 1e-6, cs, pos, self.rot, self.pairs)
        if hq:
            got = q_out.cpu().float().numpy().astype(np.float64)
            assert np.all(np.abs(got - yq) <= ref.rope_tolerance(yq, mq, "bf16"))
        olds = self.views(before)
        for name, view, old, y, m, scale in (("k", self.k, olds[0], yk, mk, self.ks),
                                             ("v", self.v, olds[1], parts[2], np.abs(parts[2]), self.vs)):
            now = view.cpu()
            n_pages, page = now.shape[:2]
            flat = now.reshape(n_pages * page, hkv, d).contiguous()
            was = old.reshape(n_pages * page, hkv, d).contiguous()
            s = self.slots.numpy()
            kept = np.nonzero((s >= 0) & (s < n_pages * page))[0]
            rest = np.setdiff1d(np.arange(n_pages * page), s[kept])
            assert torch.equal(flat[rest], was[rest]), f"{name}: a slot that no token names changed"
            raw = flat[s[kept]]
            if self.kind == "bf16":
                got = raw.view(torch.bfloat16).float().numpy().astype(np.float64)
                assert np.all(np.abs(got - y[kept]) <= ref.rope_tolerance(y[kept], m[kept], "bf16")), name
            else:
                got = raw.view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
                sc = scale.cpu().numpy().astype(np.float64)[None, :, None]
                want = np.clip(y[kept] / sc, -ref.E4M3_MAX, ref.E4M3_MAX)
                assert np.all(np.abs(got - want) <= ref.rope_tolerance(want, m[kept] / sc, "e4m3")), name


def run(w, **kw):
    say("rope_store", w.fused.shape, w.kind, w.d)
    before, fused = w.pool.cpu().clone(), w.fused.cpu().clone()
    q_out = torch.full(w.q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    w.call(q_out, **kw)
    w.check(q_out, before, fused)
    assert torch.equal(w.fused.cpu().view(torch.int16), fused.view(torch.int16)), "an input changed"
    return q_out


CASES = [
    # tokens, q heads, kv heads, head_dim, page, kind, order, norm, rot, pairs
    (1, 1, 1, 64, 1, "bf16", "tokens", True, 64, False),
    (1, 40, 8, 128, 16, "bf16", "heads", True, 128, False),
    (2, 3, 1, 256, 4, "e4m3", "tokens", True, 256, True),
    (3, 5, 5, 128, 16, "e4m3", "heads", True, 64, False),
    (17, 7, 1, 64, 8, "bf16", "heads", False, 32, True),
    (77, 64, 8, 64, 32, "e4m3", "tokens", False, 32, True),
    (33, 0, 2, 128, 16, "bf16", "tokens", True, 128, False),      # keys and values alone
    (9, 4, 2, 128, 16, "bf16", "tokens", False, 0, False),        # no norm, no rotation: a plain store
    (5, 4, 2, 256, 64, "bf16", "tokens", True, 8, False),         # the narrowest rotation
    (700, 40, 8, 128, 16, "bf16", "heads", True, 128, False),     # many tokens: four heads for each lane
    (1100, 3, 1, 64, 16, "e4m3", "heads", True, 64, True),
    (600, 33, 3, 256, 128, "e4m3", "tokens", True, 128, True),
    (513, 20, 4, 256, 2, "bf16", "tokens", True, 256, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_against_the_formulas(case):
    run(World(*case, seed=sum(v for v in case if isinstance(v, int))))


def test_in_place_gives_the_same_bits():
    w = World(700, 40, 8, 128, 16, "bf16", "heads", True, 128, False, seed=5)
    want = run(w).cpu()
    w.call(w.q)
    torch.cuda.synchronize()
    assert torch.equal(w.q.cpu().view(torch.int16), want.view(torch.int16))


def test_a_large_batch_gives_the_bits_of_its_halves():
    """Past 128 MiB the projections are read another way: the same bits as two smaller calls."""
    say("rope_store, 4800 tokens and its halves")
    t, hq, hkv, d = 4800, 40, 8, 128
    assert 4 * t * (hq + 2 * hkv) * d > 128 << 20 > 4 * (t // 2) * (hq + 2 * hkv) * d
    w = World(t, hq, hkv, d, 16, "bf16", "heads", True, 128, False, seed=11)
    whole = torch.empty(w.q.shape, dtype=torch.bfloat16, device=DEV)
    w.call(whole)
    pool, cs, pos, slots = w.pool.clone(), torch.from_numpy(w.cs).to(DEV), w.pos.to(DEV), w.slots.to(DEV)
    halves = torch.empty_like(whole)
    w.pool.zero_()
    for r in (slice(0, t // 2), slice(t // 2, t)):
        decode.qkv_rope_store(w.cache, w.q[r], w.nk[r], w.nv[r], pos[r], cs, slots[r], halves[r], w.wq, w.wk)
    torch.cuda.synchronize()
    assert torch.equal(whole.view(torch.int16), halves.view(torch.int16))
    stored = w.k.reshape(-1, hkv, d)[slots[(slots >= 0) & (slots < w.k.shape[0] * 16)]]
    now, was = w.views(w.pool), w.views(pool)
    s = slots[(slots >= 0) & (slots < w.k.shape[0] * 16)]
    assert stored.shape[0] == t - 2
    for a, b in zip(now, was):
        assert torch.equal(a[s // 16, s % 16], b[s // 16, s % 16])


def test_a_position_outside_the_table_gives_nan_queries_and_stores_nothing():
    w = World(6, 2, 1, 64, 4, "bf16", "tokens", True, 64, False, seed=6)
    w.slots = torch.arange(6)
    w.pos[1], w.pos[4] = -1, 500
    before = w.pool.cpu().clone()
    q_out = torch.zeros(w.q.shape, dtype=torch.bfloat16, device=DEV)
    w.call(q_out)
    torch.cuda.synchronize()
    bad = np.array([1, 4])
    got = q_out.cpu().float().numpy()
    assert np.all(np.isnan(got[bad])) and np.all(np.isfinite(np.delete(got, bad, 0)))
    now = w.k.cpu().reshape(-1, 1, 64)
    assert torch.equal(now[bad], before[:, 0].reshape(-1, 1, 64)[bad])


def test_nan_infinite_and_large_values():
    """NaN stays NaN in its own head only; values past 448 * scale are limited in an 8-bit cache."""
    w = World(4, 2, 2, 64, 4, "e4m3", "tokens", False, 0, False, seed=7)
    w.slots = torch.arange(4)
    w.nv[0, 0, 5] = float("nan")
    w.nv[1, 1, 6] = float("inf")
    w.nv[2, 0, 7] = -3.0e38
    w.nv[3, 1, 8] = 1e-30
    q_out = torch.zeros(w.q.shape, dtype=torch.bfloat16, device=DEV)
    w.call(q_out)
    torch.cuda.synchronize()
    got = w.v.cpu().reshape(-1, 2, 64)[:4].view(torch.float8_e4m3fn).float().numpy()
    assert np.isnan(got[0, 0, 5]) and np.isnan(got).sum() == 1
    assert got[1, 1, 6] == 448 and got[2, 0, 7] == -448 and got[3, 1, 8] == 0


def test_every_bf16_value_is_stored_as_it_is():
    """Values pass to a BF16 cache unchanged, bit for bit but for the kind of a NaN."""
    d, hkv = 256, 2
    pats = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    tokens = pats.size // (hkv * d)
    w = World(tokens, 1, hkv, d, 16, "bf16", "tokens", True, 256, False, seed=8)
    w.slots = torch.arange(tokens)
    w.nv = torch.from_numpy(pats.view(np.int16).copy()).view(tokens, hkv, d).to(DEV)
    w.call(torch.empty(w.q.shape, dtype=torch.bfloat16, device=DEV))
    torch.cuda.synchronize()
    got = w.v.cpu().reshape(-1, hkv, d)[:tokens].contiguous().numpy().view(np.uint16).reshape(-1)
    nan = (pats & 0x7FFF) > 0x7F80
    assert np.array_equal(got[~nan], pats[~nan]) and np.all((got[nan] & 0x7FFF) > 0x7F80)


def test_captured_and_replayed_on_a_side_stream():
    w = World(65, 8, 2, 128, 16, "bf16", "tokens", True, 128, False, seed=9)
    dcs, pos, slots = torch.from_numpy(w.cs).to(DEV), w.pos.to(DEV), w.slots.to(DEV)
    q_out = torch.empty(w.q.shape, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        decode.qkv_rope_store(w.cache, w.q, w.nk, w.nv, pos, dcs, slots, q_out, w.wq, w.wk)
    for k in range(3):
        w.fused.copy_(bf16(tuple(w.fused.shape), torch.Generator().manual_seed(50 + k), 2.0))
        before, fused = w.pool.cpu().clone(), w.fused.cpu().clone()
        g.replay()
        w.check(q_out, before, fused)


def test_refused_call_leaves_everything_untouched():
    w = World(4, 2, 2, 64, 4, "bf16", "tokens", True, 64, False, seed=10)
    before = w.pool.cpu().clone()
    q_out = torch.full(w.q.shape, 3.0, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(x.XferError):
        decode.qkv_rope_store(w.cache, w.q, w.nk, w.nv, w.pos.to(DEV), torch.from_numpy(w.cs).to(DEV),
                              w.slots.to(DEV), q_out, eps=-1.0)
    torch.cuda.synchronize()
    assert torch.equal(w.pool.cpu(), before) and bool((q_out == 3.0).all())
