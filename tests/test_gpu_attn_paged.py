"""GPU: attention of one new token over a paged cache (xfer_attn_paged)
against the formula in 64 bits.  Every slot that no row sees holds NaN, pages
are shuffled, and the bytes around the output are compared."""
import numpy as np
import pytest
import torch

import bf16_wire_all_amd as x
from bf16_wire_all_amd import decode
from tests import decode_reference as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAN16, NAN8 = 0x7FC0, 0x7F


class World:
    def __init__(self, lens, hq, hkv, d, page, kind="bf16", order="tokens", window=0, sinks=0, out="bf16", seed=1,
                 max_len=None, holes=(), sharp=1.5, gap_pages=2):
        """holes: (row, page of the row) pairs whose page number is out of the cache."""
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hq, self.hkv, self.d, self.page, self.kind = list(lens), hq, hkv, d, page, kind
        self.window, self.sinks, self.rows = window, sinks, len(self.lens)
        self.max_len = max_len or max(max(self.lens), 1)
        used = [-(-n // page) for n in self.lens]
        n_pages = sum(used) + gap_pages
        width = max(1, -(-self.max_len // page), max(used))
        perm = torch.randperm(n_pages, generator=g)
        table = torch.full((self.rows, width + 1), 0x7FFFFFFF, dtype=torch.int32)  # past a row: never a page
        at = 0
        for r, n in enumerate(used):
            table[r, :n] = perm[at:at + n].int()
            at += n
        for r, p in holes:
            table[r, p] = -1 if (r + p) % 2 else n_pages
        self.table = table[:, :width].to(DEV)                # rows width + 1 apart
        shape = (n_pages, page, hkv, d) if order == "tokens" else (n_pages, hkv, page, d)
        kv = []
        seen = torch.zeros((n_pages, page), dtype=torch.bool)
        self.at = []                                          # (page, slot) of each row's visible tokens
        for r, n in enumerate(self.lens):
            j = ref.visible(min(n, self.max_len), window, sinks)
            keep = [t for t in j if (r, t // page) not in set(holes)]
            j = np.array(keep, dtype=int)
            pages, slots = table[r][torch.from_numpy(j // page)].long(), torch.from_numpy(j % page)
            seen[pages, slots] = True
            self.at.append((pages, slots))
        for _ in range(2):
            a = torch.randn(shape, generator=g)
            a = a.to(torch.bfloat16) if kind == "bf16" else a.to(torch.float8_e4m3fn)
            bits = a.view(torch.int16 if kind == "bf16" else torch.uint8)
            bits = bits.transpose(1, 2) if order == "heads" else bits
            bits[~seen] = NAN16 if kind == "bf16" else NAN8
            kv.append(bits)
        self.k, self.v = kv
        self.ks = self.vs = None
        if kind == "e4m3":
            self.ks, self.vs = torch.rand(hkv, generator=g) + 0.25, torch.rand(hkv, generator=g) + 0.25
        dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        if order == "heads":
            self.dk, self.dv = (t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) for t in kv)
        else:
            self.dk, self.dv = dev(self.k.contiguous()), dev(self.v.contiguous())
        self.cache = decode.kv_cache(self.dk, self.dv, dev(self.ks), dev(self.vs))
        fused = (torch.randn((self.rows, (hq + 2) * d), generator=g) * sharp).to(torch.bfloat16)
        self.q = fused[:, :hq * d].view(self.rows, hq, d)
        self.dq = fused.to(DEV)[:, :hq * d].view(self.rows, hq, d)
        self.dlens = torch.tensor(self.lens, dtype=torch.int32).to(DEV)
        self.scale = d ** -0.5
        self.out_dtype = torch.bfloat16 if out == "bf16" else torch.float32
        self.out_kind = out

    def workspace(self):
        n = decode.attn_workspace_bytes(self.cache, self.rows, self.hq, self.max_len, self.window, self.sinks)
        return torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=DEV), n

    def call(self, out, ws, stream=None):
        decode.attn_paged(self.cache, self.dq, self.table, self.dlens, self.max_len, self.scale, out, ws,
                          window=self.window, sinks=self.sinks, stream=stream)

    def want(self):
        outs, tols = [], []
        for r in range(self.rows):
            pages, slots = self.at[r]
            kv = []
            for bits, scale in ((self.k, self.ks), (self.v, self.vs)):
                a = bits[pages, slots].contiguous()
                a = a.view(torch.bfloat16 if self.kind == "bf16" else torch.float8_e4m3fn).float().numpy()
                a = a.astype(np.float64)
                kv.append(a if scale is None else a * scale.numpy().astype(np.float64)[:, None])
            o, t = ref.attention(self.q[r].float().numpy().astype(np.float64), kv[0], kv[1], self.scale)
            outs.append(o)
            tols.append(t)
        o, t = np.stack(outs), np.stack(tols)
        return o, t * (1 + ref.HALF[self.out_kind]) + ref.HALF[self.out_kind] * np.abs(o)

    def check(self, got):
        o, tol = self.want()
        got = got.cpu().float().numpy().astype(np.float64)
        off = np.abs(got - o)
        assert np.all(np.isfinite(got)), "a value that no row sees came through"
        assert np.all(off <= tol), (float(np.max(off / np.maximum(tol, 1e-300))), np.argwhere(off > tol)[:4])


def run(w, calls=1):
    say("attn_paged", w.rows, w.lens[:4], w.hq, w.hkv, w.d, w.page, w.kind, w.window, w.sinks)
    pad = torch.full((w.rows, w.hq + 1, w.d), 5.0, dtype=w.out_dtype, device=DEV)
    out = pad[:, :w.hq]
    ws, n = w.workspace()
    for _ in range(calls):
        w.call(out, ws[:n] if n else None)
        torch.cuda.synchronize()
        w.check(out)
    assert bool((pad[:, w.hq:] == 5.0).all()), "write past a row of the output"
    assert bool((ws[n:] == 0xFF).all()), "write past the workspace"
    return out


EDGE = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_lengths_about_every_tile_edge(d, kind):
    run(World(EDGE, 4, 2, d, 16, kind, "heads", seed=d))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (10, 2), (16, 1), (17, 1), (40, 8), (64, 2), (80, 2), (33, 1)])
@pytest.mark.parametrize("d,kind", [(64, "bf16"), (128, "e4m3"), (256, "bf16")])
def test_head_groups(hq, hkv, d, kind):
    run(World([1, 40, 513], hq, hkv, d, 32, kind, "tokens", seed=hq, out="f32"))


@pytest.mark.parametrize("page", [1, 2, 4, 8, 64, 256])
@pytest.mark.parametrize("order", ["tokens", "heads"])
def test_page_sizes(page, order):
    run(World([700, 3, 129, 511], 8, 2, 128, page, "bf16", order, seed=page))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (33, 0), (100, 4), (256, 5), (512, 64), (5000, 4), (31, 200)])
def test_window_and_first_tokens(window, sinks):
    lens = [0, 1, 5, 34, 35, 100, 104, 105, 260, 261, 262, 700, 1500]
    run(World(lens, 6, 2, 64, 16, "bf16", "tokens", window, sinks, seed=window + sinks))
    run(World(lens, 6, 2, 128, 8, "e4m3", "heads", window, sinks, out="f32", seed=window + sinks))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_long_rows_in_pieces(kind, out):
    w = World([9000, 1, 4097, 0, 8191], 10, 2, 128, 16, kind, "heads", out=out, seed=3)
    assert w.workspace()[1] > 0
    run(w, calls=2)


@pytest.mark.parametrize("d,kind", [(64, "bf16"), (128, "e4m3"), (256, "bf16")])
def test_fewer_units_than_workgroups(d, kind):
    """The grid is laid out for rows of max_len: shorter rows leave workgroups that must find nothing to do."""
    run(World([0, 3, 700, 1, 0], 4, 2, d, 16, kind, max_len=16000, seed=15))
    run(World([1], 4, 1, d, 16, kind, max_len=130000, seed=16))
    run(World(EDGE, 4, 2, d, 16, kind, "heads", max_len=5000, seed=d))


def test_many_short_rows_and_one_long():
    run(World([1 + 7 * i % 60 for i in range(200)] + [3000], 4, 1, 64, 16, seed=4))


@pytest.mark.parametrize("d,kind", [(64, "e4m3"), (128, "bf16")])
def test_more_rows_than_threads(d, kind):
    """Rows beyond one for each thread of a workgroup, in runs and as a whole."""
    lens = [(i * 37) % 90 for i in range(701)]
    run(World(lens, 2, 1, d, 16, kind, seed=17))
    lens[300] = 9000
    run(World(lens, 2, 1, d, 16, kind, seed=18))


@pytest.mark.parametrize("d,kind,hq,hkv,top", [(64, "e4m3", 8, 2, 1100), (64, "bf16", 20, 1, 700), (128, "e4m3", 5, 1, 700),
                                              (128, "bf16", 24, 1, 380), (256, "e4m3", 4, 2, 380)])
def test_a_whole_row_to_each_compute_unit(d, kind, hq, hkv, top):
    """Few rows of middling length: no row is cut up, and more waves share it."""
    lens = [top, 0, 1, 129, 255, 256, 257, top - 1]
    w = World(lens, hq, hkv, d, 16, kind, seed=19, out="f32" if hq == 5 else "bf16")
    assert w.workspace()[1] == 0
    run(w, calls=2)
    w = World([9000, 40, 5000], hq, hkv, d, 32, kind, "heads", window=top - 3, sinks=3, seed=20)
    assert w.workspace()[1] == 0
    run(w)
    run(World(lens, hq, hkv, d, 16, kind, holes=[(0, 0), (0, 9), (7, 3), (6, 15), (6, 16)], seed=21))


@pytest.mark.parametrize("d,kind,hq,hkv,out", [(64, "e4m3", 8, 4, "bf16"), (64, "bf16", 6, 2, "f32"), (128, "e4m3", 16, 8, "f32"),
                                              (128, "bf16", 12, 12, "bf16"), (128, "bf16", 40, 2, "f32"),
                                              (64, "e4m3", 132, 4, "bf16"), (256, "e4m3", 12, 4, "f32"),
                                              (256, "e4m3", 40, 2, "bf16")])
def test_heads_side_by_side(d, kind, hq, hkv, out):
    """Tokens whose heads lie one after the other, under a bound that a large batch would need."""
    lens = [3000, 0, 1, 31, 32, 33, 127, 700, 2, 1025]
    bound = 100 * 2 ** 20 // (len(lens) * hkv * d * (2 if kind == "bf16" else 1) * 2) + 1000
    w = World(lens, hq, hkv, d, 16, kind, seed=22, max_len=bound, out=out)
    assert w.workspace()[1] > 0
    run(w, calls=2)
    run(World(lens, hq, hkv, d, 8, kind, seed=23, max_len=bound, out=out, holes=[(0, 3), (7, 0), (7, 87), (9, 127), (9, 128)]))
    lens = [9000] + lens
    run(World(lens, hq, hkv, d, 16, kind, seed=24, max_len=2 * bound, window=5000, sinks=33, out=out))


def test_lengths_below_the_bound_and_above_it():
    """max_len is a bound: shorter rows are served, longer ones are cut to it."""
    run(World([10, 500, 999], 4, 2, 64, 16, max_len=40000, seed=5))
    run(World([10, 500, 999], 4, 2, 64, 16, max_len=400, seed=5))


def test_holes_are_not_visible():
    """Page numbers past the cache, whole rows of them included: zeros where nothing is left."""
    holes = [(0, 0), (1, 1), (1, 2), (2, 0), (2, 1), (2, 2), (3, 5)]
    w = World([20, 64, 48, 500], 4, 2, 128, 16, holes=holes, seed=6)
    out = run(w)
    assert bool((out[2] == 0).all())
    run(World([40, 64, 48, 500], 4, 2, 64, 16, "e4m3", holes=holes, window=300, sinks=2, seed=6))


def test_zero_rows_are_zeros_also_in_pieces():
    for lens in ([0, 0, 0], [0, 20000, 0]):
        out = run(World(lens, 8, 2, 128, 16, seed=7))
        assert bool((out[0] == 0).all()) and bool((out[2] == 0).all())


def test_sharp_scores_and_a_late_maximum():
    """Scores of hundreds, and a key that passes all before it by far at the end of the row."""
    w = World([1000, 300], 4, 1, 128, 16, sharp=40.0, out="f32", seed=8)
    run(w)
    for r in range(2):
        p, s = w.at[r][0][-1], w.at[r][1][-1]
        w.k[p, s] = (w.q[r, :1].float() * 3).to(torch.bfloat16).view(torch.int16)
    w.dk.copy_(w.k)
    run(w)


def test_a_nan_that_is_seen_reaches_its_heads_alone():
    w = World([40, 600], 4, 2, 64, 16, seed=9)
    p, s = w.at[1][0][7], w.at[1][1][7]
    w.dv[p, s, 1, 3] = NAN16
    out = torch.empty((2, 4, 64), dtype=torch.bfloat16, device=DEV)
    ws, n = w.workspace()
    w.call(out, ws)
    torch.cuda.synchronize()
    bad = torch.isnan(out.cpu().float())
    want = torch.zeros_like(bad)
    want[1, 2:, 3] = True
    assert torch.equal(bad, want)


def test_offsets_past_32_bits():
    """Pages up to 12 GB into the keys' buffer (most of it is never touched)."""
    d, page, hkv = 128, 16, 2
    row = page * hkv * d
    stride = 1 << 23                                       # elements between pages: 16 MiB
    pool = torch.empty(800 * stride, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(10)
    used = [799, 3, 300, 512]
    k = pool.as_strided((800, page, hkv, d), (stride, hkv * d, d, 1))
    v = pool.as_strided((800, page, hkv, d), (stride, hkv * d, d, 1), storage_offset=2 * row)
    w = World([60], 4, hkv, d, page, seed=10)
    for i, p in enumerate(used):
        for view, host in ((k, w.k), (v, w.v)):
            host_page = int(w.table[0, i])
            view[p].copy_(host[host_page].view(torch.bfloat16))
    say("attn_paged, offsets past 32 bits")
    out = torch.empty((1, 4, d), dtype=torch.bfloat16, device=DEV)
    table = torch.tensor([used], dtype=torch.int32, device=DEV)
    decode.attn_paged(decode.kv_cache(k, v), w.dq, table, w.dlens, 60, w.scale, out, None)
    torch.cuda.synchronize()
    w.check(out)
    # and the store writes there
    q = torch.zeros((1, 0, d), dtype=torch.bfloat16, device=DEV)
    new = torch.randn((1, hkv, d), generator=g).to(torch.bfloat16).to(DEV)
    decode.qkv_rope_store(decode.kv_cache(k, v), q, new, new * 2, None, None,
                          torch.tensor([799 * page + 15], device=DEV), q)
    torch.cuda.synchronize()
    assert torch.equal(k[799, 15], new[0]) and torch.equal(v[799, 15], new[0] * 2)


def test_captured_and_replayed_with_other_lengths():
    w = World([100, 3000, 7], 8, 2, 128, 16, seed=11, max_len=5000)
    ws, n = w.workspace()
    out = torch.empty((3, 8, 128), dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w.call(out, ws[:n])
    whole = (w.lens, w.at)
    for lens in ([100, 3000, 7], [1, 2999, 0], [99, 130, 6], [100, 3000, 7]):
        w.lens = lens
        w.at = [(p[:m], q[:m]) for (p, q), m in zip(whole[1], lens)]
        w.dlens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        w.check(out)
        eager = torch.empty_like(out)
        w.call(eager, ws[:n])
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_two_streams_with_workspaces_of_their_own():
    a, b = World([9000, 20], 8, 2, 128, 16, seed=12), World([300, 7000], 8, 2, 128, 16, seed=13)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty((2, 8, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    wss = [w.workspace()[0] for w in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for w, s, o, ws in zip((a, b), streams, outs, wss):
            w.call(o, ws, stream=s)
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])


def test_refused_call_leaves_the_output_untouched():
    w = World([9000], 8, 2, 128, 16, seed=14)
    out = torch.full((1, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(x.XferError):
        w.call(out, None)                                  # rows in pieces need a workspace
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())
