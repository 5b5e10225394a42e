"""GPU: attention of rows with shared prefixes (xfer_attn_shared) against the
formula in 64 bits, every row by itself.  Every slot that no row reads holds
NaN, the page numbers of shared tokens are out of range in all rows but a
group's first, and the bytes around the output are compared."""
import numpy as np
import pytest
import torch

import bf16_wire_all_amd as x
from bf16_wire_all_amd import decode
from tests import decode_reference as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAN = {"bf16": 0x7FC0, "e4m3": 0x7F}
# of a softmax weight in the product: two BF16 numbers are off by up to 2^-17 of it, three hold it whole
SPLIT = {"bf16": 2.0 ** -17, "f32": 0.0}
HOLE = 0x7FFFFFFF


class World:
    """groups: a list of (shared tokens, [each row's length]); a list alone: rows outside every group."""

    def __init__(self, groups, hq, hkv, d, page=16, kind="bf16", order="tokens", out="bf16", seed=1, holes=(), sharp=1.5,
                 max_len=None, starts=None, shared=None, same_pages=False):
        g = torch.Generator().manual_seed(seed)
        self.hq, self.hkv, self.d, self.page, self.kind, self.out_kind = hq, hkv, d, page, kind, out
        rows, first, given = [], [0], []
        for item in groups:                      # (group's first row, shared tokens of the row, length)
            p, lens = item if isinstance(item, tuple) else (0, item)
            lead = len(rows)
            p_used = min(p, lens[0]) if len(lens) > 1 else 0
            rows += [(lead, p_used if n >= p_used else 0, n) for n in lens]
            first.append(len(rows))
            given.append(p)
        self.rows, self.n = rows, len(rows)
        self.max_len = max_len or max(max(n for _, _, n in rows), 1)
        width = -(-self.max_len // page)
        table = torch.full((self.n, width + 1), HOLE, dtype=torch.int64)
        count = 0
        for r, (lead, p, n) in enumerate(rows):
            a = 0 if r == lead or p == 0 else p // page       # its own pages; of shared ones the first row's alone are valid
            if same_pages and r != lead:
                a = -(-min(rows[lead][2], n) // page)
                table[r, :a] = table[lead, :a]
            b = -(-n // page)
            if b > a:
                table[r, a:b] = torch.arange(count, count + b - a)
                count += b - a
        n_pages = count + 2
        perm = torch.randperm(n_pages, generator=g)
        table = torch.where(table == HOLE, HOLE, perm[table.clamp(max=n_pages - 1)])
        for r, pg in holes:
            table[r, pg] = n_pages + r
        self.n_pages = n_pages
        seen = torch.zeros((n_pages, page), dtype=torch.bool)
        self.at = []
        for r, (lead, p, n) in enumerate(rows):
            j = torch.arange(n)
            pages = torch.where(j < p, table[lead, j // page], table[r, j // page])
            keep = pages < n_pages
            pages, slots = pages[keep], (j % page)[keep]
            seen[pages, slots] = True
            self.at.append((pages, slots))
        shape = (n_pages, page, hkv, d) if order == "tokens" else (n_pages, hkv, page, d)
        kv = []
        for _ in range(2):
            a = torch.randn(shape, generator=g).to(torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
            bits = a.view(torch.int16 if kind == "bf16" else torch.uint8)
            bits = bits.transpose(1, 2) if order == "heads" else bits
            bits[~seen] = NAN[kind]
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
        fused = (torch.randn((self.n, (hq + 2) * d), generator=g) * sharp).to(torch.bfloat16)
        self.q = fused[:, :hq * d].view(self.n, hq, d)
        self.dq = fused.to(DEV)[:, :hq * d].view(self.n, hq, d)
        self.table = table.to(torch.int32).to(DEV)[:, :width]
        self.lens = torch.tensor([n for _, _, n in rows], dtype=torch.int32, device=DEV)
        self.starts = torch.tensor(first if starts is None else starts, dtype=torch.int32, device=DEV)
        self.shared = torch.tensor(given if shared is None else shared, dtype=torch.int32, device=DEV)
        self.scale = d ** -0.5
        self.dtype = torch.bfloat16 if out == "bf16" else torch.float32
        need = decode.attn_shared_workspace_bytes(self.cache, self.n, len(self.shared), hq, self.max_len)
        assert need > 0
        self.need = need
        self.ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)

    def values(self, bits, scale, r):
        pages, slots = self.at[r]
        a = bits[pages, slots].contiguous().view(torch.bfloat16 if self.kind == "bf16" else torch.float8_e4m3fn)
        a = a.float().numpy().astype(np.float64)
        return a if scale is None else a * scale.numpy().astype(np.float64)[:, None]

    def want(self, r):
        """A row's results, and how far binary32 with one rounding may be from them."""
        k, v = self.values(self.k, self.ks, r), self.values(self.v, self.vs, r)
        q, group = self.q[r].float().numpy().astype(np.float64), self.hq // self.hkv
        out, tol = ref.attention(q, k, v, self.scale)
        for h in range(self.hq if len(k) else 0):
            s = k[:, h // group] @ q[h] * self.scale
            p = np.exp(s - s.max())
            p /= p.sum()
            # ref.attention counts 2^-18 for the split, in the numerator twice and in the quotient once
            tol[h] += (SPLIT[self.out_kind] - 2.0 ** -18) * (2 * (p @ np.abs(v[:, h // group])) + np.abs(out[h]))
        return out, tol * (1 + ref.HALF[self.out_kind]) + ref.HALF[self.out_kind] * np.abs(out)

    def buffer(self):
        """[rows, heads, d] within rows 8 elements longer, full of marks."""
        size = 2 if self.out_kind == "bf16" else 4
        row = self.hq * self.d + 8
        raw = torch.full((self.n, row * size), 0x5A, dtype=torch.uint8, device=DEV)
        return raw, raw.view(self.dtype)[:, :self.hq * self.d].unflatten(1, (self.hq, self.d))

    def call(self, out, stream=None):
        decode.attn_shared(self.cache, self.dq, self.table, self.lens, self.max_len, self.starts, self.shared, self.scale,
                           out, self.ws[:self.need], stream=stream)

    def run(self, rows=None, calls=1):
        raw, out = self.buffer()
        for i in range(calls):
            self.call(out)
            torch.cuda.synchronize()
            got = out.cpu().double().numpy()
            if i:
                assert np.array_equal(got, first, equal_nan=True)
            first = got
        assert (raw.cpu()[:, -8 * (2 if self.out_kind == "bf16" else 4):] == 0x5A).all()
        assert (self.ws[self.need:] == 0xFF).all()
        for r in range(self.n) if rows is None else rows:
            o, tol = self.want(r)
            off = np.abs(got[r] - o) - tol
            assert not np.isnan(got[r]).any(), f"row {r}: NaN"
            assert off.max() <= 0, f"row {r} {self.rows[r]}: off by {np.abs(got[r] - o).max()}, {off.max()} more than allowed"
        return got


RAGGED = [(300, [301, 420, 300, 333, 305]), [77], (64, [64, 65, 200]), (1, [1, 2, 9]), [0, 5]]
KINDS = [("bf16", "tokens"), ("bf16", "heads"), ("e4m3", "tokens"), ("e4m3", "heads")]


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 5, 1), (128, 16, 8), (256, 6, 2), (64, 40, 2), (128, 34, 1), (256, 20, 1)])
@pytest.mark.parametrize("kind,order", KINDS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_ragged_groups(d, hq, hkv, kind, order, out):
    say("ragged", d, hq, hkv, kind, order, out)
    World(RAGGED, hq, hkv, d, 16, kind, order, out, seed=d + hq).run(calls=2)


@pytest.mark.parametrize("page", [1, 2, 4, 8, 32, 64, 1024])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_pages(page, kind):
    """Shared tokens that end within a page: the first row's page holds them, the others' rows go on in their own."""
    say("pages", page, kind)
    World([(130, [150, 131, 130, 300]), (63, [63, 64, 70]), (1000, [1000, 1003])], 8, 2, 128, page, kind, "heads").run()


@pytest.mark.parametrize("rows,heads,d", [(2, 1, 128), (33, 1, 64), (40, 4, 128), (130, 1, 128), (17, 8, 64), (48, 5, 128),
                                          (24, 16, 256), (65, 2, 256), (100, 3, 128)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_many_rows_of_one_group(rows, heads, d, kind, out):
    say("rows", rows, heads, d, kind, out)
    p = 700
    lens = [p + (i * 7) % 50 for i in range(rows)]
    World([(p, lens)], 2 * heads, 2, d, 16, kind, "heads", out, seed=rows).run(rows=sorted({0, 1, 31 % rows, 32 % rows, rows // 2, rows - 1}))


@pytest.mark.parametrize("p", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 4097, 20000])
@pytest.mark.parametrize("rows", [3, 50])
def test_prefix_lengths(p, rows):
    say("prefix", p, rows)
    World([(p, [p + i % 3 for i in range(rows)])], 8, 2, 128, 16, "bf16", "heads", "f32", seed=p).run(rows=[0, 1, 2, rows - 1])


def test_long_shared_tokens_of_few_and_of_many_rows():
    say("long")
    World([(60000, [60000, 60400]), (30000, [30000 + i for i in range(40)]), [1, 3000]], 8, 1, 128, 16, "bf16", "heads",
          seed=5).run(rows=[0, 1, 2, 25, 41, 42, 43])


def test_drafted_positions():
    """Rows of one request: the same pages to the end, lengths one apart."""
    groups = [(n, [n + i for i in range(m)]) for n, m in ((500, 4), (1000, 5), (17, 4), (64, 3))]
    for kind in ("bf16", "e4m3"):
        say("drafted", kind)
        World(groups, 40, 8, 128, 16, kind, "heads", same_pages=True).run()


def test_a_shared_token_is_read_from_the_first_row_s_page_alone():
    """Rows whose own pages of the shared tokens hold other numbers give what the first row's pages say."""
    w = World([(100, [150, 160, 170])], 8, 2, 128, 16)
    first = w.run()
    w.table[1:, :6] = w.table[0, 6]          # valid pages, and the wrong ones
    assert np.array_equal(w.run(), first)


def test_rows_that_do_not_see_all_shared_tokens_read_theirs_alone():
    say("short rows")
    World([(200, [230, 199, 0, 200, 1, 450])], 8, 2, 128, 16).run()
    # the first row's length limits what is shared
    World([(500, [90, 600, 90, 89, 0])], 8, 2, 128, 16).run()
    World([(500, [0, 600, 20])], 8, 2, 128, 16).run()


def test_lengths_above_max_len_and_numbers_past_the_rows():
    groups = [(48, [64, 64, 64]), [64]]
    w = World(groups, 4, 2, 64, 16, max_len=64)
    want = w.run()
    w.lens = torch.tensor([64, -1, 70, 1 << 30], dtype=torch.int32, device=DEV)   # cut to max_len
    assert np.array_equal(w.run(), want)
    for starts, shared in (([0, 3, 9], [48, 7]), ([0, 3, -1], [48, 0]), ([0, 3, 1], [48, 30]), ([0, 3, 3], [48, 5]),
                           ([0, 3, 2], [48, 1 << 30])):
        w.starts, w.shared = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in (starts, shared))
        say("starts", starts, shared)
        assert np.array_equal(w.run(), want), starts


def test_any_numbers_stay_within_the_buffers():
    """Random starts and shared counts, over rows whose tables are all the same: each row gives its own result."""
    rng = np.random.default_rng(2)
    n = 40
    w = World([(160, [160 + i % 5 for i in range(n)])], 8, 2, 64, 16, same_pages=True, out="f32")
    w.table[:, :10] = w.table[0, :10]
    groups = 25
    w.need = decode.attn_shared_workspace_bytes(w.cache, n, groups, 8, w.max_len)
    w.ws = torch.full((w.need + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    for i in range(6):
        starts = rng.integers(-3, n + 5, groups + 1)
        w.starts = torch.tensor(np.sort(starts) if i % 2 else starts, dtype=torch.int32, device=DEV)
        w.shared = torch.tensor(rng.integers(0, 161, groups), dtype=torch.int32, device=DEV)
        say("any", i)
        w.run(rows=range(0, n, 3))


def test_any_numbers_of_many_rows_stay_within_the_buffers():
    """More rows than a workgroup plans for itself: starts, prefixes and lengths without sense read and write nothing else."""
    w = World([(40, [50, 60])] * 100 + [(300, [310] * 60)] + [[30]] * 40, 8, 2, 64, 16, "bf16", "tokens")
    raw, out = w.buffer()
    g = torch.Generator().manual_seed(6)
    for i in range(8):
        w.starts.copy_(torch.randint(-2 ** 31, 2 ** 31, w.starts.shape, generator=g, dtype=torch.int64).int() if i % 2 else
                       torch.randint(0, 400, w.starts.shape, generator=g).int())
        w.shared.copy_(torch.randint(-2 ** 31, 2 ** 31, w.shared.shape, generator=g, dtype=torch.int64).int() if i % 3 else
                       torch.randint(0, 320, w.shared.shape, generator=g).int())
        w.lens.copy_(torch.randint(0, 2 ** 31, w.lens.shape, generator=g, dtype=torch.int64).int() if i == 7 else
                     torch.randint(0, 320, w.lens.shape, generator=g).int())
        say("any numbers of many rows", i)
        w.call(out)
        torch.cuda.synchronize()
        assert (raw.cpu()[:, -16:] == 0x5A).all() and (w.ws[w.need:] == 0xFF).all()


@pytest.mark.parametrize("rows", [40, 300])
def test_two_graphs_that_share_a_workspace(rows):
    worlds = [World([(500 + 90 * s, [600 + i % 50 for i in range(rows)])], 8, 2, 128, 16, seed=s, max_len=660) for s in (1, 2)]
    worlds[1].ws = worlds[0].ws
    outs, graphs, want = [w.buffer()[1] for w in worlds], [], []
    for w, o in zip(worlds, outs):
        w.call(o)
        torch.cuda.synchronize()
        want.append(o.clone())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            w.call(o)
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].fill_(3)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])


def few_and_many(group, rows):
    """Groups of up to 16, 17 to 32 and more query heads, one that is shorter than a tile, and rows alone up to `rows`."""
    groups = [(200, [200 + i for i in range(n)]) for n in (2, -(-17 // group), -(-33 // group), -(-150 // group)) if n > 1]
    groups += [(7, [9, 8]), (1500, [1501, 1999, 1500])]
    n = sum(len(lens) for _, lens in groups)
    return groups + [[i % 70] for i in range(rows - n)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_every_way_through(d, kind, out):
    """Few rows and more than a workgroup plans for itself; no group, groups of few and of many query heads; heads of a row past 16."""
    for group, rows, alone in ((4, 2, False), (5, 4, False), (2, 260, True), (20, 257, True), (3, 254, False), (3, 255, False),
                               (9, 100, False), (20, 300, False), (1, 600, False)):
        say("ways", d, kind, out, group, rows, alone)
        if alone:
            w = World([[1 + 37 * i % 150] for i in range(rows)], 2 * group, 2, d, 16, kind, "tokens", out, starts=[0], shared=[])
        elif rows <= 4:
            w = World([(300, [301] * rows)], 2 * group, 2, d, 16, kind, "tokens", out)
        else:
            w = World(few_and_many(group, rows), 2 * group, 2, d, 16, kind, "tokens", out)
        w.run(rows=sorted({*range(0, w.n, 1 + w.n // 12), w.n - 1}))


def test_very_many_groups():
    say("4096 groups")
    groups = [(20, [21, 20])] * 700 + [(0, [3])] * 3000 + [(5, [6, 7])] * 396
    assert len(groups) == 4096
    World(groups, 2, 1, 64, 16).run(rows=list(range(0, 1400, 97)) + list(range(1400, 5192, 411)))


def test_no_groups_is_attention_of_one_token():
    w = World([[100], [3000], [0], [17]], 8, 2, 128, 16, out="f32")
    w.starts, w.shared = w.starts[:1], w.shared[:0]
    w.run()
    w.starts, w.shared = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV)
    w.run()


def test_holes_among_shared_and_own_tokens():
    for kind in ("bf16", "e4m3"):
        say("holes", kind)
        w = World([(320, [400, 330, 500]), (64, [64, 70]), [33]], 8, 2, 128, 16, kind,
                  holes=[(0, 3), (0, 19), (1, 20), (2, 31), (3, 0), (3, 1), (3, 2), (3, 3), (5, 0), (5, 1), (5, 2)])
        got = w.run()
        assert (got[3] == 0).all() and (got[5] == 0).all()       # nothing to see


@pytest.mark.parametrize("rows", [3, 70])
def test_numbers_that_are_not_finite(rows):
    """A value's infinity or NaN reaches its dim of every row that sees it, a score's its head, and no other row."""
    w = World([(300, [300 + i for i in range(rows)]), [40]], 4, 2, 128, 16, out="f32")
    clean = w.run(rows=[0, rows])
    def put(t, token, head, dim, bits, row=0):
        pages, slots = w.at[row]
        t[int(pages[token]), int(slots[token]), head, dim] = int(np.uint16(bits).view(np.int16))
    put(w.dv, 7, 0, 5, 0x7F80)
    put(w.dv, 8, 0, 6, 0xFF80)
    put(w.dv, 200, 1, 7, 0x7F80), put(w.dv, 201, 1, 7, 0xFF80)
    put(w.dv, 9, 1, 9, 0x7FC0)
    put(w.dv, 300, 0, 11, 0x7F80, row=1)                         # a token of row 1 alone
    put(w.dv, 301, 1, 12, 0x7FC0, row=2)                         # and of row 2
    _, out = w.buffer()
    say("not finite", rows)
    w.call(out)
    got = out.cpu().double().numpy()
    bad = np.zeros(got.shape, bool)
    assert (got[:rows, :2, 5] == np.inf).all() and (got[:rows, :2, 6] == -np.inf).all()
    assert np.isnan(got[:rows, 2:, 7]).all() and np.isnan(got[:rows, 2:, 9]).all()
    assert (got[1, :2, 11] == np.inf).all() and np.isnan(got[2, 2:, 12]).all()
    bad[:rows, :2, 5:7] = bad[:rows, 2:, 7] = bad[:rows, 2:, 9] = bad[1, :2, 11] = bad[2, 2:, 12] = True
    assert np.isfinite(got[~bad]).all()
    for r in (0, rows):
        assert np.array_equal(got[r][~bad[r]], clean[r][~bad[r]])
    # a score of NaN or +inf makes its head NaN in every row, one of -inf takes its token out
    w = World([(300, [300 + i for i in range(rows)]), [40]], 4, 2, 128, 16, out="f32")
    put(w.dk, 3, 0, 0, 0x7FC0)
    _, out = w.buffer()
    w.call(out)
    got = out.cpu().double().numpy()
    assert np.isnan(got[:rows, :2]).all() and np.isfinite(got[:rows, 2:]).all() and np.isfinite(got[rows]).all()
    w = World([(300, [300 + i for i in range(rows)]), [40]], 4, 2, 128, 16, out="f32")
    put(w.dk, 3, 1, 0, 0x7F80)
    w.dq[:, 2:, 0] = -1.0
    w.q[:, 2:, 0] = -1.0
    w.dq[0, 2, 0] = 1.0                                          # +inf for this one
    w.q[0, 2, 0] = 1.0
    raw, out = w.buffer()
    w.call(out)
    got = out.cpu().double().numpy()
    assert np.isnan(got[0, 2]).all()
    w.k[w.at[0][0][3], w.at[0][1][3], 1] = 0                     # the same without the token
    w.at = [(torch.cat([p[:3], p[4:]]), torch.cat([s[:3], s[4:]])) if r < rows else (p, s) for r, (p, s) in enumerate(w.at)]
    for r in (0, 1, rows - 1):
        o, tol = w.want(r)
        heads = [3] if r == 0 else [2, 3]
        assert (np.abs(got[r] - o) <= tol)[heads].all()


def test_scores_that_are_all_minus_infinity_give_zeros():
    w = World([(64, [64, 80, 64])], 2, 1, 64, 16, out="f32")
    w.dk[..., 0] = -0x80                                         # 0xFF80: -inf
    w.dq[:, :, 0] = 1.0
    _, out = w.buffer()
    w.call(out)
    assert (out == 0).all()


def test_sharp_scores_raise_the_maximum_late():
    for rows in (3, 40):
        w = World([(3000, [3000 + i for i in range(rows)])], 4, 1, 128, 16, sharp=40.0, out="f32")
        say("sharp", rows)
        w.run(rows=[0, rows - 1])


def test_values_past_4_gib():
    page = 16 * 8 * 128 * 2
    n_pages = (5 << 30) // page
    k, v = (torch.zeros((n_pages, 16, 8, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k[-3:] = torch.randn(k[-3:].shape, device=DEV).to(torch.bfloat16)
    v[-3:] = torch.randn(v[-3:].shape, device=DEV).to(torch.bfloat16)
    far = torch.tensor([n_pages - 1, n_pages - 3, n_pages - 2], dtype=torch.int32, device=DEV)
    near = torch.arange(3, dtype=torch.int32, device=DEV)
    q = torch.randn((40, 8, 128), device=DEV).to(torch.bfloat16)
    lens = torch.full((40,), 48, dtype=torch.int32, device=DEV)
    starts, shared = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, 40], [32]))
    outs = []
    for cache, table in ((decode.kv_cache(k, v), far), (decode.kv_cache(k[far.long()], v[far.long()]), near)):
        out = torch.zeros((40, 8, 128), device=DEV)
        ws = torch.empty(decode.attn_shared_workspace_bytes(cache, 40, 1, 8, 48), dtype=torch.uint8, device=DEV)
        say("far pages")
        decode.attn_shared(cache, q, table[None].expand(40, 3).contiguous(), lens, 48, starts, shared, 0.1, out, ws)
        outs.append(out)
    assert torch.equal(*outs) and bool((outs[0] != 0).any())


@pytest.mark.parametrize("rows", [4, 60])
def test_another_stream_and_a_captured_graph(rows):
    w = World([(600, [640 + i for i in range(rows)]), [100]], 8, 2, 128, 16, same_pages=True)
    raw, out = w.buffer()
    _, eager = w.buffer()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    w.call(out, stream=side)
    torch.cuda.synchronize()
    w.call(eager)
    assert torch.equal(out, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.call(out)
    for i in range(4):
        w.lens.copy_(torch.tensor([640 - 30 * i + j for j in range(rows)] + [100 - i], dtype=torch.int32))
        w.shared.copy_(torch.tensor([(600, 37, 0, 700)[i], 0], dtype=torch.int32))
        w.dq.copy_(torch.randn(w.dq.shape, device=DEV).to(torch.bfloat16))
        w.call(eager)
        out.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i


def test_two_calls_at_once():
    worlds = [World([(2000, [2010 + i for i in range(50)])], 8, 2, 128, 16, seed=s) for s in (1, 2)]
    outs = [w.buffer()[1] for w in worlds]
    alone = []
    for w, o in zip(worlds, outs):
        w.call(o)
        torch.cuda.synchronize()
        alone.append(o.clone())
        o.fill_(0)
    streams = [torch.cuda.Stream() for _ in worlds]
    torch.cuda.synchronize()
    for _ in range(5):
        for w, o, s in zip(worlds, outs, streams):
            w.call(o, stream=s)
    torch.cuda.synchronize()
    for o, want in zip(outs, alone):
        assert torch.equal(o, want)


def test_the_binding_refuses_what_it_cannot_read():
    w = World([(32, [40, 41])], 8, 2, 128, 16)
    _, out = w.buffer()
    good = dict(q=w.dq, page_table=w.table, lens=w.lens, max_len=w.max_len, starts=w.starts, shared=w.shared, scale=w.scale,
                out=out, workspace=w.ws)
    decode.attn_shared(w.cache, **good)
    for bad in (dict(starts=w.starts[:1]), dict(starts=w.starts.long()), dict(shared=w.shared.float()), dict(starts=w.starts.cpu()),
                dict(shared=w.shared.cpu()), dict(lens=w.lens[:1]), dict(q=w.dq.half()), dict(out=out[:1]),
                dict(page_table=w.table.long()), dict(max_len=49)):
        with pytest.raises(ValueError):
            decode.attn_shared(w.cache, **{**good, **bad})
    with pytest.raises(x.XferError):
        decode.attn_shared(w.cache, **{**good, "workspace": w.ws[:64]})
    with pytest.raises(x.XferError):
        decode.attn_shared(w.cache, **{**good, "workspace": None})
