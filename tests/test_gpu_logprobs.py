"""GPU: log probabilities, ranks, alternatives and entropy from two column
shards (xfer_logprobs_merge) against the definition in 64 bits.  Ids and ranks
have to be equal."""
import math

import numpy as np
import pytest
import torch

import bf16_wire_all_amd as x
from bf16_wire_all_amd import decode
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = float("inf")
GUARD = 64


def values_of(bits):
    with np.errstate(invalid="ignore"):
        return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def reference(v, ids, T, tokens, n_top):
    """One row: values with their ids -> dict of results and how far binary32 weights may be from them.

    A weight is off by its exponent's rounding and the constant's (2 * 2^-24 |x|) and the power's last place
    (2^-23); a thread adds up to 64 of them (64 * 2^-24), in binary64 from there on.  Weights below binary32's
    subnormal numbers are lost.  The result is rounded once (2^-24)."""
    counted = ~np.isnan(v) & (v > -INF)
    order = np.lexsort((ids[counted], -v[counted]))
    ov, oi = v[counted][order], ids[counted][order]
    n = len(ov)
    out = {"entropy": 0.0, "entropy_tol": 0.0}
    lp, tol = np.full(n, -INF), np.zeros(n)
    if n:
        if not T > 0:
            lp[0] = 0.0
        else:
            with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
                d = ov - ov[0]
                xs = np.where(ov == ov[0], 0.0, -INF if np.isinf(ov[0]) else d / T)
            w = np.exp(xs)
            wx = np.where(w > 0, w * np.where(w > 0, xs, 0.0), 0.0)
            rest = w[1:].sum()
            log_z = math.log1p(rest)
            h = -wx.sum() / (1 + rest)
            err_r = 2.0 ** -24 * (66 * rest + 2 * -wx.sum()) + n * 2.0 ** -149
            with np.errstate(invalid="ignore"):
                err_wx = 2.0 ** -24 * (70 * -wx.sum() + 2 * np.where(w > 0, w * xs * xs, 0.0).sum()) + n * 2.0 ** -140
            lp = xs - log_z
            tol = err_r / (1 + rest) + 2.0 ** -24 * np.where(np.isinf(lp), 0, np.abs(lp)) + 1e-13
            out["entropy"] = log_z + h
            out["entropy_tol"] = (err_r + err_wx + h * err_r) / (1 + rest) + 2.0 ** -24 * out["entropy"] + 1e-13
    place = {int(i): k for k, i in enumerate(oi)}
    ranks = [place.get(int(t), -1) for t in tokens]
    out["rank"] = ranks
    out["logprob"] = [lp[r] if r >= 0 else -INF for r in ranks]
    out["tol"] = [tol[r] if r >= 0 else 0.0 for r in ranks]
    out["top_idx"] = [int(oi[k]) if k < n else -1 for k in range(n_top)]
    out["top_logprob"] = [lp[k] if k < n else -INF for k in range(n_top)]
    out["top_tol"] = [tol[k] if k < n else 0.0 for k in range(n_top)]
    return out


def near(got, want, tol):
    with np.errstate(over="ignore"):
        rounded = float(np.float32(want))          # past binary32's largest: infinite
    return got == rounded or (math.isfinite(rounded) and abs(got - want) <= tol)


class Call:
    """The shards lie in buffers of their own with padded rows of NaN; guards around every output."""

    def __init__(self, bits, n0, tokens, n_top, temperature=None, swap=False, entropy=True):
        rows, cols = bits.shape
        self.bits, self.n0, self.n1, self.rows, self.n_top = bits, n0, cols - n0, rows, n_top
        bufs = []
        for part in (bits[:, :n0], bits[:, n0:]):
            b = np.full((rows, -(-part.shape[1] // 8) * 8 + 8), 0x7FC0, np.uint16)
            b[:, :part.shape[1]] = part
            bufs.append(torch.from_numpy(b.view(np.int16)).to(DEV))
        off = (self.n1, 0) if swap else (0, n0)
        self.s = decode.shard(bufs[0], n0, off[0]), decode.shard(bufs[1], self.n1, off[1])
        self.ids = np.concatenate([np.arange(n0) + off[0], np.arange(self.n1) + off[1]])
        self.tokens = np.asarray(tokens, np.int32).reshape(rows, -1)
        self.nt = self.tokens.shape[1]
        self.T = temperature
        self.dT = None if temperature is None else torch.tensor(temperature, dtype=torch.float32, device=DEV)
        self.dt = torch.from_numpy(self.tokens.copy()).to(DEV)
        need = decode.logprobs_workspace_bytes(rows, n0, self.n1, self.nt, n_top)
        self.ws = torch.full((need + GUARD,), 0xFF, dtype=torch.uint8, device=DEV)
        self.need = need
        self.out = [torch.full((rows * n * size + GUARD,), 0x5A, dtype=torch.uint8, device=DEV)
                    for n, size in ((self.nt, 8), (n_top, 8), (1, 4))]
        self.entropy = entropy

    def run(self, stream=None):
        r = self.rows
        decode.logprobs_merge(*self.s, self.dt if self.nt else None, self.out[0][:r * self.nt * 8] if self.nt else None,
                              self.out[1][:r * self.n_top * 8] if self.n_top else None,
                              self.out[2][:r * 4].view(torch.float32) if self.entropy else None,
                              self.ws[:self.need] if self.need else None, temperature=self.dT, stream=stream)

    def results(self):
        torch.cuda.synchronize()
        r = self.rows
        host = [o.cpu().numpy() for o in self.out]
        for o, n in zip(host, (r * self.nt * 8, r * self.n_top * 8, r * 4 if self.entropy else 0)):
            assert (o[n:] == 0x5A).all()
        assert (self.ws[self.need:] == 0xFF).all()
        return (host[0][:r * self.nt * 8].view(decode.TOKEN_LOGPROB).reshape(r, self.nt),
                host[1][:r * self.n_top * 8].view(decode.TOP_LOGPROB).reshape(r, self.n_top), host[2][:r * 4].view(np.float32))

    def check(self, rows=None):
        tok, top, ent = self.results()
        for r in range(self.rows if rows is None else rows):
            T = 1.0 if self.T is None else float(np.float32(self.T[r]))
            want = reference(values_of(self.bits[r]), self.ids, T, self.tokens[r], self.n_top)
            assert list(tok[r]["rank"]) == want["rank"], f"row {r}"
            assert list(top[r]["idx"]) == want["top_idx"], f"row {r}"
            for got, w, tol in (*zip(tok[r]["logprob"], want["logprob"], want["tol"]),
                                *zip(top[r]["logprob"], want["top_logprob"], want["top_tol"])):
                assert near(float(got), w, tol), f"row {r}: {got} for {w}, {tol} allowed"
            if self.entropy:
                assert near(float(ent[r]), want["entropy"], want["entropy_tol"]), f"row {r}: {ent[r]} for {want['entropy']}"


def logits(rows, cols, seed, scale=2.5, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn((rows, cols), generator=g) * scale + 8.0 * (torch.rand((rows, cols), generator=g) < 1e-3)
    if masked:
        v = v.masked_fill(torch.rand(v.shape, generator=g) < masked, -INF)
    return v.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def some_tokens(rows, cols, n, seed):
    t = np.random.default_rng(seed).integers(0, cols, (rows, n)).astype(np.int32)
    if n > 3:
        t[::3, 1], t[1::3, 2], t[2::3, 3] = -1, cols, 2 ** 31 - 1
    return t


@pytest.mark.parametrize("rows,n0,n1,n_tokens,n_top,masked", [
    (1, 1, 1, 1, 1, 0), (1, 7, 9, 16, 32, 0), (3, 1000, 900, 2, 5, 0), (5, 2304, 1695, 3, 20, 0.7), (2, 64768, 64512, 1, 5, 0),
    (16, 16384, 16385, 4, 32, 0.5), (1, 200000, 1, 2, 7, 0), (1, 3, 250001, 0, 32, 0.9), (40, 30001, 20003, 1, 0, 0),
    (1100, 999, 1003, 1, 3, 0.2), (1500, 20000, 18000, 1, 1, 0), (1030, 40001, 17, 2, 32, 0.1), (7, 129, 4095, 0, 0, 0)])
@pytest.mark.parametrize("swap", [False, True])
def test_sizes(rows, n0, n1, n_tokens, n_top, masked, swap):
    say("logprobs", rows, n0, n1, n_tokens, n_top, masked, swap)
    if rows > 100 and swap:
        rows = rows // 2 + 513          # still a workgroup for each row, on another count
    c = Call(logits(rows, n0 + n1, rows + n0, masked=masked), n0, some_tokens(rows, n0 + n1, n_tokens, 5), n_top,
             temperature=None if swap else list(np.linspace(0.3, 3, rows)), swap=swap)
    c.run()
    c.check()
    first = [a.tobytes() for a in c.results()]
    c.run()
    assert first == [a.tobytes() for a in c.results()]


TEMPERATURES = [1.0, 0.0, -1.0, float("nan"), INF, 1e-30, 1e-42, 1e30, 0.01, 100.0, 2.0 ** -70, -0.0]
BF = lambda v: int(torch.tensor(v).to(torch.bfloat16).view(torch.int16)) & 0xFFFF


def special_rows(cols):
    """Rows where the order, the largest or the weights are not the usual ones."""
    base = logits(1, cols, 77)[0]
    rows = {"plain": base}
    def put(name, fill=None, **at):
        r = base.copy() if fill is None else np.full(cols, fill, np.uint16)
        for k, v in at.items():
            r[int(k[1:]) % cols] = v
        rows[name] = r
    put("all equal", BF(1.5))
    put("all masked", 0xFF80)
    put("all nan", 0x7FC0)
    put("nan of both signs", 0xFFC1, _5=BF(2.0), _6=0x7F81, _900=BF(2.0))
    put("one element", 0xFF80, _301=BF(-3.0))
    put("an infinity", _17=0x7F80)
    put("three infinities and a nan", _17=0x7F80, _18=0x7F80, _1501=0x7F80, _3=0x7FC0)
    put("infinities alone", 0x7F80)
    put("nan beside numbers", _0=0x7FC0, _1=0xFFC0, _2=0x7FFF, _3=0x7F81)
    put("zeros of both signs", 0x8000, _100=0, _50=0x8000, _1900=0)
    put("zeros above negatives", BF(-1.0), _40=0x8000, _41=0, _39=0x8000)
    rows["all negative"] = base | 0x8000
    put("largest number", 0xFF7F, _8=0x7F7F, _9=0x7F7E)
    put("lowest numbers", 0xFF7F, _9=0xFF80)
    put("subnormal", 0x0001, _4=0x0003, _5=0x8001)
    put("far apart", BF(-200.0), _7=BF(50.0))
    put("near one", BF(-20.0), _7=BF(3.0))
    rows["rising"] = np.sort(base.view(np.int16)).view(np.uint16)
    rows["two values"] = np.where(np.arange(cols) % 2, BF(1.0), BF(1.0078125)).astype(np.uint16)
    few = np.full(cols, 0xFF80, np.uint16)
    few[64:64 + 40] = base[:40]                   # all of them with a few lanes
    rows["few lanes"] = few
    return rows


@pytest.mark.parametrize("cols,n0", [(2000, 1003), (50000, 20000)])
@pytest.mark.parametrize("n_top", [1, 32])
def test_special_rows_at_special_temperatures(cols, n0, n_top):
    rows = special_rows(cols)
    for T in TEMPERATURES:
        bits = np.stack(list(rows.values()))
        tokens = np.tile(np.array([0, 5, 7, 17, 1501, 301, cols - 1, -5], np.int32), (len(bits), 1))
        say("special", cols, n_top, T)
        c = Call(bits, n0, tokens, n_top, temperature=[T] * len(bits))
        c.run()
        try:
            c.check()
        except AssertionError as e:
            raise AssertionError(f"T = {T}, rows {list(enumerate(rows))}: {e}") from None


def test_special_rows_of_several_slices_to_a_workgroup():
    """From 1,536 rows on a workgroup goes through a row's slices one after the other: larger ones later, and none."""
    cols, n0 = 50000, 20000
    rows = special_rows(cols)
    falling = rows["rising"][::-1]
    late = np.full(cols, 0xFF80, np.uint16)
    late[-300:] = rows["plain"][:300]
    early = np.full(cols, 0xFF80, np.uint16)
    early[:300] = rows["plain"][:300]
    steps = rows["plain"].copy()
    for i, v in enumerate((-3.0, 20.0, 20.0, 200.0)):   # the largest of each slice, twice the same
        steps[[100 + i * 10000 + j for j in (3, 777)]] = BF(v)
    infinite = steps.copy()
    infinite[-5:] = [0x7F80, BF(1.0), 0x7F80, 0x7FC0, 0xFF80]
    made = list(rows.values()) + [falling, late, early, steps, infinite]
    n = -(-1536 // len(made)) * len(made)
    bits = np.stack(made)
    tokens = np.tile(np.array([0, 103, 10103, cols - 1], np.int32), (n, 1))
    for T in (1.0, 0.05, 0.0):
        say("several slices", T)
        c = Call(np.tile(bits, (n // len(made), 1)), n0, tokens, 8, temperature=[T] * n)
        c.run()
        got = [t.reshape(-1, len(made), *t.shape[1:]) for t in c.results()]
        for t in got:
            assert all(t[i].tobytes() == t[0].tobytes() for i in range(1, len(t)))
        c.check(len(made))


@pytest.mark.parametrize("cols,n0,rows", [(40000, 20000, 1100), (16384 * 3, 16384, 1030), (300000, 100, 1)])
def test_more_equal_elements_than_the_list_holds(cols, n0, rows):
    bits = np.full((rows, cols), BF(0.25), np.uint16)
    rng = np.random.default_rng(3)
    for r in range(rows):
        bits[r, rng.integers(0, cols, 20)] = BF(0.5)
        bits[r, rng.integers(0, cols, 3000)] = 0xFF80
    say("ties", cols, rows)
    c = Call(bits[:, :], n0, some_tokens(rows, cols, 2, 9), 32)
    c.run()
    c.check()


def test_a_logprob_near_zero_keeps_its_digits():
    cols = 1000
    bits = np.full((4, cols), BF(-10.0), np.uint16)
    for r, v in enumerate((10.0, 20.0, 30.0, 60.0)):
        bits[r, 500 + r] = BF(v)
    c = Call(bits, 300, np.array([[500], [501], [502], [503]]), 2)
    c.run()
    c.check()
    tok, _, ent = c.results()
    want = [-math.log1p(999 * math.exp(-10.0 - v)) for v in (10.0, 20.0, 30.0, 60.0)]
    assert np.allclose(tok["logprob"][:, 0], want, rtol=2e-5, atol=0)
    assert (ent > 0).all()


def test_no_entropy_asked_for_and_a_token_named_twice():
    c = Call(logits(3, 5000, 1), 2000, [[7, 7, 4999], [0, 1, 0], [2000, 1999, 2000]], 0, entropy=False)
    c.run()
    c.check()


def test_rows_of_one_buffer_and_a_wide_vocabulary():
    """Both shards are column ranges of one tensor of 2 x 2,097,152 columns."""
    cols = 2097152
    bits = logits(1, 2 * cols, 6)
    t = torch.from_numpy(bits.view(np.int16)).to(DEV)
    s0, s1 = decode.shard(t[:, :cols], cols, 0), decode.shard(t[:, cols:], cols, cols)
    tokens = torch.tensor([[5, 2 * cols - 1]], dtype=torch.int32, device=DEV)
    out, top = torch.zeros((1, 2, 2), dtype=torch.int32, device=DEV), torch.zeros((1, 9, 2), dtype=torch.int32, device=DEV)
    ws = torch.empty(decode.logprobs_workspace_bytes(1, cols, cols, 2, 9), dtype=torch.uint8, device=DEV)
    say("wide")
    decode.logprobs_merge(s0, s1, tokens, out, top, None, ws)
    want = reference(values_of(bits[0]), np.arange(2 * cols), 1.0, [5, 2 * cols - 1], 9)
    assert out[0, :, 1].tolist() == want["rank"] and top[0, :, 1].tolist() == want["top_idx"]
    for got, w, tol in zip(out.view(torch.float32)[0, :, 0].tolist(), want["logprob"], want["tol"]):
        assert near(got, w, tol)


@pytest.mark.parametrize("rows", [6, 1200])
def test_another_stream_and_a_captured_graph(rows):
    c = Call(logits(rows, 20000, 4), 9000, some_tokens(rows, 20000, 2, 1), 5, temperature=[0.7] * rows)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.run(stream=side)
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for i in range(3):
        bits = logits(rows, 20000, 50 + i)
        for s, part in zip(c.s, (bits[:, :9000], bits[:, 9000:])):
            s.tensor[:, :part.shape[1]] = torch.from_numpy(part.view(np.int16)).to(DEV)
        c.run()
        want = [a.tobytes() for a in c.results()]
        for o in c.out:
            o.fill_(0x5A)
        torch.cuda.synchronize()
        graph.replay()
        assert want == [a.tobytes() for a in c.results()]


def test_two_calls_at_once_and_two_graphs_that_share_a_workspace():
    calls = [Call(logits(9, 30000, 60 + i), 11000, some_tokens(9, 30000, 3, i), 7, temperature=[1.1] * 9) for i in range(2)]
    want = []
    for c in calls:
        c.run()
        want.append([a.tobytes() for a in c.results()])
        c.check()
    streams = [torch.cuda.Stream() for _ in calls]
    for c in calls:
        for o in c.out:
            o.fill_(0x5A)
    torch.cuda.synchronize()
    for _ in range(5):
        for c, stream in zip(calls, streams):
            c.run(stream=stream)
    for c, w in zip(calls, want):
        assert [a.tobytes() for a in c.results()] == w
    calls[1].ws = calls[0].ws
    graphs = [torch.cuda.CUDAGraph() for _ in calls]
    for graph, c in zip(graphs, calls):
        with torch.cuda.graph(graph):
            c.run()
    for i in (1, 0, 0, 1, 0):
        for o in calls[i].out:
            o.fill_(0x5A)
        torch.cuda.synchronize()
        graphs[i].replay()
        assert [a.tobytes() for a in calls[i].results()] == want[i]


def test_the_binding_refuses_what_it_cannot_read():
    c = Call(logits(3, 200, 1), 100, some_tokens(3, 200, 2, 1), 4)
    r = c.rows
    good = dict(tokens=c.dt, token_out=c.out[0][:r * 16], top_out=c.out[1][:r * 32], entropy=c.out[2][:r * 4].view(torch.float32),
                workspace=c.ws)
    decode.logprobs_merge(*c.s, **good)
    for bad in (dict(tokens=c.dt.long()), dict(tokens=c.dt.cpu()), dict(tokens=c.dt[:2]), dict(tokens=None),
                dict(token_out=c.out[0][:r * 8]), dict(token_out=None), dict(top_out=c.out[1][:r * 8 + 8]),
                dict(entropy=good["entropy"][:2]), dict(entropy=good["entropy"].double()), dict(tokens=c.dt.t()),
                dict(temperature=torch.ones(r, device=DEV, dtype=torch.float16)), dict(temperature=torch.ones(r + 1, device=DEV)),
                dict(tokens=None, token_out=None, top_out=None, entropy=None)):
        with pytest.raises(ValueError):
            decode.logprobs_merge(*c.s, **{**good, **bad})
    with pytest.raises(x.XferError):
        decode.logprobs_merge(*c.s, **{**good, "top_out": torch.zeros(r * 33 * 8, dtype=torch.uint8, device=DEV)})
