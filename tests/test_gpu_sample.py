"""GPU: sampling from two column shards (xfer_sample_merge) against the
definition in 64 bits, row by row.  The taken id has to be the definition's;
a row whose drawn number falls within 1e-12 of an element's border would not
be decided by it, and none of these does (checked)."""
import numpy as np
import pytest
import torch

import bf16_wire_all_amd as x
from bf16_wire_all_amd import decode
from tests import decode_reference as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
GUARD = 64
SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 40, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.8, 50, 0.95, 0.02),
            (0.0, 0, 1.0, 0.0), (1.3, 0, 0.999, 0.001), (2.0, 1000, 0.5, 0.0), (1.0, 1, 1.0, 0.0), (5.0, 0, 1.0, 0.5)]
CUTS = [(1.0, 0, 1.0, 0.05), (1.0, 0, 1.0, 1.0), (0.3, 0, 1.0, 1e-6), (1.0, 50, 1.0, 0.0), (2.0, 7, 0.9, 0.0),
        (1.0, 64, 0.8, 0.2), (1.0, 500, 1.0, 0.01), (0.0, 0, 1.0, 0.3), (-2.0, 5, 1.0, 0.3), (1e30, 0, 1.0, 0.5),
        (float("inf"), 0, 1.0, 0.5), (1e-30, 0, 1.0, 0.5), (1.0, 2000, 1.0, 0.0)]


def values_of(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def run(bits, n0, params, u, swap=False, calls=1):
    """bits: uint16 [rows, n0 + n1]; the shards lie in buffers of their own with padded rows of NaN."""
    rows, cols = bits.shape
    n1 = cols - n0
    say("sample", rows, n0, n1, "swapped" if swap else "")
    bufs = []
    for part in (bits[:, :n0], bits[:, n0:]):
        ld = -(-part.shape[1] // 8) * 8 + 8
        b = np.full((rows, ld), 0x7FC0, np.uint16)
        b[:, :part.shape[1]] = part
        bufs.append(torch.from_numpy(b.view(np.int16)).to(DEV))
    off = (n1, 0) if swap else (0, n0)
    s0, s1 = decode.shard(bufs[0], n0, off[0]), decode.shard(bufs[1], n1, off[1])
    params = np.array(params, dtype=decode.SAMPLE_PARAMS)
    dp = torch.from_numpy(params.view(np.uint8).copy()).to(DEV)
    du = torch.from_numpy(np.asarray(u, np.float32)).to(DEV)
    need = decode.sample_workspace_bytes(rows, n0, n1)
    ws = torch.full((need + GUARD,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((rows * 8 + GUARD,), 0x5A, dtype=torch.uint8, device=DEV)
    ids = np.concatenate([np.arange(n0) + off[0], np.arange(n1) + off[1]])
    wants = []
    for r in range(rows):
        p = params[r]
        wants.append(ref.sample(values_of(bits[r]), ids, float(p["temperature"]), int(p["top_k"]), float(p["top_p"]),
                                float(p["min_p"]), float(np.float32(u[r]))))
    for _ in range(calls):
        decode.sample_merge(s0, s1, dp, du, out[:rows * 8], ws[:need])
        torch.cuda.synchronize()
        got = out[:rows * 8].cpu().numpy().view(decode.SAMPLED)
        for r in range(rows):
            idx, prob, margin = wants[r]
            assert idx < 0 or margin > 1e-12, f"row {r}: the input does not decide"
            assert got["idx"][r] == idx, (r, params[r], u[r], got[r], wants[r])
            assert abs(got["prob"][r] - prob) <= 2.0 ** -23 * prob, (r, got[r], wants[r])
    assert bool((out[rows * 8:] == 0x5A).all()) and bool((ws[need:] == 0xFF).all())
    return got


def logits(rows, cols, seed, scale=2.5):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn((rows, cols), generator=g) * scale
    a += 8 * (torch.rand((rows, cols), generator=g) < 3e-4)
    return a.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16).copy()


def drawn(rows, seed):
    return torch.rand(rows, generator=torch.Generator().manual_seed(seed)).numpy()


SHAPES = [(1, 1, 1), (7, 1, 9), (5, 7, 8), (20, 255, 1025), (12, 2304, 1695), (10, 16384, 16384), (10, 16384, 16385),
          (10, 3, 32768), (10, 32769, 3), (6, 40001, 33000), (20, 64768, 64512), (4, 75968, 75968), (3, 1, 200001)]


@pytest.mark.parametrize("rows,n0,n1", SHAPES)
@pytest.mark.parametrize("swap", [False, True])
def test_shapes(rows, n0, n1, swap):
    seed = rows + n0 + n1
    run(logits(rows, n0 + n1, seed), n0, [SETTINGS[(r + seed) % len(SETTINGS)] for r in range(rows)],
        drawn(rows, seed + swap), swap)


@pytest.mark.parametrize("setting", SETTINGS, ids=str)
def test_settings(setting):
    rows = 24
    run(logits(rows, 5000, 3), 3000, [setting] * rows, drawn(rows, 4))
    run(logits(rows, 40000, 5), 17000, [setting] * rows, drawn(rows, 6), calls=2)


def test_the_widest_shards():
    run(logits(2, 2097152 + 2000000, 7), 2097152, [SETTINGS[0], SETTINGS[4]], drawn(2, 8))


@pytest.mark.parametrize("rows,n0,n1", [(300, 20001, 20003), (70, 40960, 40961), (100, 33000, 40001)])
def test_more_slices_than_workgroups(rows, n0, n1):
    """Workgroups of the count go from slice to slice; every seventh row is masked but for a few elements."""
    bits = logits(rows, n0 + n1, rows)
    bits[3::7, 100::] = 0xFF80
    bits[5::7, :n0 + 50] = 0xFF80
    run(bits, n0, [(SETTINGS + CUTS)[r % (len(SETTINGS) + len(CUTS))] for r in range(rows)], drawn(rows, rows + 1))


def test_masked_rows():
    """A mask of -inf leaves much, little, one element or nothing."""
    rows = 40
    for cols, n0 in ((3000, 1200), (70000, 30000)):
        m = logits(rows, cols, 9)
        g = np.random.default_rng(10)
        for r in range(rows):
            keep = (cols, cols // 3, 5, 1, 0)[r % 5]
            gone = np.ones(cols, bool)
            gone[g.permutation(cols)[:keep]] = False
            m[r, gone] = 0xFF80
        got = run(m, n0, [SETTINGS[r % len(SETTINGS)] for r in range(rows)], drawn(rows, 11))
        assert np.all(got["idx"][4::5] == -1) and np.all(got["prob"][4::5] == 0)


def test_nan_is_never_taken_and_infinity_takes_all():
    rows = 30
    m = logits(rows, 2000, 12)
    g = np.random.default_rng(13)
    for r in range(rows):
        at = g.permutation(2000)
        m[r, at[:300]] = np.where(g.random(300) < 0.5, 0x7FC1, 0xFFFF)
        if r % 3 == 1:
            m[r, at[300:303]] = 0x7F80
    got = run(m, 900, [SETTINGS[r % len(SETTINGS)] for r in range(rows)], drawn(rows, 14))
    for r in range(1, rows, 3):
        assert m[r, got["idx"][r]] == 0x7F80


def test_ties_and_both_zeros():
    """Few values, both zeros and shards in either order: equal logits go by id."""
    letters = np.array([0x0000, 0x8000, 0x3F80, 0xBF80, 0x3F00], np.uint16)
    g = np.random.default_rng(15)
    m = letters[g.integers(0, 5, (60, 777))]
    for swap in (False, True):
        run(m, 300, [SETTINGS[r % len(SETTINGS)] for r in range(60)], drawn(60, 16), swap)


@pytest.mark.parametrize("cols,n0", [(30000, 11000), (200000, 90000)])
def test_one_value_everywhere(cols, n0):
    """A row of equal logits: more of one value than 16 bits count, every id its share."""
    m = np.full((8, cols), 0x4040, np.uint16)
    u = np.array([0, 0.1, 0.25001, 0.5001, 0.7, 0.9, 0.99999, 1 - 2 ** -24], np.float32)
    got = run_uniform(m, n0, u)
    assert np.array_equal(got["idx"], np.minimum((u.astype(np.float64) * cols).astype(np.int64), cols - 1))


def run_uniform(m, n0, u):
    rows, cols = m.shape
    params = [(1.0, 0, 1.0, 0.0)] * rows
    # u = 0 lies on the first element's border, where the sums are whole numbers and exact
    s = [decode.shard(torch.from_numpy(np.ascontiguousarray(np.pad(p, ((0, 0), (0, -p.shape[1] % 8)))).view(np.int16))
                      .to(DEV), p.shape[1], o) for p, o in ((m[:, :n0], 0), (m[:, n0:], n0))]
    dp = torch.from_numpy(np.array(params, decode.SAMPLE_PARAMS).view(np.uint8).copy()).to(DEV)
    out = torch.zeros((rows, 2), dtype=torch.int32, device=DEV)
    ws = torch.empty(decode.sample_workspace_bytes(rows, n0, cols - n0), dtype=torch.uint8, device=DEV)
    decode.sample_merge(s[0], s[1], dp, torch.from_numpy(u).to(DEV), out, ws)
    torch.cuda.synchronize()
    got = out.cpu().numpy().view(decode.SAMPLED).reshape(-1)
    assert np.all(np.abs(got["prob"] * cols - 1) < 1e-6)
    return got


def test_borders_are_exact_where_the_weights_are():
    """Equal logits have weight 1: top-p, min-p and u on exact borders."""
    m = np.full((6, 16), 0x3F80, np.uint16)
    rows = [((1.0, 0, 0.5, 0.0), 1 - 2.0 ** -24, 7), ((1.0, 0, 0.5 + 2.0 ** -20, 0.0), 1 - 2.0 ** -24, 8),
            ((1.0, 8, 0.25, 0.0), 1 - 2.0 ** -24, 1), ((1.0, 0, 1.0, 1.0), 0.5, 8), ((1.0, 0, 1.0, 0.0), 0.25, 4),
            ((1.0, 0, 0.0, 0.0), 0.99, 0)]
    s = [decode.shard(torch.from_numpy(np.ascontiguousarray(m[:, :8]).view(np.int16)).to(DEV), 8, o) for o in (0, 8)]
    dp = torch.from_numpy(np.array([r[0] for r in rows], decode.SAMPLE_PARAMS).view(np.uint8).copy()).to(DEV)
    du = torch.tensor([r[1] for r in rows], dtype=torch.float32, device=DEV)
    out = torch.zeros((6, 2), dtype=torch.int32, device=DEV)
    ws = torch.empty(decode.sample_workspace_bytes(6, 8, 8), dtype=torch.uint8, device=DEV)
    decode.sample_merge(s[0], s[1], dp, du, out, ws)
    torch.cuda.synchronize()
    assert out[:, 1].tolist() == [r[2] for r in rows]


@pytest.mark.parametrize("cols,n0", [(32768, 16000), (60000, 30000)])
def test_more_distinct_values_than_shared_memory_keeps(cols, n0):
    rows = 12
    g = np.random.default_rng(17)
    m = g.integers(0, 1 << 16, (rows, cols)).astype(np.uint16)
    m[(m & 0x7FFF) >= 0x4400] &= 0xBFFF  # below 2^9, so that many elements have a weight
    params = [((64.0, 0, 1.0, 0.0), (200.0, 30000, 1.0, 0.0), (100.0, 0, 0.7, 0.0), (300.0, 0, 1.0, 0.3))[r % 4]
              for r in range(rows)]
    run(m, n0, params, drawn(rows, 18))


@pytest.mark.parametrize("n0,n1", [(1000, 1200), (40000, 30001), (16385, 16383)])
@pytest.mark.parametrize("shape", ["apart", "below zero", "about zero", "tiny", "few", "infinite", "equal"])
def test_settings_that_leave_most_elements_out(shape, n0, n1):
    """What a part of a row may leave out depends on that part's own first elements: they differ between
    the parts here, in size and in sign."""
    rows, cols = len(CUTS), n0 + n1
    rng = np.random.default_rng(n0 + len(shape))
    v = rng.standard_normal((rows, cols)) * 2.0
    if shape == "apart":
        v[:, :n0] += 3.0
        v[:, n0 // 2:n0] += 3.0
    elif shape == "below zero":
        v -= 20.0
    elif shape == "about zero":
        v = -np.abs(v)
        v[:, ::97] = 0.0
    elif shape == "tiny":
        v *= 1e-38
    elif shape == "few":
        v[:, :] = -np.inf
        v[:, 5::cols // 9] = rng.standard_normal(v[:, 5::cols // 9].shape)
    elif shape == "infinite":
        v[:, [3, n0 - 1, n0 + 2, cols - 1]] = np.inf
        v[:, 10:500] = np.nan
    elif shape == "equal":
        v = np.round(v)
    bits = torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16).copy()
    if shape == "infinite":
        bits[:, 10:200] = 0x7FC1                       # NaN of both signs
        bits[:, 200:500] = 0xFFFF
    run(bits, n0, CUTS, rng.random(rows))


def test_odd_settings():
    """Temperatures and limits past their ranges mean what the header says."""
    inf, nan = float("inf"), float("nan")
    params = [(-1.0, 0, 1.0, 0.0), (nan, 5, 0.5, 0.0), (1e-30, 0, 1.0, 0.0), (inf, 0, 1.0, 0.0), (inf, 100, 0.5, 0.0),
              (1.0, 4000000000, 1.0, 0.0), (1.0, 0, -1.0, 0.0), (1.0, 0, nan, 0.0), (1.0, 0, 2.0, 0.0),
              (1.0, 0, 1.0, -3.0), (1.0, 0, 1.0, nan), (1.0, 0, 1.0, 7.0), (1e30, 0, 0.9, 0.0)]
    for cols, n0 in ((3000, 1700), (50000, 20000)):
        run(logits(len(params), cols, 19), n0, params, drawn(len(params), 20))
    u = [-1.0, nan, 0.99999994, 5.0]
    m = logits(4, 3000, 21)
    params = [(1.0, 0, 1.0, 0.0)] * 4
    ids = np.arange(3000)
    s = [decode.shard(torch.from_numpy(np.ascontiguousarray(p).view(np.int16)).to(DEV), 1504 if o == 0 else 1496, o)
         for p, o in ((m[:, :1504], 0), (m[:, 1504:], 1504))]
    out = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    ws = torch.empty(decode.sample_workspace_bytes(4, 1504, 1496), dtype=torch.uint8, device=DEV)
    decode.sample_merge(s[0], s[1], torch.from_numpy(np.array(params, decode.SAMPLE_PARAMS).view(np.uint8).copy()).to(DEV),
                        torch.tensor(u, dtype=torch.float32, device=DEV), out, ws)
    torch.cuda.synchronize()
    got = out[:, 1].tolist()
    order = [np.lexsort((ids, -values_of(m[r]))) for r in range(4)]
    assert got[0] == order[0][0] and got[1] == order[1][0] and got[3] == order[3][-1]


def test_frequencies_follow_the_weights():
    """20,000 evenly spaced numbers over one row take each element its share of times, give or take one."""
    n, t = 20000, 0.9
    row = logits(1, 40, 22)
    m = np.repeat(row, n, 0)
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    s = [decode.shard(torch.from_numpy(np.ascontiguousarray(m[:, a:a + 24]).view(np.int16)).to(DEV), c, a)
         for a, c in ((0, 24), (24, 16))]
    dp = torch.from_numpy(np.array([(t, 0, 1.0, 0.0)] * n, decode.SAMPLE_PARAMS).view(np.uint8).copy()).to(DEV)
    out = torch.zeros((n, 2), dtype=torch.int32, device=DEV)
    ws = torch.empty(decode.sample_workspace_bytes(n, 24, 16), dtype=torch.uint8, device=DEV)
    say("sample frequencies", n)
    decode.sample_merge(s[0], s[1], dp, torch.from_numpy(u).to(DEV), out, ws)
    torch.cuda.synchronize()
    v = values_of(row[0])
    w = np.exp(v / t)
    got = np.bincount(out[:, 1].cpu().numpy(), minlength=40)
    assert np.all(np.abs(got - w / w.sum() * n) <= 1.01)


def test_greedy_agrees_with_the_argmax():
    m = logits(64, 129280, 23)
    dl = torch.from_numpy(m.view(np.int16)).to(DEV)
    s0, s1 = x.shard(dl.data_ptr(), 129280, 64, 64768, 0), x.shard(dl.data_ptr() + 2 * 64768, 129280, 64, 64512, 64768)
    rec = torch.zeros(64 * 8, dtype=torch.uint8, device=DEV)
    x.argmax_merge(s0, s1, x.ARGMAX, rec, torch.empty(x.argmax_workspace_bytes(64, 64768, 64512), dtype=torch.uint8, device=DEV))
    dp = torch.zeros(64 * 16, dtype=torch.uint8, device=DEV)  # temperature 0
    out = torch.zeros(64 * 8, dtype=torch.uint8, device=DEV)
    ws = torch.empty(decode.sample_workspace_bytes(64, 64768, 64512), dtype=torch.uint8, device=DEV)
    decode.sample_merge(s0, s1, dp, torch.rand(64, device=DEV), out, ws)
    torch.cuda.synchronize()
    assert np.array_equal(rec.cpu().numpy().view(x.MAX_IDX)["idx"], out.cpu().numpy().view(decode.SAMPLED)["idx"])


def test_captured_and_replayed_with_other_inputs():
    rows, n0, n1 = 6, 20000, 30000
    bufs = [torch.zeros((rows, n), dtype=torch.int16, device=DEV) for n in (n0, n1)]
    s = [decode.shard(b, n, o) for b, n, o in zip(bufs, (n0, n1), (0, n0))]
    params = np.array([SETTINGS[r] for r in range(rows)], decode.SAMPLE_PARAMS)
    dp = torch.from_numpy(params.view(np.uint8).copy()).to(DEV)
    du = torch.zeros(rows, device=DEV)
    out = torch.zeros((rows, 2), dtype=torch.int32, device=DEV)
    ws = torch.empty(decode.sample_workspace_bytes(rows, n0, n1), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        decode.sample_merge(s[0], s[1], dp, du, out, ws)
    for k in range(4):
        m = logits(rows, n0 + n1, 30 + k)
        u = drawn(rows, 40 + k)
        bufs[0].copy_(torch.from_numpy(m[:, :n0].view(np.int16).copy()))
        bufs[1].copy_(torch.from_numpy(m[:, n0:].view(np.int16).copy()))
        du.copy_(torch.from_numpy(u))
        g.replay()
        torch.cuda.synchronize()
        got = out[:, 1].tolist()
        for r in range(rows):
            assert got[r] == ref.sample(values_of(m[r]), np.arange(n0 + n1), *(float(params[r][f]) for f in ("temperature",)),
                                        int(params[r]["top_k"]), float(params[r]["top_p"]), float(params[r]["min_p"]),
                                        float(u[r]))[0]


def test_refused_call_leaves_the_output_untouched():
    b = torch.zeros((2, 64), dtype=torch.int16, device=DEV)
    out = torch.full((2, 2), 9, dtype=torch.int32, device=DEV)
    with pytest.raises(x.XferError):
        decode.sample_merge(decode.shard(b, 64, 0), decode.shard(b, 64, 32), torch.zeros(32, dtype=torch.uint8, device=DEV),
                            torch.zeros(2, device=DEV), out, torch.zeros(1 << 16, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert bool((out == 9).all())


def test_the_largest_number_below_one_takes_the_definition_s_element():
    u = np.float32(0.99999994)
    m = logits(4, 3000, 21)
    got = run(m, 1504, [(1.0, 0, 1.0, 0.0)] * 4, [u] * 4)
    assert np.all(got["idx"] >= 0)
