"""GPU: infinities and NaN among the keys and values that a row sees
(xfer_attn_paged).  A head whose scores are all -inf gets zeros whatever the
values are; an infinite value makes its dim of every head infinite, however
small its weight; and neither reaches another dim, head or row."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_attn_paged import NAN16, World

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF16, NINF16 = 0x7F80, 0xFF80 - 0x10000
# each way that a call is cut up: (rows' lengths, q heads, kv heads, head_dim, order, max_len)
FORMS = {
    "one unit": ([40, 70, 9], 8, 2, 64, "tokens", None),
    "whole rows": ([700, 300, 512], 8, 2, 256, "heads", None),
    "whole rows, eight waves": ([700, 300, 512], 8, 2, 128, "tokens", None),
    "whole rows, 20 heads": ([700, 300, 512], 40, 2, 64, "heads", None),
    "runs": ([9000, 4097, 300], 8, 2, 128, "heads", None),
    "runs past the caches": ([9000, 4097, 300], 8, 2, 128, "heads", 40000),
    "runs, 20 heads": ([9000, 4097, 300], 40, 2, 128, "heads", None),
    "heads side by side": ([9000, 4097, 300], 8, 4, 64, "tokens", 70000),
    "two heads side by side": ([9000, 4097, 300], 4, 2, 64, "tokens", 140000),
}


def world(form, out, seed, **kw):
    lens, hq, hkv, d, order, max_len = FORMS[form]
    return World(lens, hq, hkv, d, 16, "bf16", order, out=out, seed=seed, max_len=max_len, **kw)


def put(w, which, r, t, h, d, bits):
    """Element d of head h of row r's visible token t: a bit pattern, here and on the GPU."""
    host, dev = ((w.k, w.dk), (w.v, w.dv))[which]
    p, s = w.at[r][0][t], w.at[r][1][t]
    host[p, s, h, d] = bits
    dev[p, s, h, d] = bits


def call(w):
    out = torch.full((w.rows, w.hq, w.d), 7.0, dtype=w.out_dtype, device=DEV)
    ws, n = w.workspace()
    say("attn_paged, non-finite", w.lens, w.hq, w.hkv, w.d, n)
    w.call(out, ws[:n] if n else None)
    torch.cuda.synchronize()
    assert bool((ws[n:] == 0xFF).all())
    return out.cpu().float().numpy().astype(np.float64)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS)
def test_infinite_values(form, out):
    """Row 0: one infinity, early or late, of either sign, and both.  Row 1: a NaN beside an infinity."""
    w = world(form, out, 31)
    o, tol = w.want()
    last, last1 = w.lens[0] - 1, w.lens[1] - 1
    marks = [(0, 3, 0, 5, INF16), (0, last, 0, 6, NINF16), (0, last // 2, 1, 9, NINF16), (0, 0, 1, 40, INF16),
             (0, 1, 1, 41, INF16), (0, last, 1, 41, INF16),                     # one sign twice
             (0, 2, 0, 63, INF16), (0, last, 0, 63, NINF16),                    # both signs
             (1, 0, 0, 7, INF16), (1, last1, 0, 7, NAN16), (1, last1 // 2, 1, 8, NAN16), (1, last1, 1, 0, INF16)]
    for r, t, h, d, bits in marks:
        put(w, 1, r, t, h, d, bits)
    group = w.hq // w.hkv
    inf = float("inf")
    for r, h, d, value in ((0, 0, 5, inf), (0, 0, 6, -inf), (0, 1, 9, -inf), (0, 1, 40, inf), (0, 1, 41, inf),
                           (0, 0, 63, np.nan), (1, 0, 7, np.nan), (1, 1, 8, np.nan), (1, 1, 0, inf)):
        o[r, h * group:(h + 1) * group, d] = value
    got = call(w)
    assert np.array_equal(np.isnan(got), np.isnan(o))
    assert np.array_equal(got[np.isinf(o)], o[np.isinf(o)])
    fine = np.isfinite(o)
    assert np.all(np.abs(got[fine] - o[fine]) <= tol[fine])


@pytest.mark.parametrize("form", FORMS)
def test_infinite_values_of_the_smallest_weights(form):
    """Scores hundreds below the largest, whose weights binary32 cannot hold."""
    w = world(form, "f32", 32, sharp=0.01)
    r, h = 0, 1
    group = w.hq // w.hkv
    w.dq[r, h * group:(h + 1) * group, 0] = 100.0   # times element 0 of the keys: it decides
    pages, slots = (a.to(DEV) for a in w.at[r])
    w.dk[pages, slots, h, 0] = 0
    low = min(len(pages) - 1, 128)                  # the first part of a row that is cut up
    w.dk[pages[:low], slots[:low], h, 0] = int(torch.tensor([-1000.0]).to(torch.bfloat16).view(torch.int16))
    put(w, 1, r, 0, h, 3, INF16)
    put(w, 1, r, 0, h, 4, NINF16)
    got = call(w)
    assert np.all(got[r, h * group:(h + 1) * group, 3] == np.inf)
    assert np.all(got[r, h * group:(h + 1) * group, 4] == -np.inf)
    got[r, h * group:(h + 1) * group, 3:5] = 0
    assert np.all(np.isfinite(got))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS)
def test_scores_of_minus_infinity_leave_zeros(form, out):
    """All of a head's keys give -inf: zeros, with finite values, infinities and NaN alike."""
    w = world(form, out, 33)
    o, tol = w.want()
    group, n = w.hq // w.hkv, w.lens[0]
    w.q[0, :group, 2] = 1.5
    w.dq[0, :group, 2] = 1.5
    pages, slots = (a.to(DEV) for a in w.at[0])
    w.dk[pages, slots, 0, 2] = NINF16
    for t, d, bits in ((0, 1, INF16), (n - 1, 1, NINF16), (n // 2, 5, NAN16), (1, 6, NINF16)):
        put(w, 1, 0, t, 0, d, bits)
    got = call(w)
    assert np.all(got[0, :group] == 0)
    got[0, :group] = o[0, :group]
    assert np.all(np.abs(got - o) <= tol)


def test_a_key_that_is_not_finite_reaches_its_heads_alone():
    w = world("runs", "bf16", 34)
    o, tol = w.want()
    put(w, 0, 1, 5, 1, 3, NAN16)
    got = call(w)
    bad = np.zeros(got.shape, bool)
    bad[1, 4:] = True
    assert np.array_equal(np.isnan(got), bad)
    assert np.all(np.abs(got - o)[~bad] <= tol[~bad])


def test_nan_in_an_8_bit_cache_reaches_its_dim_alone():
    w = World([300, 5000], 8, 2, 128, 16, "e4m3", seed=35, out="f32")
    o, tol = w.want()
    put(w, 1, 1, 4000, 1, 9, 0x7F)
    put(w, 1, 0, 299, 0, 100, 0x7F)
    got = call(w)
    bad = np.zeros(got.shape, bool)
    bad[1, 4:, 9] = bad[0, :4, 100] = True
    assert np.array_equal(np.isnan(got), bad)
    assert np.all(np.abs(got - o)[~bad] <= tol[~bad])


@pytest.mark.parametrize("form", FORMS)
def test_infinite_scores(form):
    """A score of +inf makes its heads NaN; one of -inf takes its token out."""
    w = world(form, "f32", 36)
    group, n = w.hq // w.hkv, [w.lens[0] - 1, 5]
    for r in (0, 1):                                # heads of the first kv head: a key's infinity keeps its sign
        w.q[r, :group, 2] = 1.5
        w.dq[r, :group, 2] = 1.5
    o, tol = w.want()                               # of row 0 and the other heads
    pages, slots = w.at[1]
    keep = torch.arange(len(pages)) != n[1]
    w.at[1] = pages[keep], slots[keep]
    without, without_tol = w.want()                 # row 1 without that token
    w.at[1] = pages, slots
    o[1, :group], tol[1, :group] = without[1, :group], without_tol[1, :group]
    put(w, 0, 0, n[0], 0, 2, INF16)
    put(w, 0, 1, n[1], 0, 2, NINF16)
    got = call(w)
    bad = np.zeros(got.shape, bool)
    bad[0, :group] = True
    assert np.array_equal(np.isnan(got), bad)
    assert np.all(np.abs(got - o)[~bad] <= tol[~bad])
