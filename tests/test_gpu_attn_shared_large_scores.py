"""GPU: attention of rows with shared prefixes where scores are large: what is
alike stays alike in every tile, and what lies far apart stays finite."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_attn_shared import World

pytestmark = pytest.mark.gpu


def world(rows, out, d=128, keys=None, queries=1.0):
    """Every key is `keys` (of its token) in dim 0 and 0 elsewhere, every query `queries`; lengths past a tile's end."""
    w = World([(300, [300 + i % 40 for i in range(rows)]), [75]], 4, 1, d, 16, out=out, seed=rows)
    for r, (pages, slots) in enumerate(w.at):
        w.k[pages, slots] = 0
        w.k[pages, slots, :, 0] = torch.tensor(keys(np.arange(len(pages))), dtype=torch.float32).to(torch.bfloat16).view(torch.int16)[:, None]
    w.dk.copy_(w.k)
    w.q[:] = 0
    w.q[..., 0] = queries
    w.dq.copy_(w.q)
    return w


def check(w, rows, counted):
    """`counted`(tokens) says which of a row's tokens share all the weight, evenly: the mean of their values, but for sums
    of n numbers in binary32, the weights' split, one division, and scores that are rounded in one way through and not in
    the other: 2^-24 of up to 128 powers of two, above which they are rounded in both."""
    raw, out = w.buffer()
    w.call(out)
    got = out.cpu().double().numpy()
    assert (raw.cpu()[:, -8 * (2 if w.out_kind == "bf16" else 4):] == 0x5A).all()
    half = 2.0 ** -8 if w.out_kind == "bf16" else 2.0 ** -24
    split = 2.0 ** -17 if w.out_kind == "bf16" else 0.0
    for r in rows:
        v = w.values(w.v, None, r)[:, 0]
        top = counted(np.arange(len(v)))
        v = v[top] if top.any() else v                       # or all of them are alike
        mean, size = v.mean(0), np.abs(v).mean(0)
        tol = 2 * (split + (len(v) + 70) * 2.0 ** -24 + 2.0 ** -17) * size
        tol = tol * (1 + half) + half * np.abs(mean)
        assert np.isfinite(got[r]).all(), r
        assert (np.abs(got[r] - mean) <= tol).all(), (r, np.abs(got[r] - mean).max())


SIZES = [1.0, 2.0 ** 9, 2.0 ** 15, 2.0 ** 20, 2.0 ** 30, 2.0 ** 60]


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_are_all_alike_weigh_alike(rows, out, size, sign):
    """1.5 * 1.25 * size^2 * 0.3, of either sign: no power of two, so that a product with the scale is rounded."""
    w = world(rows, out, keys=lambda j: np.full(len(j), sign * 1.5 * size), queries=1.25 * size)
    w.scale = 0.3
    say("alike", rows, out, size, sign)
    check(w, [0, 1, rows - 1, rows], lambda j: j >= 0)


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES[2:] + [2.0 ** 63])
@pytest.mark.parametrize("first_low", [True, False])
@pytest.mark.parametrize("scale", [1.5, -1.5])
def test_scores_that_lie_far_apart_stay_finite(rows, out, size, first_low, scale):
    """Scores of 1.5 size^2 and its negative, by turns of 70 tokens: for the largest their difference is past binary32."""
    up = lambda j: (j // 70 % 2 == 1) == first_low  # noqa: E731
    flip = -1 if scale < 0 else 1
    w = world(rows, out, keys=lambda j: np.where(up(j), flip * size, -flip * size), queries=size)
    w.scale = scale
    say("apart", rows, out, size, first_low, scale)
    check(w, [0, 1, rows - 1, rows], up)


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 63])
def test_other_heads(rows, d, size):
    up = lambda j: j % 100 > 80  # noqa: E731
    w = world(rows, "f32", d, keys=lambda j: np.where(up(j), size, -size), queries=size)
    w.scale = 1.5
    say("heads of", d, rows, size)
    check(w, [0, 1, rows - 1, rows], up)
