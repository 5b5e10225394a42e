"""GPU: attention of rows with shared prefixes where a head's scores are all
alike: a scale of 0, below 0 or too small to tell scores apart, for all heads or
for one (of an E4M3 cache), with tokens that are not there beside them."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_attn_shared import World

pytestmark = pytest.mark.gpu

# a prefix that ends within a tile, one that has holes and a whole one; groups of few heads and of many
HOLES = [(0, 3), (0, 18)]


def world(rows, kind, holes, out="f32", d=128):
    return World([(300, [300 + i % 40 for i in range(rows)]), (320, [321, 320, 330][:min(rows, 3)]), [33]], 8, 2, d, 16, kind,
                 "heads", out, seed=rows, holes=HOLES if holes else ())


@pytest.mark.parametrize("rows", [3, 40, 70])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("holes", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-45, -1e-45])
def test_a_scale_of_zero_gives_the_mean_of_the_values(rows, kind, holes, scale):
    w = world(rows, kind, holes)
    w.scale = scale
    say("scale", scale, rows, kind, holes)
    w.run(rows=[0, 1, rows - 1, rows, rows + 3 if rows > 3 else rows])


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_a_negative_scale(rows, d, kind, out):
    """What the negated queries give with the positive one."""
    w = world(rows, kind, True, out, d)
    w.dq.neg_()
    w.scale = -w.scale
    raw, got = w.buffer()
    say("negative", rows, d, kind, out)
    w.call(got)
    got = got.cpu().double().numpy()
    w.scale = -w.scale
    for r in (0, 1, rows - 1, rows):
        want, tol = w.want(r)
        assert (np.abs(got[r] - want) <= tol).all(), r


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("value", [0.0, -0.75])
def test_a_head_s_scale_of_zero_and_below(rows, value):
    w = world(rows, "e4m3", True)
    w.ks[1] = value
    w.cache.tensors[2][1] = value
    say("k_scale", rows, value)
    w.run(rows=[0, 1, rows - 1, rows])


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_holes_alone_give_zeros_whatever_a_head_s_scale_is(rows, value):
    """A head whose scale is no number has NaN in every row that sees a token, and zeros in the others."""
    w = World([(64, [64] * rows), (96, [97] * rows), [16], [33]], 8, 2, 128, 16, "e4m3", "heads", "f32",
              holes=[(0, p) for p in range(4)] + [(2 * rows, 0)])
    w.ks[1] = value
    w.cache.tensors[2][1] = value
    raw, out = w.buffer()
    say("holes alone", rows, value)
    w.call(out)
    got = out.cpu().double().numpy()
    assert (got[:rows] == 0).all() and (got[2 * rows] == 0).all()
    assert np.isnan(got[rows:2 * rows, 4:]).all() and np.isnan(got[2 * rows + 1, 4:]).all()
    for r in (rows, 2 * rows - 1, 2 * rows + 1):
        with np.errstate(invalid="ignore"):
            want, tol = w.want(r)
            assert (np.abs(got[r] - want) <= tol)[:4].all()
