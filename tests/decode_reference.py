"""The decode-step operators' formulas in 64 bits (numpy), one element or row
at a time where that keeps them plain, and how far a binary32 computation
with one rounding at its end may be from them."""
import numpy as np

# Half a step, relative to the value, of a rounding to nearest.
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24, "e4m3": 2.0 ** -4}
E4M3_MAX = 448.0
E4M3_TINY = 2.0 ** -10  # half the step below the smallest normal number


def rope_heads(x, weight, eps, cos_sin, positions, rot_dim, interleaved):
    """x: [tokens, heads, D] -> (y, mag): the normalised and rotated heads, and
    for each element the sum of the two magnitudes its rotation adds up (of
    an element that is not rotated, its own magnitude)."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y, mag = x.copy(), np.abs(x)
    half = rot_dim // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c = cos_sin[positions, i].astype(np.float64)[:, None]
        s = cos_sin[positions, half + i].astype(np.float64)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        m = np.abs(x[..., a]) + np.abs(x[..., b])
        mag[..., a] = mag[..., b] = m
    return y, mag


def rope_tolerance(y, mag, kind):
    """The norm's sum takes at most 8 + 5 additions, each off by 2^-24, halved
    by the square root; the reciprocal root 2^-23, two products 2^-23, the
    rotation's two products and sum 3 * 2^-24 of each side: below 2^-20 of the
    magnitudes together.  Then the one rounding of the result."""
    err = 2.0 ** -20 * mag
    if kind == "e4m3":
        return err * (1 + HALF["e4m3"]) + np.maximum(HALF["e4m3"] * np.abs(y), E4M3_TINY)
    return err * (1 + HALF[kind]) + HALF[kind] * np.abs(y)


def visible(n, window, sinks):
    """Positions of the tokens that a row of n tokens sees."""
    j = np.arange(n)
    return j if window == 0 else j[(j >= n - window) | (j < sinks)]


def attention(q, k, v, scale):
    """One row: q [heads, D], k, v [tokens, kv heads, D] in the values they
    stand for -> (out, tolerance before the last rounding).

    The products of BF16 (or E4M3) numbers are exact in binary32; their sum of
    D terms is off by at most 2 * D * 2^-24 of the magnitudes (twice what plain
    additions may lose, for the matrix cores' own order), the scale and the
    logarithm's base by 2^-22 of the score.  A weight is off by that, by
    2^-18 of its split and 2^-21 of the power; numerator and denominator each
    carry it; every addition of the sums adds 2^-24."""
    heads, d = q.shape
    n, kv, _ = k.shape
    out, tol = np.zeros((heads, d)), np.zeros((heads, d))
    if n == 0:
        return out, tol
    group = heads // kv
    for h in range(heads):
        kh, vh = k[:, h // group], v[:, h // group]
        s = kh @ q[h] * scale
        w = np.exp(s - s.max())
        w /= w.sum()
        out[h] = w @ vh
        delta = 2 * d * 2.0 ** -24 * (np.abs(kh) @ np.abs(q[h])) * scale + 2.0 ** -22 * np.abs(s)
        # an error of the largest score moves every weight alike
        weight = delta + delta[s.argmax()] + 2.0 ** -18 + 2.0 ** -21 + (n + 64) * 2.0 ** -24
        tol[h] = 2 * ((w * weight) @ np.abs(vh)) + (w @ weight) * np.abs(out[h])
    return out, tol


def sample(values, ids, temperature, top_k, top_p, min_p, u):
    """One row: values (float64, in any order) with their ids -> (id, probability, margin), margin
    being how near u * Z comes to a border of the drawn element, relative to Z."""
    order = np.lexsort((ids, -values))
    order = order[values[order] > -np.inf]                 # NaN compares false
    if order.size == 0:
        return -1, 0.0, 1.0
    x = values[order]
    greedy = not temperature > 0
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.exp((x - x[0]) / (1.0 if greedy else temperature))
    w[x == x[0]] = 1.0
    if np.isinf(x[0]):
        w[x != x[0]] = 0.0
    n = 1 if greedy else x.size if top_k == 0 else min(top_k, x.size)
    w = w[:n]
    if top_p < 1:
        sums = np.cumsum(w)
        w = w[:max(1, int(np.searchsorted(sums, top_p * sums[-1], side="left")) + 1)]
    if min_p == min_p:
        w = w[w >= min(min_p, 1.0)]
    sums = np.cumsum(w)
    target = (u if u > 0 else 0.0) * sums[-1]
    at = min(int(np.searchsorted(sums, target, side="right")), w.size - 1)
    margin = np.min(np.abs(sums - target)) / sums[-1]
    return int(ids[order[at]]), float(w[at] / sums[-1]), float(margin)
