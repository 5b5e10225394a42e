"""The wire's records in 64 bits (numpy): elements as places in a table of all
values, scales as whole exponents."""
import numpy as np

TABLE = {8: np.array([m / 8 * 2.0 ** -6 for m in range(8)]
                     + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]),
         4: np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])}
SIGN = {8: 0x80, 4: 8}


def nearest(y, bits):
    """The code of each y (|y| at most the table's last): nearest, of even code where two are as near; the sign of zero kept."""
    t = TABLE[bits]
    a = np.abs(y)
    assert a.size == 0 or a.max() <= t[-1]
    hi = np.clip(np.searchsorted(t, a), 1, len(t) - 1)
    lo = hi - 1
    up = (t[hi] - a < a - t[lo]) | ((t[hi] - a == a - t[lo]) & (hi % 2 == 0))
    return np.where(up, hi, lo).astype(np.uint8) | np.where(np.signbit(y), SIGN[bits], 0).astype(np.uint8)


def scale_byte(x, bits):
    """[..., 32] finite float64 -> e + 127."""
    top = np.abs(x).max(-1)
    largest = TABLE[bits][-1]
    e = np.full(top.shape, -127)
    while True:
        more = top > largest * 2.0 ** e
        if not more.any():
            return (e + 127).astype(np.uint8)
        e = np.where(more, e + 1, e)


def quantize(x, bits):
    """x [tokens, n] float64, n a multiple of 32 -> (codes [tokens, n], scale bytes [tokens, n / 32])."""
    b = x.reshape(len(x), -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    s = scale_byte(b, bits)
    codes = nearest(b / 2.0 ** (s[..., None].astype(np.int64) - 127), bits)
    return np.where(bad[..., None], 0, codes).astype(np.uint8).reshape(x.shape), np.where(bad, 255, s).astype(np.uint8)


def records(x, bits):
    """The records' bytes of x [tokens, n]."""
    codes, s = quantize(x, bits)
    data = codes if bits == 8 else codes[:, 0::2] | codes[:, 1::2] << 4
    r = np.concatenate([data, s], 1)
    return np.pad(r, ((0, 0), (0, -r.shape[1] % 16)))


def values(record, n, bits):
    """What records of n elements stand for, float64 [tokens, n]."""
    data, s = record[:, :n * bits // 8], record[:, n * bits // 8:n * bits // 8 + n // 32]
    codes = data if bits == 8 else np.stack([data & 15, data >> 4], -1).reshape(len(record), n)
    mag = codes & (SIGN[bits] - 1)
    t = np.append(TABLE[8], np.nan) if bits == 8 else TABLE[4]
    v = np.where(codes & SIGN[bits], -t[mag], t[mag])
    scale = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.int64) - 127))
    return (v.reshape(len(record), -1, 32) * scale[..., None]).reshape(len(record), n)


def bf16_bits(v):
    """float64 -> BF16 patterns, nearest even; NaN as 0x7FC0.  Exact for what has at most 24 significant bits and no
    more bits below binary32's subnormals than that."""
    f = np.abs(v)
    with np.errstate(over="ignore", invalid="ignore"):
        u = f.astype(np.float32)
        assert np.array_equal(u.astype(np.float64)[np.isfinite(u)], f[np.isfinite(u)])
    w = u.view(np.uint32).astype(np.uint64)
    r = ((w + 0x7FFF + (w >> 16 & 1)) >> 16).astype(np.uint16)
    r = np.where(np.isinf(u), 0x7F80, r) | np.where(np.signbit(v), 0x8000, 0).astype(np.uint16)
    return np.where(np.isnan(v), 0x7FC0, r).astype(np.uint16)
