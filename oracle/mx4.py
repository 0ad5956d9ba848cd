"""Oracle of microscaled 4-bit floats: NumPy, from the definition in
include/muon.h, sharing no code with the library.  Rounding is done in float64
on the value grid itself (no bit tricks), so codes and scales can be compared
for equality."""

import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALE_MOST = 252
NAN = 255
GOLDEN, ROOT3 = np.uint32(0x9E3779B9), np.uint32(0xBB67AE85)


def _mix(x):
    with np.errstate(over="ignore"):
        x = (x ^ (x >> np.uint32(16))) * GOLDEN
        x = (x ^ (x >> np.uint32(15))) * ROOT3
    return x ^ (x >> np.uint32(16))


def words(seed, index, rows, cols):
    """The random word of each element of the index-th matrix of a list."""
    u = lambda k: np.array([k & 0xFFFFFFFF], np.uint32)  # noqa: E731
    with np.errstate(over="ignore"):
        key = _mix(_mix(_mix(u(seed)) + u(seed >> 32)) + u(index))
        row = _mix(key + np.arange(rows, dtype=np.uint32))
        group = _mix(row[:, None] + np.arange(-(-cols // 16), dtype=np.uint32))
        w = group[:, :, None] + np.arange(16, dtype=np.uint32) * GOLDEN
    return w.reshape(rows, -1)[:, :cols]


def _lines(x, axis, fill):
    """Lines of whole blocks, [lines, blocks, 32]."""
    x = np.asarray(x)
    x = x if axis == 1 else x.T
    pad = -x.shape[1] % BLOCK
    return np.pad(x, ((0, 0), (0, pad)), constant_values=fill).reshape(x.shape[0], -1, BLOCK)


def quantize(x, axis, word=None):
    """(codes [lines, 16 blocks], scales [lines, blocks]) of a matrix of float32 or bfloat16 values, given as
    float64; word: the elements' random words, or None for rounding to nearest."""
    v = _lines(np.asarray(x, np.float64), axis, 0.0)
    bad = ~np.isfinite(v).all(-1)
    a = np.where(bad[..., None], 0.0, np.abs(v))
    amax = a.max(-1)
    mant, k = np.frexp(amax)                       # mant in [0.5, 1): amax <= 6 2^(k-3) up to mant 0.75
    e = np.where(amax > 0, k - 3 + (mant > 0.75), -127)
    e = np.clip(e, -127, SCALE_MOST - 127)
    a = np.minimum(np.ldexp(a, -e[..., None]), 6.0)
    low = np.minimum(np.searchsorted(MAGNITUDES, a, side="right") - 1, 6)
    share = (a - MAGNITUDES[low]) / (MAGNITUDES[low + 1] - MAGNITUDES[low])
    if word is None:
        up = (share > 0.5) | ((share == 0.5) & (low % 2 == 1))
    else:
        up = share + (_lines(word, axis, 0) >> np.uint32(10)) / 2.0 ** 22 >= 1
    code = low + up + 8 * np.signbit(v)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    code = code.reshape(code.shape[0], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), np.where(bad, NAN, e + 127).astype(np.uint8)


def dequantize(codes, scales, rows, cols, axis):
    """The values, float64."""
    code = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1, BLOCK)
    v = np.where(code & 8, -1.0, 1.0) * MAGNITUDES[code & 7]
    v = np.ldexp(v, scales[:, :code.shape[1], None].astype(np.int64) - 127)
    v = np.where((scales[:, :code.shape[1]] == NAN)[..., None], np.nan, v).reshape(codes.shape[0], -1)
    return v[:, :cols] if axis == 1 else v[:, :rows].T
