"""Oracle of AdamW's packed (8-bit) moments and of gradient clipping: NumPy,
from the definitions in include/muon.h, sharing no code with the library.

Two views of one definition:
- bytes: the float32 arithmetic (every operation rounded by itself, as NumPy
  does), the random words and the rounding, so bytes and scales can be
  compared for equality;
- values: float64 throughout, for what the update should be.
"""

import numpy as np

BLOCK = 256
GOLDEN, ROOT3 = np.uint32(0x9E3779B9), np.uint32(0xBB67AE85)
F32_INF = 0x7F800000
MOST = 0x7F700000              # 1.875 * 2^127, the largest magnitude a byte stands for
SCALE_LEAST = 9

# e4m3 (OCP): 4 exponent bits of bias 7, 3 mantissa bits, subnormals, no
# infinity, NaN where all seven magnitude bits are set
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)])
E4M3[127] = np.nan


def moment_bytes(n):
    return -(-n // BLOCK) * (BLOCK + 2)


def _mix(x):
    with np.errstate(over="ignore"):
        x = (x ^ (x >> np.uint32(16))) * GOLDEN
        x = (x ^ (x >> np.uint32(15))) * ROOT3
    return x ^ (x >> np.uint32(16))


def words(seed, t, tensor, n):
    """The random word of each of n elements."""
    u = lambda k: np.array([k & 0xFFFFFFFF], np.uint32)  # noqa: E731
    with np.errstate(over="ignore"):
        key = _mix(_mix(_mix(_mix(u(seed)) + u(seed >> 32)) + u(t)) + u(tensor))
        group = _mix(key + np.arange(-(-n // 16), dtype=np.uint32))
        w = group[:, None] + np.arange(16, dtype=np.uint32) * GOLDEN
    return w.reshape(-1)[:n]


def _blocks(x):
    x = np.asarray(x).reshape(-1)
    return np.concatenate([x, np.zeros(-x.size % BLOCK, x.dtype)]).reshape(-1, BLOCK)


def encode(m, v, word=None):
    """Float32 moments (flat) to their two buffers; word: the elements' random
    words, None rounds to nearest, ties to even."""
    m, v = _blocks(np.asarray(m, np.float32)), _blocks(np.asarray(v, np.float32)).copy()
    nb = m.shape[0]
    w = None if word is None else _blocks(np.asarray(word, np.uint32)).astype(np.int64)
    ok = np.isfinite(m)
    mag = np.minimum(np.where(ok, np.abs(m), np.float32(0)), np.float32(1.875 * 2.0 ** 127))
    vbits = np.minimum((v.view(np.uint32) & 0x7FFFFFFF).astype(np.int64), MOST)
    vbits[~ok] = 0
    # first moment
    top = mag.max(1).view(np.uint32).astype(np.int64)
    e = np.maximum(((top + 0x1FFFFF) >> 23) - 8, SCALE_LEAST)
    a = mag.astype(np.float64) * 2.0 ** (127.0 - e)[:, None]
    low = np.searchsorted(E4M3[:127], a, side="right") - 1
    gap = np.where(low < 126, E4M3[np.minimum(low + 1, 126)] - E4M3[low], 32.0)
    share = (a - E4M3[low]) / gap
    up = (share > 0.5) | ((share == 0.5) & (low % 2 == 1)) if w is None else share + (w >> 12) / 2.0 ** 20 >= 1
    code = np.where(ok, low + up, 127) | (np.signbit(m).astype(np.int64) << 7)
    # second moment
    base = np.maximum(((vbits.max(1) + 0xFFFFF) >> 20) - 255, 0)
    idx = vbits + (0x7FFFF + ((vbits >> 20) & 1) if w is None else (w & 0xFFFFF)) >> 20
    code2 = np.maximum(idx - base[:, None], (vbits > 0).astype(np.int64))
    assert code2.max(initial=0) <= 255 and base.max(initial=0) <= 0xFFFF

    def buffer(c, s):
        return np.concatenate([c.astype(np.uint8).reshape(-1), s.astype("<u2").view(np.uint8)])
    assert nb * (BLOCK + 2) == buffer(code, e).size
    return buffer(code, e), buffer(code2, base)


def decode(first, second, n):
    """The float64 values of two buffers."""
    nb = -(-n // BLOCK)
    code, e = first[:nb * BLOCK].reshape(nb, BLOCK), first[nb * BLOCK:].view("<u2").astype(np.int64)
    e = np.maximum(e, SCALE_LEAST)          # a zero-filled buffer
    m = E4M3[code & 127] * np.where(code & 128, -1.0, 1.0) * (2.0 ** (e - 127.0))[:, None]
    code2, base = second[:nb * BLOCK].reshape(nb, BLOCK).astype(np.int64), second[nb * BLOCK:].view("<u2")
    bits = np.where(code2 > 0, (code2 + base.astype(np.int64)[:, None]) << 20, 0)
    v = bits.astype(np.uint32).view(np.float32).astype(np.float64)
    return m.reshape(-1)[:n], v.reshape(-1)[:n]


def moments_f32(g, m, v, betas, factor=1.0):
    """m' and v' in float32, every operation rounded by itself."""
    f = np.float32
    b1, b2 = f(betas[0]), f(betas[1])
    with np.errstate(all="ignore"):
        g = np.asarray(g, f) * f(factor)
        m1 = b1 * np.asarray(m, f) + (f(1) - b1) * g
        v1 = b2 * np.asarray(v, f) + ((f(1) - b2) * g) * g
    return m1, v1


def update(w, m1, v1, t, lr, betas, eps, weight_decay):
    """The updated weight in float64, and the size of its update term."""
    m1, v1, w = (np.asarray(x, np.float64) for x in (m1, v1, w))
    with np.errstate(all="ignore"):
        term = lr * (m1 / (1 - betas[0] ** t)) / (np.sqrt(v1 / (1 - betas[1] ** t)) + eps)
        return w - lr * weight_decay * w - term, np.abs(term)


def clip(grads, max_norm):
    """(norm, factor) of a list of gradients."""
    with np.errstate(all="ignore"):
        norm = float(np.sqrt(sum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads)))
    if norm <= max_norm or max_norm == np.inf:
        return norm, 1.0
    return norm, max_norm / norm
