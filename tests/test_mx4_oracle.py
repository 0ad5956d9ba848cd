"""Pins of the oracle of microscaled 4-bit floats (CPU only): the definition
by brute force, the errors that include/muon.h states, the mean of random
rounding, and planted mistakes that a pin has to notice."""

import itertools

import numpy as np
import pytest

from oracle import mx4 as orc

GRID = [s * m for s in (1.0, -1.0) for m in orc.MAGNITUDES]


def values(x, axis=1, word=None):
    codes, scales = orc.quantize(x, axis, word)
    return orc.dequantize(codes, scales, x.shape[0], x.shape[1], axis)


def by_hand(line, word=None):
    """One block, one element after another, in Python numbers."""
    if not all(np.isfinite(line)):
        return 255, [0] * 32
    amax = max(abs(v) for v in line)
    e = 0
    while e < 252 and amax > 6.0 * 2.0 ** (e - 127):
        e += 1
    codes = []
    for i, v in enumerate(line):
        a = min(abs(v) / 2.0 ** (e - 127), 6.0)
        near = sorted(range(8), key=lambda c: (abs(orc.MAGNITUDES[c] - a), c % 2))[0]
        if word is not None:
            step = 0.5 if a < 2 else 1.0 if a < 4 else 2.0
            target = min(np.floor(a / step + (int(word[i]) >> 10) / 2.0 ** 22) * step, 6.0)
            near = list(orc.MAGNITUDES).index(target)
        codes.append(near + (8 if np.signbit(v) else 0))
    return e, codes


def lines(rng):
    """Blocks of every magnitude, with ties, zeros, the ends of the range and numbers that are not finite."""
    out = []
    for e in (-149, -140, -127, -126, -20, 0, 5, 100, 124, 125, 126, 127):
        for k in range(6):
            x = (rng.standard_normal(32) * 2.0 ** min(e, 124)).astype(np.float32)
            if k == 1:
                x = (rng.integers(-28, 29, 32) * 0.25 * 2.0 ** max(min(e, 124), -147)).astype(np.float32)   # ties
            if k == 2:
                x[rng.integers(0, 32, 20)] = 0.0
            if k == 3:
                x[:] = -0.0
                x[7] = np.float32(2.0 ** max(e, -149))
            if k == 4:
                x = np.full(32, np.float32(3.4028234663852886e38) if e > 125 else np.float32(6 * 2.0 ** e), np.float32)
            if k == 5:
                x[3] = (np.nan, np.inf, -np.inf)[e % 3]
            out.append(x)
    return np.stack(out)


@pytest.mark.parametrize("random", [False, True])
def test_definition_by_hand(random):
    rng = np.random.default_rng(5)
    x = lines(rng)
    word = orc.words(77, 3, *x.shape) if random else None
    codes, scales = orc.quantize(x.astype(np.float64), 1, word)
    for i, row in enumerate(x.astype(np.float64)):
        e, c = by_hand(row, None if word is None else word[i])
        assert scales[i, 0] == e, i
        assert [int(b) for b in np.stack([codes[i] & 15, codes[i] >> 4], -1).reshape(-1)] == c, i


def test_scale_rule_in_bits():
    """The formula that the comments state, against the smallest power of two."""
    rng = np.random.default_rng(6)
    amax = np.concatenate([rng.integers(0, 0x7F800000, 200000), np.arange(0x400000, 0x7F000000, 0x400000),
                           np.arange(0x400000, 0x7F000000, 0x400000) + 1, [0, 1, 0x7F7FFFFF]]).astype(np.uint32)
    by_bits = np.clip(((amax.astype(np.int64) + 0x3FFFFF) >> 23) - 2, 0, 252)
    x = np.zeros((amax.size, 1))
    x[:, 0] = amax.view(np.float32)
    assert np.array_equal(orc.quantize(x, 1)[1][:, 0], by_bits)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (33, 1), (5, 32), (64, 33), (31, 100)])
def test_forms_are_each_others_transpose(rows, cols):
    x = np.random.default_rng(rows * cols).standard_normal((rows, cols))
    a, b = orc.quantize(x, 0), orc.quantize(x.T, 1)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    assert a[0].shape == (cols, -(-rows // 32) * 16) and a[1].shape == (cols, -(-rows // 32))
    assert np.array_equal(orc.dequantize(*a, rows, cols, 0), orc.dequantize(*b, cols, rows, 1).T)
    w = orc.words(9, 0, rows, cols)
    r = orc.quantize(x, 0, w)
    assert np.array_equal(r[0], orc.quantize(x.T, 1, np.ascontiguousarray(w.T))[0])


def test_values_are_held():
    """Every number of the grid times any scale comes back as it was, and a second rounding changes nothing."""
    for e in (-127, -50, 0, 80, 125):
        x = np.array([[v * 2.0 ** e for v in GRID * 2]])
        assert np.array_equal(values(x), x)
    rng = np.random.default_rng(3)
    once = values(rng.standard_normal((50, 96)))
    assert np.array_equal(values(once), once)


def test_errors_of_rounding():
    """To nearest at most half the distance of the two numbers around, and a fifth of the block's largest (the
    element 5 scales, itself the largest, is held as 4); at random less than the distance."""
    x = np.random.default_rng(4).standard_normal((4000, 32))
    most = np.abs(x).max(1, keepdims=True)
    assert np.all(np.abs(values(x) - x) <= most / 5)
    a = np.abs(x)
    held = np.abs(values(x))
    step = lambda scale: np.where(a < 2 * scale, 0.5, np.where(a < 4 * scale, 1, 2)) * scale  # noqa: E731
    scale = 2.0 ** (orc.quantize(x, 1)[1].astype(float) - 127)
    assert np.all(np.abs(held - a) <= step(scale) / 2)
    w = orc.words(1, 0, *x.shape)
    assert np.all(np.abs(np.abs(values(x, 1, w)) - a) < step(scale))


def test_random_rounding_has_the_values_mean():
    """1000 seeds: the mean of independent errors of at most one step has a deviation of at most step / 2 / sqrt(1000);
    five of those for 960 elements (a chance of 6e-4 in all at the very most)."""
    x = np.random.default_rng(8).standard_normal((30, 32))
    mean = np.mean([values(x, 1, orc.words(s, 0, 30, 32)) for s in range(1000)], 0)
    scale = 2.0 ** (orc.quantize(x, 1)[1].astype(float) - 127)
    step = np.where(np.abs(x) < 2 * scale, 0.5, np.where(np.abs(x) < 4 * scale, 1, 2)) * scale
    assert np.all(np.abs(mean - x) <= 5 * step / 2 / np.sqrt(1000))


def test_words_differ_by_all_they_depend_on():
    base = orc.words(1, 0, 40, 100)
    for other in (orc.words(2, 0, 40, 100), orc.words(1 + (1 << 32), 0, 40, 100), orc.words(1, 1, 40, 100)):
        assert np.mean(other == base) < 1e-3
    assert np.unique(base).size > 0.999 * base.size
    assert np.array_equal(orc.words(1, 0, 7, 33), base[:7, :33])      # a function of the place alone
    share = (orc.words(3, 0, 500, 500) >> np.uint32(10)) / 2.0 ** 22
    counts = np.histogram(share, 16, (0, 1))[0]
    assert np.abs(counts - 250000 / 16).max() < 5 * np.sqrt(250000 / 16)


def _mistakes():
    def ties_up(a, low, share, word):
        return share >= 0.5

    def ties_down(a, low, share, word):
        return share > 0.5
    return {"ties up": ties_up, "ties down": ties_down}


@pytest.mark.parametrize("name", sorted(_mistakes()))
def test_planted_mistakes_in_ties_are_noticed(name):
    """The hand-made blocks hold ties both ways."""
    wrong = _mistakes()[name]
    x = lines(np.random.default_rng(5)).astype(np.float64)
    right, scales = orc.quantize(x, 1)
    differ = False
    for i, row in enumerate(x):
        if scales[i, 0] == 255:
            continue
        a = np.minimum(np.abs(row) / 2.0 ** (int(scales[i, 0]) - 127), 6)
        low = np.minimum(np.searchsorted(orc.MAGNITUDES, a, side="right") - 1, 6)
        share = (a - orc.MAGNITUDES[low]) / (orc.MAGNITUDES[low + 1] - orc.MAGNITUDES[low])
        code = low + wrong(a, low, share, None) + 8 * np.signbit(row)
        differ |= not np.array_equal(code[::2] | (code[1::2] << 4), right[i])
    assert differ


def test_grid_is_the_format():
    """e2m1: exponent bias 1, one bit of mantissa, no infinity."""
    for code, (e, m) in enumerate(itertools.product(range(4), range(2))):
        assert orc.MAGNITUDES[code] == (0.5 * m if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1))
