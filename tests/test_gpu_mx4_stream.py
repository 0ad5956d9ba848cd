"""GPU tests of rounding matrices that are more than the memory-side cache holds
(256 MB), whose values are loaded past the caches: every form, type and rounding,
against the same call on parts that are small enough not to be, and against the
oracle at the ends.  A part that begins at the first row and column has the same
random words, and the same blocks but for the one that it cuts."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from matrix_aware_optimizer_muon_amd import binding as B
from oracle import mx4 as orc
from tests.parity_common import say

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

SIZES = {torch.bfloat16: (16417, 8201), torch.float32: (16417, 4105)}     # 269 MB


def quantized(x, axes, rounding):
    """The forms of x that are named, by one call."""
    forms = {a: mm.mx4_empty(*x.shape, axis=a) for a in axes}
    d = mm.mx4_desc(x, *forms.values())
    for f in forms.values():
        f.codes.fill_(0x77), f.scales.fill_(0x77)
    status = B.load_library().muon_mx4_quantize(B.ctypes.byref(d), 1, B.ROUNDINGS[rounding], 77,
                                                torch.cuda.current_stream().cuda_stream)
    assert status == 0
    return forms


@pytest.mark.parametrize("dtype", SIZES, ids=["bf16", "f32"])
@pytest.mark.parametrize("axes", [(1,), (0,), (1, 0)])
@pytest.mark.parametrize("rounding", ["nearest", "random"])
def test_as_in_parts(dtype, axes, rounding):
    rows, cols = SIZES[dtype]
    say(f"case: {rows}x{cols} {dtype} {axes} {rounding}")
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp2(torch.randint(-6, 6, (1, cols), generator=gen, device="cuda").float())
    x = x.to(dtype)
    assert x.numel() * x.element_size() > 256 << 20
    whole = quantized(x, axes, rounding)
    r, c = 15360, cols // 128 * 128 - 512
    for part in (x[:r], x[:, :c]):
        assert part.numel() * part.element_size() < 256 << 20
        for a, f in quantized(part, axes, rounding).items():
            lines, blocks = (part.shape[0], -(-part.shape[1] // 32)) if a == 1 else (part.shape[1], -(-part.shape[0] // 32))
            assert torch.equal(whole[a].codes[:lines, :16 * blocks], f.codes[:, :16 * blocks])
            assert torch.equal(whole[a].scales[:lines, :blocks], f.scales[:, :blocks])
    # the last rows and columns, which neither part holds: blocks from multiples of 32 on
    r, c = rows // 32 * 32 - 64, cols // 32 * 32 - 96
    end = x[r:, c:].float().cpu().numpy().astype(np.float64)
    word = _words(77, rows, cols)[r:, c:] if rounding == "random" else None
    for a, f in whole.items():
        codes, scales = orc.quantize(end, a, word)
        at, block = (r, c // 32) if a == 1 else (c, r // 32)
        got = f.codes[at:, 16 * block:16 * block + codes.shape[1]].cpu().numpy()
        assert np.array_equal(got, codes)
        assert np.array_equal(f.scales[at:, block:block + scales.shape[1]].cpu().numpy(), scales)


def _words(seed, rows, cols):
    """The oracle's words of all rows, but only of the last 512 columns or so (zeros before them)."""
    out = np.zeros((rows, cols), np.uint32)
    first = (cols - 512) // 16
    with np.errstate(over="ignore"):
        u = lambda k: np.array([k], np.uint32)  # noqa: E731
        key = orc._mix(orc._mix(orc._mix(u(seed)) + u(0)) + u(0))
        row = orc._mix(key + np.arange(rows, dtype=np.uint32))
        group = orc._mix(row[:, None] + np.arange(first, -(-cols // 16), dtype=np.uint32))
        w = group[:, :, None] + np.arange(16, dtype=np.uint32) * orc.GOLDEN
    out[:, first * 16:] = w.reshape(rows, -1)[:, :cols - first * 16]
    return out


@pytest.mark.parametrize("dtype", SIZES, ids=["bf16", "f32"])
@pytest.mark.parametrize("axis", [1, 0])
def test_read_back_past_the_caches(dtype, axis):
    """Values of more than 4 MB whose rows begin at multiples of 16 bytes, edges inside tiles and blocks, in a wider
    buffer whose other bytes stay; and one of 4 MB, which is kept."""
    for rows, cols, gap in ((2101, 1032, 8), (1301, 2052, 12), (1024, 1024, 0)):
        es = torch.empty((), dtype=dtype).element_size()
        if cols * es % 16 or (cols + gap) * es % 16:
            cols, gap = cols + 4, 0
        say(f"case: {rows}x{cols} {dtype} axis {axis}")
        lines, blocks = (rows, -(-cols // 32)) if axis == 1 else (cols, -(-rows // 32))
        gen = torch.Generator(device="cuda").manual_seed(rows)
        codes = torch.randint(0, 256, (lines, 16 * blocks), generator=gen, device="cuda", dtype=torch.uint8)
        scales = torch.randint(100, 150, (lines, -(-blocks // 4) * 4), generator=gen, device="cuda", dtype=torch.uint8)
        scales[3, 1] = 255
        wide = torch.full((rows, cols + gap), 5.0, dtype=dtype, device="cuda")
        mm.mx4_dequantize(mm.Mx4(codes, scales, rows, cols, axis), out=wide[:, :cols])
        want = orc.dequantize(codes.cpu().numpy(), scales.cpu().numpy(), rows, cols, axis)
        assert np.array_equal(wide[:, :cols].double().cpu().numpy(), want, equal_nan=True)
        assert bool((wide[:, cols:] == 5.0).all())
