"""GPU parity of the second moment of activations in microscaled 4-bit floats.

Products of two numbers of the format are exact in float32, and where the
scales are near 1 so are all their sums: with scales of 1 and 2 a product is a
multiple of 1/4 of at most 144, and 2^24 / 4 / 144 = 29127 samples sum without
rounding.  There the sums are compared for equality with float64, and with those of the
same activations given in float32.

With scales of any size a float32 sum of n products, in whatever order and each
addition off by at most one unit of 2^-23, is off by at most
n 2^-23 sum |x_i x_j|; decaying and adding the sums before is one rounding of
2^-24 of the result."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from oracle import mx4 as orc
from tests.parity_common import say

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def held(n, d, seed=0, scales=(127, 129), wide=0):
    """n samples of d features, codes of every value and scales in a range; behind the samples whatever there is:
    codes, and scales of 255 (NaN)."""
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + n * 31 + d)
    nb = -(-n // 32)
    codes = torch.randint(0, 256, (d, 16 * (nb + wide)), generator=gen, device="cuda", dtype=torch.uint8)
    exps = torch.full((d, -(-nb // 4) * 4 + 4 * wide), 255, device="cuda", dtype=torch.uint8)
    exps[:, :nb] = torch.randint(*scales, (d, nb), generator=gen, device="cuda", dtype=torch.uint8)
    return mm.Mx4(codes[:, :16 * nb], exps[:, :nb], n, d, axis=0)


def decoded(q):
    """d x n float64, on the GPU."""
    grid = torch.tensor(orc.MAGNITUDES, device="cuda")
    c = torch.stack([q.codes & 15, q.codes >> 4], -1).reshape(q.cols, -1)[:, :q.rows]
    x = grid[(c & 7).long()] * (1.0 - 2.0 * (c >> 3).double())
    e = q.scales.double().repeat_interleave(32, 1)[:, :q.rows]
    return x * torch.where(e == 255, torch.nan, torch.exp2(e - 127))


def handle(d, nblocks=1, **kw):
    w, g = (torch.zeros(4, d * nblocks, device="cuda") for _ in range(2))
    m = torch.zeros(4, d * nblocks, device="cuda")
    return mm.MuonStep([mm.tensor_desc(w, g, m, precond=0)], mm.default_hparams(),
                       preconds=[mm.MuonPrecond(d, nblocks, 0)], keepalive=[w, g, m], **kw)


def padding(opt, d):
    """The sums' rows and columns behind the d-th."""
    sums = opt.precond_sums(0, 0)[0]
    ld = sums.stride(0)
    full = torch.as_strided(sums, (ld, ld), (ld, 1), sums.storage_offset())
    return full[d:], full[:, d:]


SIZES = [(1, 1), (1, 768), (31, 5), (32, 128), (33, 129), (64, 100), (255, 127), (256, 256), (257, 257), (1000, 200),
         (511, 384), (4101, 768), (20000, 300), (29000, 31), (2049, 1025), (700, 1600)]


@pytest.mark.parametrize("n,d", SIZES)
def test_sums_are_exact(n, d):
    say(f"case: sums of {n} samples, {d} features")
    opt = handle(d)
    sums, count = opt.precond_sums(0, 0)
    assert sums.shape == (d, d) and float(count) == 0 and not bool(sums.any())
    a, b = held(n, d), held(max(1, n // 3), d, 1, wide=3)
    xa, xb = decoded(a), decoded(b)
    sa, sb = xa @ xa.t().contiguous(), xb @ xb.t().contiguous()
    opt.precond_accumulate(0, 0, a, beta=1.0)
    assert torch.equal(sums.double(), sa) and float(count) == n
    opt.precond_accumulate(0, 0, b, beta=0.5)
    assert torch.equal(sums.double(), 0.5 * sa + sb) and float(count) == 0.5 * n + b.rows
    sums.fill_(float("nan"))
    opt.precond_accumulate(0, 0, a, beta=0.0)      # what was there does not count
    assert torch.equal(sums.double(), sa) and float(count) == n
    assert not any(bool(p.any()) for p in padding(opt, d))
    assert torch.equal(sums, sums.t())
    opt.close()


@pytest.mark.parametrize("n,d", [(511, 1300), (512, 1300), (513, 1300), (600, 1153), (767, 1281), (768, 1600), (800, 2000),
                                 (1023, 1153), (1024, 1200), (1025, 1400), (1536, 1100), (1600, 500), (1792, 130),
                                 (2303, 1290), (2816, 40), (5120, 1025), (7000, 3), (9999, 2700), (34309, 2100),
                                 (34560, 2100), (100001, 2049), (4096, 2560), (5003, 2561), (8200, 2500), (9000, 3300),
                                 (20011, 1601), (3000, 4100), (12000, 4096), (520, 5000), (2600, 5000), (700, 4200),
                                 (65537, 700)])
def test_sums_are_exact_in_every_way(n, d):
    """Bands and tiles of every size, whole and cut, with every length of the last stage's kind.  Scales of 1: products
    are multiples of 1/4 up to 36, exact for 116508 samples."""
    say(f"case: sums of {n} samples, {d} features")
    opt = handle(d)
    sums, count = opt.precond_sums(0, 0)
    q = held(n, d, scales=(127, 128), wide=1)
    x = decoded(q)
    want = x @ x.t().contiguous()
    for beta in (0.0, 1.0):
        sums.fill_(3.0 if beta else float("nan"))
        count.fill_(7.0)
        opt.precond_accumulate(0, 0, q, beta=beta)
        assert torch.equal(sums.double(), want + 3.0 * beta) and float(count) == n + 7.0 * beta
        assert not any(bool(p.any()) for p in padding(opt, d))
    assert opt.flags() == 0
    opt.close()


@pytest.mark.parametrize("n,d", [(100, 64), (5003, 300), (40000, 129), (65536, 768), (40000, 2100)])
def test_sums_with_scales_of_any_size(n, d):
    say(f"case: sums of {n} samples, {d} features, scales 2^-20 .. 2^20")
    opt = handle(d)
    sums, count = opt.precond_sums(0, 0)
    old = torch.randn(d, d, device="cuda")
    old = old + old.t()
    sums.copy_(old)
    q = held(n, d, scales=(107, 148))
    x = decoded(q)
    want, size = x @ x.t().contiguous(), x.abs() @ x.abs().t().contiguous()
    opt.precond_accumulate(0, 0, q, beta=0.9)
    part = 0.9 * old.double()
    bound = n * 2.0 ** -23 * size + 2.0 ** -24 * (part.abs() + size)
    err = (sums.double() - (part + want)).abs()
    say(f"  largest error over its bound {float((err / bound).max()):.2e}, relative (F) "
        f"{float((err.norm() / want.norm())):.2e}")
    assert bool((err <= bound).all())
    opt.close()


def test_ends_of_the_scales():
    """Scale 2^-127 squared is below float32: zero.  2^100 squared is above: infinite, as in float32 arithmetic."""
    opt = handle(3)
    codes = torch.full((3, 16), 0x22, dtype=torch.uint8, device="cuda")      # ones
    scales = torch.tensor([[0], [227], [127]], dtype=torch.uint8, device="cuda")
    scales = torch.cat([scales] * 4, 1)
    opt.precond_accumulate(0, 0, mm.Mx4(codes, scales, 32, 3, axis=0))
    sums = opt.precond_sums(0, 0)[0]
    assert float(sums[0, 0]) == 0 and float(sums[1, 1]) == float("inf") and float(sums[2, 2]) == 32
    assert float(sums[0, 1]) == 32 * 2.0 ** -27 and float(sums[1, 2]) == 32 * 2.0 ** 100
    opt.close()


def test_not_finite_features():
    """A block that is not finite makes its feature's row and column NaN, and the factorisation fails as with NaN."""
    q = held(500, 200, 4)
    q.scales[77, 3] = 255
    opt = handle(200)
    opt.precond_accumulate(0, 0, q)
    sums = opt.precond_sums(0, 0)[0]
    bad = torch.isnan(sums)
    assert bool(bad[77].all()) and bool(bad[:, 77].all()) and int(bad.sum()) == 399
    opt.precond_refresh_accumulated(0, 0, damping=1.0)
    torch.cuda.synchronize()
    assert opt.flags() & 2
    opt.close()


@pytest.mark.parametrize("n,d", [(100, 64), (4096, 200), (5000, 768)])
def test_refresh_equals_the_float32_activations(n, d):
    """The running sums of both have the same bits, so S^-1 and the step have.  Of a one-shot refresh the diagonal
    (a product and a sum, fused or not) may differ by a rounding of 2^-24, which the inverse carries on times its
    condition, at most |S| / 0.5."""
    say(f"case: refresh from {n} samples, {d} features")
    q = held(n, d)
    x = decoded(q).t().float().contiguous()
    got = []
    for acts in (q, x):
        for online in (False, True):
            w, g, m = torch.zeros(d, d, device="cuda"), torch.eye(d, device="cuda"), torch.zeros(d, d, device="cuda")
            opt = mm.MuonStep([mm.tensor_desc(w, g, m, precond=0)], mm.default_hparams(ns_steps=0),
                              preconds=[mm.MuonPrecond(d, 1, 0)])
            if online:
                opt.precond_accumulate(0, 0, acts)
                opt.precond_refresh_accumulated(0, 0, damping=0.5)
            else:
                opt.precond_refresh(0, 0, acts, damping=0.5)
            opt.step()
            torch.cuda.synchronize()
            assert opt.flags() == 0
            got.append((w, m))
            opt.close()
    assert torch.equal(got[1][0], got[3][0]) and torch.equal(got[1][1], got[3][1])
    xd = x.double()
    s = xd.t().contiguous() @ xd / n + 0.5 * torch.eye(d, device="cuda", dtype=torch.float64)
    want = torch.linalg.inv(s) * (1 - np.float32(0.95))
    cond = float(torch.linalg.matrix_norm(s, 2)) / 0.5
    # 1 / n, the product and the sum: three roundings of S; S^-1 and its part in the momentum: two more
    for _, m in got:
        assert float((m.double() - want).norm() / want.norm()) <= 2.0 ** -24 * (3 * cond + 2)


def test_blocks_slots_and_quantised_activations():
    """Through the whole path: activations rounded along the samples, into two blocks of a slot; the other block stays."""
    n, d = 3001, 192
    opt = handle(d, nblocks=2)
    x = torch.randn(n, d, device="cuda").bfloat16()
    q = mm.mx4_quantize(x, axis=0, rounding="random", seed=9)
    v = mm.mx4_dequantize(q).double()
    opt.precond_accumulate(0, 1, q)
    other, one = opt.precond_sums(0, 0), opt.precond_sums(0, 1)
    assert not bool(other[0].any()) and float(other[1]) == 0 and float(one[1]) == n
    want, size = v.t().contiguous() @ v, v.abs().t().contiguous() @ v.abs()
    assert bool(((one[0].double() - want).abs() <= n * 2.0 ** -23 * size).all())
    opt.close()


def test_refusals_on_a_handle():
    opt = handle(100)
    good = held(64, 100)
    for acts in (held(64, 99), mm.Mx4(good.codes.new_zeros(64, 64), good.codes.new_zeros(64, 4), 64, 100, axis=1)):
        with pytest.raises(ValueError):
            opt.precond_accumulate(0, 0, acts)
        with pytest.raises(ValueError):
            opt.precond_refresh(0, 0, acts)
    for slot, block, beta in ((1, 0, 1.0), (-1, 0, 1.0), (0, 1, 1.0), (0, 0, 1.5), (0, 0, -0.1), (0, 0, float("nan"))):
        with pytest.raises(mm.MuonError):
            opt.precond_accumulate(slot, block, good, beta=beta)
    for damping in (-1.0, float("nan"), float("inf")):
        with pytest.raises(mm.MuonError):
            opt.precond_refresh(0, 0, good, damping=damping)
    for slot, block in ((1, 0), (0, 1), (0, -1)):
        with pytest.raises(mm.MuonError):
            opt.precond_sums(slot, block)
    bad = mm.Mx4(torch.zeros(100, 40, dtype=torch.uint8, device="cuda")[:, :32], good.scales, 64, 100, axis=0)
    with pytest.raises(mm.MuonError):
        opt.precond_accumulate(0, 0, bad)          # lines not 16 bytes apart
    assert float(opt.precond_sums(0, 0)[1]) == 0
    opt.close()


def test_static_handle():
    q = held(1000, 130)
    x = decoded(q)
    opt = handle(130, static_scratch=True)
    with pytest.raises(ValueError):
        opt.precond_sums(0, 0)
    opt.precond_accumulate(0, 0, q)
    opt.precond_refresh_accumulated(0, 0, damping=1.0)
    torch.cuda.synchronize()
    assert opt.flags() == 0 and x.shape == (130, 1000)
    opt.close()


def test_captured_and_replayed():
    """Replays add up as calls do, with the program's own work between them."""
    d, q = 300, held(3000, 300)
    opt, plain = handle(d), handle(d)
    sums, count = opt.precond_sums(0, 0)
    opt.precond_accumulate(0, 0, q, beta=0.5)
    sums.zero_(), count.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        opt.precond_accumulate(0, 0, q, beta=0.5)
    for k in range(5):
        q.codes.copy_(held(3000, 300, k).codes)
        g.replay()
        plain.precond_accumulate(0, 0, q, beta=0.5)
        want = plain.precond_sums(0, 0)
        torch.cuda.synchronize()
        assert torch.equal(sums, want[0]) and torch.equal(count, want[1])
    opt.close(), plain.close()


def test_side_stream():
    d, q = 768, held(9000, 768)
    want = decoded(q)
    want = want @ want.t().contiguous()
    opt = handle(d)
    side = torch.cuda.Stream()
    for _ in range(4):
        sums, _ = opt.precond_sums(0, 0)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            late = held(9000, 768, 5)
            for _ in range(10):
                late.codes.add_(0)
            late.codes.copy_(q.codes), late.scales.copy_(q.scales)
        opt.precond_accumulate(0, 0, late, beta=0.0, stream=side)
        del late
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(sums.double(), want)
    opt.close()


def test_more_than_4_gib_of_codes():
    """The widest preconditioner: lines past 2^32 bytes; every 64th feature is the same."""
    n, d = 540000, 16384
    say(f"case: {n} samples, {d} features")
    few = held(n, 64, scales=(124, 126))
    small = handle(64)
    small.precond_accumulate(0, 0, few)
    x = decoded(few)
    want = small.precond_sums(0, 0)[0]
    size = x.abs() @ x.abs().t().contiguous()
    assert bool(((want.double() - x @ x.t().contiguous()).abs() <= n * 2.0 ** -23 * size).all())
    opt = handle(d)
    opt.precond_accumulate(0, 0, _repeated(few, d))
    sums = opt.precond_sums(0, 0)[0]
    for at in range(0, d, 4096):
        got = sums[at:at + 4096].double().view(64, 64, d // 64, 64)
        exact = (x @ x.t().contiguous())[None, :, None, :]
        assert bool(((got - exact).abs() <= (n * 2.0 ** -23 * size)[None, :, None, :]).all())
    opt.close(), small.close()


def _repeated(q, d):
    nb = -(-q.rows // 32)
    scales = torch.zeros(d, -(-nb // 4) * 4, dtype=torch.uint8, device="cuda")
    scales[:, :nb] = q.scales.repeat(d // q.cols, 1)
    return mm.Mx4(q.codes.repeat(d // q.cols, 1), scales, q.rows, d, axis=0)
