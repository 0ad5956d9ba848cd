"""GPU tests of the 4-bit operators at the largest sizes that their calls take:
2^30 rows or columns, lists of more tiles than a launch has, 2^25 samples in
lines of 2^24 bytes, and the widest block of few samples."""

import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from tests.parity_common import say
from tests.test_gpu_mx4_moment import decoded, handle, held

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

MOST = 1 << 30


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def long_vector():
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randint(-32768, 32768, (MOST,), generator=gen, device="cuda", dtype=torch.int16)
    return (x & 0x3FFF).bitwise_or_(x & -32768).view(torch.bfloat16)       # finite, magnitudes up to 2


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("axis", [1, 0])
def test_most_rows_and_columns(tall, axis):
    """Against the same call on parts that begin at a block."""
    shape = (MOST, 1) if tall else (1, MOST)
    say(f"case: {shape[0]}x{shape[1]} bf16, axis {axis}")
    v = long_vector()
    q = mm.mx4_quantize(v.view(shape), axis=axis)
    back = mm.mx4_dequantize(q, dtype=torch.bfloat16).view(-1)
    along = (axis == 0) == tall                     # one line of all elements, or a line for each
    n = 1 << 20
    for at in (0, 128, MOST // 2 - 64 * 1024, MOST - n - 4096, MOST - n):
        part = v[at:at + n].view((n, 1) if tall else (1, n))
        f = mm.mx4_quantize(part, axis=axis)
        if along:
            assert torch.equal(q.codes[0, at // 2:(at + n) // 2], f.codes[0])
            assert torch.equal(q.scales[0, at // 32:(at + n) // 32], f.scales[0])
        else:
            assert torch.equal(q.codes[at:at + n], f.codes) and torch.equal(q.scales[at:at + n, 0], f.scales[:, 0])
        assert torch.equal(back[at:at + n], mm.mx4_dequantize(f, dtype=torch.bfloat16).view(-1))


def test_more_tiles_than_a_launch_has():
    """Three matrices of 2^23 tiles each, of 2^24 - 1 that a launch takes, and small ones between them."""
    say("case: three matrices of 1 x 2^30 and two small ones")
    v, w = long_vector().view(1, MOST), torch.randn(100, 300, device="cuda").bfloat16()
    copies = mm.Mx4Copies([v, w, v, w, v], axis=1)
    copies.quantize()
    alone, small = mm.mx4_quantize(v), mm.mx4_quantize(w)
    for k, (f,) in enumerate(copies.copies):
        want = alone if k % 2 == 0 else small
        assert torch.equal(f.codes, want.codes)
        blocks = -(-f.cols // 32)
        assert torch.equal(f.scales[:, :blocks], want.scales[:, :blocks])


@pytest.mark.parametrize("n", [1 << 25, (1 << 25) - 4097])
def test_longest_lines(n):
    """Lines of 2^24 bytes.  One number in sixteen is 1 or -1, the others 0: sums are whole numbers below 2^24."""
    d = 5
    say(f"case: {n} samples, {d} features")
    gen = torch.Generator(device="cuda").manual_seed(n & 0xFFFF)
    codes = torch.randint(0, 256, (d, 1 << 24), generator=gen, device="cuda", dtype=torch.uint8)
    value = (codes & 15).eq_(3).to(torch.int8) * (1 - 2 * (codes >> 7).to(torch.int8))       # of the even samples
    codes = value.eq(1).to(torch.uint8).mul_(2) + value.eq(-1).to(torch.uint8).mul_(10)
    scales = torch.full((d, 1 << 20), 127, dtype=torch.uint8, device="cuda")
    q = mm.Mx4(codes, scales, n, d, axis=0)
    x = value[:, :-(-n // 2)].double()              # the odd samples are zeros
    want = x @ x.t().contiguous()
    opt = handle(d)
    sums, count = opt.precond_sums(0, 0)
    for k in (1, 2):
        opt.precond_accumulate(0, 0, q)
        assert torch.equal(sums.double(), k * want) and float(count) == k * n
    opt.close()
    with pytest.raises(mm.MuonError):
        opt = handle(d)
        opt.precond_accumulate(0, 0, mm.Mx4(codes.new_zeros(d, (1 << 24) + 16), scales.new_zeros(d, (1 << 20) + 4), n, d, axis=0))


@pytest.mark.parametrize("n", [1, 100, 511])
def test_few_samples_of_the_widest_block(n):
    d = 16384
    say(f"case: {n} samples, {d} features")
    opt = handle(d)
    q = held(n, d, scales=(127, 128))
    opt.precond_accumulate(0, 0, q, beta=0.0)
    sums = opt.precond_sums(0, 0)[0]
    x = decoded(q).float()                          # products are multiples of 1/4 up to 36: exact in float32
    for at in range(0, d, 4096):
        assert torch.equal(sums[at:at + 4096].double(), x[at:at + 4096].double() @ x.double().t().contiguous())
    opt.close()
