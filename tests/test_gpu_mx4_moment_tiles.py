"""GPU tests of the second moment of 4-bit activations where whole tiles of 256
(and of 128) finish in their own launch, alone and beside tiles that are cut into
ranges, over one round of the chip and more: sums that float32 holds exactly,
compared for equality with float64."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from matrix_aware_optimizer_muon_amd import build as BLD
from tests.parity_common import say
from tests.test_gpu_mx4_moment import _repeated, decoded, handle, held, padding

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


# Widths whose padded size is an odd number of 128s end inside a tile of 256.
# Scales of 1: products are multiples of 1/4 up to 36, exact for 2^24 / 4 / 36 = 116508 samples.
@pytest.mark.parametrize("n,d", [(9003, 4700), (5003, 6200), (20011, 5700), (6101, 5733), (4100, 6781), (3000, 7960),
                                 (2101, 6126), (3103, 5733), (3109, 4423), (513, 2851)])
@pytest.mark.parametrize("debug", [False, True])
def test_whole_tiles_are_exact(n, d, debug):
    say(f"case: sums of {n} samples, {d} features, debug library {debug}")
    opt = handle(d, library=BLD.DEBUG_LIB if debug else None)
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


def test_widest_and_past_4_gib_exactly():
    """Numbers 0, 1/2 and 1 with scales of 1: products are multiples of 1/4 up to 1, exact for 2^22 samples.  Every
    64th feature is the same."""
    n, d = 540000, 16384
    say(f"case: {n} samples, {d} features")
    gen = torch.Generator(device="cuda").manual_seed(11)
    blocks = -(-n // 32)
    code = torch.tensor([0, 1, 2, 8, 9, 10], dtype=torch.uint8, device="cuda")
    half = [code[torch.randint(0, 6, (64, 16 * blocks), generator=gen, device="cuda")] for _ in range(2)]
    few = mm.Mx4(half[0] + 16 * half[1], torch.full((64, blocks), 127, dtype=torch.uint8, device="cuda"), n, 64, axis=0)
    x = decoded(few)
    exact = x @ x.t().contiguous()
    opt = handle(d)
    opt.precond_accumulate(0, 0, _repeated(few, d))
    sums = opt.precond_sums(0, 0)[0]
    for at in range(0, d, 4096):
        got = sums[at:at + 4096].double().view(64, 64, d // 64, 64)
        assert torch.equal(got, exact[None, :, None, :].expand_as(got))
    opt.close()


@pytest.mark.parametrize("n,d", [(100, 64), (1000, 130), (9000, 300)])
def test_a_static_handle_gives_the_same(n, d):
    """Sums on the static scratch are no tensor: what the refresh makes of them is compared, through a step that leaves
    S^-1 in the momentum."""
    say(f"case: {n} samples, {d} features on the static scratch")
    q, later = held(n, d), held(max(1, n // 3), d, 1, wide=2)
    got = []
    for static in (False, True):
        w, g, m = torch.zeros(d, d, device="cuda"), torch.eye(d, device="cuda"), torch.zeros(d, d, device="cuda")
        opt = mm.MuonStep([mm.tensor_desc(w, g, m, precond=0)], mm.default_hparams(ns_steps=0),
                          preconds=[mm.MuonPrecond(d, 1, 0)], static_scratch=static)
        opt.precond_accumulate(0, 0, q)
        opt.precond_accumulate(0, 0, later, beta=0.5)
        opt.precond_refresh_accumulated(0, 0, damping=1.0)
        opt.step()
        torch.cuda.synchronize()
        assert opt.flags() == 0
        got.append(m.clone())
        opt.precond_refresh(0, 0, q, damping=1.0)
        opt.step()
        torch.cuda.synchronize()
        got.append(m.clone())
        opt.close()
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])
    x, y = decoded(q), decoded(later)
    s = (0.5 * x @ x.t().contiguous() + y @ y.t().contiguous()) / (0.5 * n + later.rows)
    s += torch.eye(d, device="cuda", dtype=torch.float64)
    want = torch.linalg.inv(s) * float(1 - np.float32(0.95))
    # rounding S (the sums exact, a product and a sum) and S^-1 in float32: 2^-24 each, the first times the condition
    cond = float(torch.linalg.matrix_norm(s, 2))
    assert float((got[0].double() - want).norm() / want.norm()) <= 2.0 ** -24 * (3 * cond + 4)
