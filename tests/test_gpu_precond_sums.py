"""GPU tests of the running sums of a preconditioner block as a program that
writes them itself meets them (muon_precond_sums)."""

import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from tests.parity_common import say
from tests.test_gpu_mx4_moment import decoded, handle, held

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


# few samples, whole tiles, tiles cut into ranges
@pytest.mark.parametrize("n,d", [(70, 100), (1000, 200), (5003, 1025), (16384, 300)])
@pytest.mark.parametrize("form", ["mx4", "bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_beta_of_zero_forgets_sums_and_count(n, d, form, bad):
    """Both, whatever they held: what follows is finite."""
    say(f"case: {n} samples, {d} features, {form}, from {bad}")
    q = held(n, d, scales=(127, 128))
    x = decoded(q)
    acts = q if form == "mx4" else x.t().contiguous().to({"bf16": torch.bfloat16, "f32": torch.float32}[form])
    opt = handle(d)
    sums, count = opt.precond_sums(0, 0)
    sums.fill_(bad), count.fill_(bad)
    opt.precond_accumulate(0, 0, acts, beta=0.0)
    assert torch.equal(sums.double(), x @ x.t().contiguous()) and float(count) == n
    opt.precond_refresh_accumulated(0, 0, damping=1.0)
    torch.cuda.synchronize()
    assert opt.flags() == 0
    opt.close()
