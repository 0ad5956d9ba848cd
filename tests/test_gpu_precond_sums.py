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


@pytest.mark.parametrize("form", ["mx4", "bf16", "f32"])
@pytest.mark.parametrize("d", [100, 256, 1025])
def test_sums_of_ranks_added_up(form, d):
    """Two handles as the ranks of a data-parallel job: their sums, whole and contiguous as a collective takes them,
    added up, against one handle that has seen all samples."""
    say(f"case: {d} features, {form}")

    def acts(n, seed):
        q = held(n, d, seed, scales=(127, 128))
        return q if form == "mx4" else decoded(q).t().contiguous().to({"bf16": torch.bfloat16, "f32": torch.float32}[form])
    ranks, whole = [handle(d), handle(d)], handle(d)
    for k, (opt, n) in enumerate(zip(ranks, (700, 301))):
        opt.precond_accumulate(0, 0, acts(n, k))
        whole.precond_accumulate(0, 0, acts(n, k))
    views = [opt.precond_sums(0, 0, padded=True) for opt in ranks]
    ld = -(-d // 128) * 128
    for sums, count in views:
        assert sums.is_contiguous() and sums.shape == (ld, ld) and count.is_contiguous()
        assert not bool(sums[d:].any()) and not bool(sums[:, d:].any())
    total = [a + b for a, b in zip(*views)]
    for opt, view in zip(ranks, views):
        for t, v in zip(view, total):
            t.copy_(v)
        sums, count = opt.precond_sums(0, 0)
        want = whole.precond_sums(0, 0)
        assert sums.data_ptr() == view[0].data_ptr() and sums.shape == (d, d)
        assert torch.equal(sums, want[0]) and torch.equal(count, want[1])
        opt.precond_refresh_accumulated(0, 0, damping=1.0)
        torch.cuda.synchronize()
        assert opt.flags() == 0
    for opt in ranks + [whole]:
        opt.close()
