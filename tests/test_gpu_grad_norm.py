"""Clipping by the global gradient norm inside the step.

The norm is a float64 sum of float64 squares of the stored gradients, rounded
once to float32 (2^-24); the sums' own roundings, 2^-53 each, stay below one
more 2^-24 for any number of elements here.  The factor is one float64
quotient, rounded once.  A clipped step multiplies each gradient by the
factor in float32: with float32 gradients it must equal, bit for bit, a step
without clipping on gradients that were multiplied beforehand.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from oracle import packed_moments as pm
from tests.parity_common import say
from tests.test_gpu_packed_adamw import Packed

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


class Mixed:
    """Muon matrices, AdamW tensors with float32 and with packed moments; the
    gradients float32 or bf16, some strided or misaligned."""

    def __init__(self, dtype, seed=0):
        tt = torch.float32 if dtype == "f32" else torch.bfloat16
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.sets = []
        for shape in ((256, 384), (130, 70), (70, 130)):
            self.sets.append(("muon", (rnd(*shape) * 0.02).to(tt), (rnd(*shape) * 1e-2).to(tt),
                              torch.zeros(shape, device="cuda")))
        wide_w, wide_g = (rnd(33, 64) * 0.02).to(tt), (rnd(33, 64) * 1e-2).to(tt)
        odd_w, odd_g = (rnd(9001) * 0.02).to(tt), (rnd(9001) * 1e-2).to(tt)
        for w, g in ((wide_w[:, :41], wide_g[:, :41]), (odd_w[1:], odd_g[1:]), ((rnd(1) * 0.1).to(tt), rnd(1).to(tt)),
                     (wide_w.clone()[:, :48], wide_g.clone()[:, :48])):
            self.sets.append(("packed", w, g, mm.packed_moment(w), mm.packed_moment(w)))
        w, g = (rnd(300, 64) * 0.02).to(tt), (rnd(300, 64) * 1e-2).to(tt)
        self.sets.append(("adam", w, g, torch.zeros(300, 64, device="cuda"), torch.zeros(300, 64, device="cuda")))

    def descs(self):
        return [mm.tensor_desc(*s[1:]) if s[0] == "muon" else mm.adam_tensor_desc(*s[1:]) for s in self.sets]

    def grads(self):
        return [s[2] for s in self.sets]

    def state(self):
        return [x.clone() for s in self.sets for x in (s[1], *s[3:])]


def _ref(grads, max_norm):
    return pm.clip([g.double().cpu().numpy() for g in grads], max_norm)


def _close(got, norm, factor):
    g = got.cpu().numpy().astype(np.float64)
    assert abs(g[0] - norm) <= 2 * 2.0 ** -24 * norm
    assert abs(g[1] - factor) <= 2 * 2.0 ** -24 * factor


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("max_norm", [1e-3, 0.5, 1e6, float("inf")])
def test_norm_and_factor(dtype, max_norm):
    say(f"case: gradient norm over a mixed handle, {dtype}, max_norm {max_norm}")
    x = Mixed(dtype)
    st = mm.MuonStep(x.descs())
    before = [g.clone() for g in x.grads()]
    st.set_max_grad_norm(max_norm)
    for _ in range(2):
        st.step()
        _close(st.grad_norm, *_ref(x.grads(), max_norm))
    assert all(torch.equal(a, b) for a, b in zip(before, x.grads()))     # read only
    assert st.flags() == 0
    st.close()


def test_clipped_step_is_the_step_on_scaled_gradients():
    say("case: clipped step against one on gradients scaled beforehand, bitwise, 3 steps")
    a, b = Mixed("f32"), Mixed("f32")
    sa, sb = mm.MuonStep(a.descs()), mm.MuonStep(b.descs())
    sa.set_max_grad_norm(0.25)
    for t in range(3):
        for k, (p, q) in enumerate(zip(a.grads(), b.grads())):
            p.copy_(torch.randn(p.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(97 * t + k)))
            p.mul_(1e-2)
        sa.step()
        for p, q in zip(a.grads(), b.grads()):
            q.copy_(p * sa.grad_norm[1])
        sb.step()
        assert sa.grad_norm[1].item() < 1
        for k, (p, q) in enumerate(zip(a.state(), b.state())):
            assert torch.equal(p, q), (t, k)
    sa.close()
    sb.close()


def test_off_is_the_plain_step_and_switching():
    say("case: clipping off, on without effect, off again: bitwise the plain step")
    a, b = Mixed("bf16"), Mixed("bf16")
    sa, sb = mm.MuonStep(a.descs()), mm.MuonStep(b.descs())
    assert sa.grad_norm is None
    for max_norm in (0.0, 1e9, float("inf"), 0.0):
        sa.set_max_grad_norm(max_norm)
        assert (sa.grad_norm is None) == (max_norm == 0)
        sa.step()
        sb.step()
        assert all(torch.equal(p, q) for p, q in zip(a.state(), b.state())), max_norm
    sa.set_max_grad_norm(1.0)
    names = [n for n, _ in sa.step_timed()]
    assert names[0] == "grad_norm" and names[1] == "adamw"
    sa.set_max_grad_norm(0)
    assert [n for n, _ in sa.step_timed()][0] == "adamw"
    sa.close()
    sb.close()


@pytest.mark.parametrize("shape,dtype", [((1,), "f32"), ((7,), "bf16"), ((8192,), "bf16"), ((8193,), "bf16"),
                                         ((5000, 1201), "bf16"), ((20000, 1024), "f32")])
def test_one_tensor(shape, dtype):
    say(f"case: gradient norm of one tensor {shape} {dtype}")
    x = Packed((300,), shape, dtype)
    hp = mm.default_hparams()
    st = mm.MuonStep([x.desc()], hp)
    x.grad(1)
    st.set_max_grad_norm(1e-2)
    st.step()
    norm, factor = _ref([x.dG], 1e-2)
    _close(st.grad_norm, norm, factor)
    if x.n < 1 << 20:
        x.check(1, 0, hp, factor=st.grad_norm[1].item())
    st.close()


def test_sizes_that_overflow_float32_squares_and_nonfinite():
    say("case: gradients of 1e30, infinite and NaN")
    f = torch.zeros(1000, device="cuda")
    g = torch.full((1000,), 1e30, device="cuda")
    m, v = torch.zeros_like(f), torch.zeros_like(f)
    st = mm.MuonStep([mm.adam_tensor_desc(f, g, m, v)])
    st.set_max_grad_norm(1.0)
    st.step()
    _close(st.grad_norm, *_ref([g], 1.0))
    assert bool(torch.isfinite(f).all()) and st.flags() == 0
    g[3] = float("inf")
    st.step()
    assert st.grad_norm.tolist() == [float("inf"), 0.0]
    # 0 * inf is NaN in that element, the others see zero gradients
    assert bool(f[3].isnan()) and bool(torch.isfinite(f[4:]).all()) and st.flags(reset=True) & 1
    g[3] = float("nan")
    st.step()
    assert st.grad_norm.isnan().all() and bool(f.isnan().all())
    st.close()


def test_graph_replays():
    say("case: clipped mixed step captured in a graph, replays against eager")
    a, b = Mixed("bf16"), Mixed("bf16")
    sa, sb = mm.MuonStep(a.descs()), mm.MuonStep(b.descs())
    for s in (sa, sb):
        s.set_max_grad_norm(0.5)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        sb.step()
    for t in range(4):
        for k, (p, q) in enumerate(zip(a.grads(), b.grads())):
            p.copy_(torch.randn(p.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(31 * t + k)))
            p.mul_(10.0 ** (t - 2))
            q.copy_(p)
        torch.cuda.synchronize()
        sa.step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(sa.grad_norm, sb.grad_norm)
        _close(sb.grad_norm, *_ref(b.grads(), 0.5))
        assert all(torch.equal(p, q) for p, q in zip(a.state(), b.state())), t
        torch.randn(1 << 20, device="cuda").sum().item()
    sa.close()
    sb.close()


def test_refusals():
    say("case: refusals of the norm setting")
    x = Packed((310,), (300,), "f32")
    st = mm.MuonStep([x.desc()])
    lib, INF = st._lib, float("inf")
    assert lib.muon_set_max_grad_norm(st._h, -1.0, None) == 9
    assert lib.muon_set_max_grad_norm(st._h, float("nan"), None) == 9
    assert lib.muon_set_max_grad_norm(st._h, INF, x.dW.data_ptr() + 2) == 4
    assert lib.muon_set_max_grad_norm(st._h, INF, x.dW.data_ptr()) == 5
    assert lib.muon_set_max_grad_norm(st._h, INF, st.workspace.data_ptr()) == 5
    assert lib.muon_set_max_grad_norm(st._h, INF, None) == 0
    assert lib.muon_set_max_grad_norm(st._h, 0.0, None) == 0
    with pytest.raises(mm.MuonError):
        st.set_max_grad_norm(-0.5)
    st.close()
    empty = mm.MuonStep([])
    empty.set_max_grad_norm(1.0)
    empty.step()
    assert empty.grad_norm.tolist() == [0.0, 1.0]
    empty.close()


def test_norm_of_a_captured_step_outlives_the_setting():
    say("case: a captured clipped step replayed after clipping was switched off")
    a, b = Mixed("bf16"), Mixed("bf16")
    sa, sb = mm.MuonStep(a.descs()), mm.MuonStep(b.descs())
    for s in (sa, sb):
        s.set_max_grad_norm(0.5)
    place = sb.grad_norm.data_ptr()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        sb.step()
    sb.set_max_grad_norm(0.0)
    others = [torch.zeros(2, device="cuda") for _ in range(64)]
    assert place not in [x.data_ptr() for x in others]
    for _ in range(3):
        sa.step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a.state(), b.state()))
        assert not any(bool(x.any()) for x in others)
    sb.set_max_grad_norm(0.5)                    # on again: the same place, with the replays' figures
    assert sb.grad_norm.data_ptr() == place and torch.equal(sa.grad_norm, sb.grad_norm)
    sa.close()
    sb.close()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_measuring_does_not_spread_a_bad_gradient(bad):
    say(f"case: measured, not clipped, with a gradient of {bad}: bitwise the plain step")
    a, b = Mixed("f32"), Mixed("f32")
    for x in (a, b):
        x.grads()[4][3] = bad                    # one element of a packed tensor
    sa, sb = mm.MuonStep(a.descs()), mm.MuonStep(b.descs())
    sa.set_max_grad_norm(float("inf"))
    for s in (sa, sb):
        s.step()
    norm, factor = sa.grad_norm.tolist()
    assert factor == 1.0 and (norm != norm if bad != bad else norm == bad)
    for p, q in zip(a.state(), b.state()):
        assert torch.equal(p.contiguous().view(torch.uint8), q.contiguous().view(torch.uint8))
    assert sa.flags() == sb.flags() == 1
    w = a.sets[4][1]
    assert bool(w[3].isnan()) and int(w.isnan().sum()) == 1
    sa.close()
    sb.close()


def test_static_handle_allocates_at_the_first_setting():
    say("case: norm of a static handle, no torch memory before it is set")
    x = Packed((340,), (500,), "f32")
    x.grad(1)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    st = mm.MuonStep([x.desc()], static_scratch=True)
    assert torch.cuda.memory_allocated() == before and st.grad_norm is None
    st.set_max_grad_norm(0.5)
    place = st.grad_norm.data_ptr()
    st.step()
    _close(st.grad_norm, *_ref([x.dG], 0.5))
    st.set_max_grad_norm(0.0)
    st.set_max_grad_norm(float("inf"))
    assert st.grad_norm.data_ptr() == place
    st.close()


def test_static_handle_norm_set_on_a_busy_stream():
    say("case: norm of a static handle set on a stream with work in flight, the step on another one")
    x = Packed((350,), (500,), "f32")
    x.grad(1)
    torch.cuda.synchronize()
    st = mm.MuonStep([x.desc()], static_scratch=True)
    busy = torch.zeros(1 << 26, device="cuda")
    for _ in range(50):
        busy.add_(1.0)
    st.set_max_grad_norm(0.5)
    side = torch.cuda.Stream()
    st.step(stream=side)
    side.synchronize()
    norm, factor = _ref([x.dG], 0.5)
    _close(st.grad_norm, norm, factor)
    torch.cuda.synchronize()
    _close(st.grad_norm, norm, factor)
    assert bool((busy == 50).all())
    st.close()
