"""The bias corrections of a step do not depend on which launch advanced the
AdamW count: the packed tensors' own launch, the count's, or the gradient
norm's.  Betas next to 1 and the step counts at which a power by repeated
squaring and one by pow round to different float32 corrections (found by
comparing both over two million steps)."""

import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from tests.parity_common import say
from tests.test_gpu_packed_adamw import Packed

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

N = 6000


def _run(hp, way, start, steps):
    x = Packed((500,), (N,), "f32")
    descs, keep = [x.desc()], []
    if way == "count":                  # a tensor with float32 moments beside it: a launch for the count
        keep = [torch.zeros(4, device="cuda") for _ in range(4)]
        descs.append(mm.adam_tensor_desc(*keep))
    st = mm.MuonStep(descs, hp, keepalive=keep)
    if way == "norm":
        st.set_max_grad_norm(float("inf"))
    if start:
        st.set_adam_step(start)
    for t in range(start + 1, start + steps + 1):
        x.grad(t)
        if way == "mixed":              # the norm on and off from step to step
            st.set_max_grad_norm(float("inf") if t % 2 else 0.0)
        st.step()
    assert st.adam_step() == start + steps
    st.close()
    return x


@pytest.mark.parametrize("beta1,beta2,start", [(0.9, 0.95, 0), (0.999999, 0.95, 276), (0.999999, 0.95, 17331),
                                               (0.999999, 0.999999, 28431), (0.9, 0.999999, 5757),
                                               (0.9, 0.999999, 20366), (0.999999, 0.999999, 35191)])
def test_corrections_do_not_depend_on_the_launch(beta1, beta2, start):
    say(f"case: packed steps from {start}, betas {beta1}, {beta2}, the count advanced by each launch that can")
    hp = mm.default_hparams(adam_beta1=beta1, adam_beta2=beta2, adam_lr=0.5, adam_weight_decay=0.0)
    ref = _run(hp, "own", start, 3)
    for way in ("count", "norm", "mixed"):
        x = _run(hp, way, start, 3)
        assert torch.equal(ref.dM, x.dM) and torch.equal(ref.dV, x.dV), way
        assert torch.equal(ref.dW, x.dW), f"{way}: {int((ref.dW != x.dW).sum())} of {N} weights differ"


def test_count_set_again_and_again():
    say("case: the count set between steps, forwards, backwards and to the first step again")
    hp = mm.default_hparams()
    x = Packed((510,), (3000,), "f32")
    st = mm.MuonStep([x.desc()], hp)
    for start in (0, 7, 3, 70000, 0, 1):
        st.set_adam_step(start)
        assert st.adam_step() == start
        for t in (start + 1, start + 2):
            x.grad(t)
            st.step()
            x.check(t, 0, hp, label=f"step {t}")
    with pytest.raises(mm.MuonError):
        st.set_adam_step(-1)
    assert st.adam_step() == 3
    st.close()


def test_count_of_a_captured_step_and_eager_ones():
    say("case: captured steps that advance the count, among eager ones and with the norm on in between")
    hp = mm.default_hparams()
    a, b = Packed((520,), (40, 130), "bf16"), Packed((520,), (40, 130), "bf16")
    eager, st = mm.MuonStep([a.desc()], hp), mm.MuonStep([b.desc()], hp)
    b.grad(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        st.step()
    for t in range(1, 9):
        a.grad(t)
        b.grad(t)
        torch.cuda.synchronize()
        st.set_max_grad_norm(float("inf") if t in (3, 6) else 0.0)
        if t in (3, 4):
            st.step()
        else:
            graph.replay()
        eager.step()
        a.check(t, 0, hp)
        b.check(t, 0, hp)
        assert torch.equal(a.dW, b.dW) and torch.equal(a.dM, b.dM), t
        torch.randn(1 << 20, device="cuda").sum().item()
    eager.close()
    st.close()
