"""Every variant of the packed AdamW kernel: both types, rows with and without
gaps, the language's root and division (an eps below 2^-39 / sqrt(1 - beta2))
and the hardware's, and the three ways in which the count is advanced; above
and below the number of chunks up to which the launch advances it itself."""

import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from tests.parity_common import say
from tests.test_gpu_packed_adamw import Packed

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [1e-8, 1e-15])
@pytest.mark.parametrize("way", ["own", "count", "norm"])
def test_small_tensors(dtype, eps, way):
    say(f"case: packed AdamW, {dtype}, eps {eps}, rows with and without gaps, count advanced by: {way}")
    hp = mm.default_hparams(adam_eps=eps)
    ts = [Packed((600, 0), (40, 130), dtype), Packed((600, 1), (40, 130), dtype, ld=137),
          Packed((600, 2), (3, 2500), dtype, ld=2512, offset=1), Packed((600, 3), (4097,), dtype, offset=3),
          Packed((600, 4), (700, 3), dtype, ld=5)]
    descs, keep = [t.desc() for t in ts], []
    if way == "count":
        keep = [torch.zeros(4, device="cuda") for _ in range(4)]
        descs.append(mm.adam_tensor_desc(*keep))
    st = mm.MuonStep(descs, hp, keepalive=keep)
    if way == "norm":
        st.set_max_grad_norm(0.05)
    for t in (1, 2, 3):
        for x in ts:
            x.grad(t)
        st.step()
        factor = st.grad_norm[1].item() if way == "norm" else 1.0
        assert way != "norm" or factor < 1
        for k, x in enumerate(ts):
            x.check(t, k, hp, factor=factor, label=f"step {t}")
    assert st.flags() == 0 and st.adam_step() == 3
    st.close()


@pytest.mark.parametrize("shape,dtype,ld,eps", [((2100, 2051), "bf16", 2056, 1e-15), ((2100, 2051), "bf16", 2051, 1e-15),
                                                ((2100, 2051), "f32", 2053, 1e-15), ((2100, 2051), "f32", None, 1e-8),
                                                ((8193, 513), "bf16", 767, 1e-8), ((2048, 2048), "bf16", 2049, 1e-8),
                                                ((2049, 2048), "bf16", None, 1e-8)])
def test_large_tensors(shape, dtype, ld, eps):
    say(f"case: packed AdamW, {shape} {dtype}, leading dimension {ld}, eps {eps}")
    hp = mm.default_hparams(adam_eps=eps)
    x = Packed((610,), shape, dtype, ld=ld)
    st = mm.MuonStep([x.desc()], hp)
    own = mm.plan_describe([x.desc()], hp)["launch_order"] == ["adamw_packed"]
    assert own == (x.n <= 2048 * 2048)
    for t in (1, 2):
        x.grad(t)
        st.step()
        x.check(t, 0, hp, label=f"step {t}")
    st.close()
