"""GPU tests of 4-bit copies of weights of one row, whose leading dimension says
nothing: slices of a wider buffer, contiguous ones, vectors."""

import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from tests.test_gpu_mx4_weights import check

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_row_of_a_wider_buffer(dtype):
    gen = torch.Generator(device="cuda").manual_seed(3)

    def wide():
        return torch.randn(5, 400, generator=gen, device="cuda").to(dtype)
    params, descs, keep = [], [], []
    for row in (slice(2, 3), slice(4, 5)):
        w, g = wide()[row, :300], wide()[row, :300]
        assert w.shape == (1, 300) and w.stride(0) == 400
        if row.start == 2:
            state = [torch.zeros(1, 300, device="cuda")]
            descs.append(mm.tensor_desc(w, g, *state))
        else:
            state = [torch.zeros(1, 300, device="cuda") for _ in range(2)]
            descs.append(mm.adam_tensor_desc(w, g, *state))
        params.append(w)
        keep += [g] + state
    v = torch.randn(77, generator=gen, device="cuda").to(dtype)
    state = [torch.randn(77, generator=gen, device="cuda").to(dtype)] + [mm.packed_moment(v) for _ in range(2)]
    descs.append(mm.adam_tensor_desc(v, *state))
    params.append(v), keep.extend(state)
    opt = mm.MuonStep(descs, mm.default_hparams(), keepalive=keep)
    copies = mm.Mx4Copies(params)
    opt.set_mx4_weights(copies)
    before = [p.clone() for p in params]
    for _ in range(2):
        opt.step()
        check(copies)
    assert not any(torch.equal(a, b) for a, b in zip(before, params))
    # another row, or fewer columns, is not the param
    for other in (params[0].clone(), params[0][:, :299], params[1][:, 1:]):
        with pytest.raises(mm.MuonError):
            opt.set_mx4_weights(mm.Mx4Copies([other]))
    opt.close()
