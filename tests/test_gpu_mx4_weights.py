"""GPU tests of the 4-bit copies that a step renews: after every step they are
the rounding to nearest of the weights it has written, whatever steps them."""

import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from matrix_aware_optimizer_muon_amd import build as BLD
from oracle import mx4 as orc
from tests.parity_common import say
from tests.test_gpu_mx4 import check_form

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


class Model:
    """Weights of every kind that a handle steps: Muon in bf16 and float32, tall and wide, split in rows, with gaps
    between rows, filters, enough matrices for two lanes; AdamW with float32 and packed moments."""

    def __init__(self, seed=0, many=9):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.params, self.descs, self.keep = [], [], []

        def tensors(shape, dtype, gap=0):
            out = []
            for std in (0.02, 0.1):
                wide = torch.randn(*shape[:-1], shape[-1] + gap, generator=gen, device="cuda").mul_(std).to(dtype)
                out.append(wide[..., :shape[-1]] if gap else wide)
            return out

        def muon(shape, dtype=torch.bfloat16, gap=0, **kw):
            w, g = tensors(shape, dtype, gap)
            m = torch.zeros(shape, device="cuda")
            self.descs.append(mm.tensor_desc(w, g, m, **kw))
            self.keep += [g, m]
            self.params.append(w)

        def adam(shape, dtype, is_packed):
            w, g = tensors(shape, dtype)
            moments = [mm.packed_moment(w) if is_packed else torch.zeros(shape, device="cuda") for _ in range(2)]
            self.descs.append(mm.adam_tensor_desc(w, g, *moments))
            self.keep += [g] + moments
            self.params.append(w)
        for k in range(many):
            muon((256, 300 + k))
        muon((520, 130)), muon((96, 200), torch.float32), muon((384, 128), split_rows=128), muon((70, 33), gap=7)
        muon((64, 32, 3, 3))
        adam((1000, 65), torch.bfloat16, True), adam((333,), torch.float32, False), adam((257, 128), torch.float32, True)
        adam((128, 301), torch.bfloat16, False)
        self.grads = [k for k in self.keep if k.dtype != torch.uint8]

    def handle(self, **kw):
        return mm.MuonStep(self.descs, mm.default_hparams(), keepalive=self.keep, **kw)


def check(copies):
    for w, forms in zip(copies.tensors, copies.copies):
        for f in forms:
            check_form(f, mm.binding._mx4_values(w)[0])


@pytest.mark.parametrize("debug", [False, True])
def test_every_step_renews_them(debug):
    say(f"case: 4-bit copies beside a step, debug library {debug}")
    model = Model()
    opt = model.handle(library=BLD.DEBUG_LIB if debug else None)
    assert any(g["lane"] > 0 for g in opt.plan()["groups"])
    both, rows = mm.Mx4Copies(model.params), mm.Mx4Copies(model.params[::2], axis=1)
    both.quantize()
    check(both)
    opt.set_mx4_weights(both)
    for _ in range(2):
        opt.step()
        check(both)
    opt.set_mx4_weights(rows)
    opt.step(lr=0.3)
    check(rows)
    stale = [f.codes.clone() for c in both.copies for f in c]
    opt.set_mx4_weights(None)
    last = [f.codes.clone() for c in rows.copies for f in c]
    opt.step(lr=0.3)
    torch.cuda.synchronize()
    assert all(torch.equal(a, f.codes) for a, f in zip(stale, (f for c in both.copies for f in c)))
    assert all(torch.equal(a, f.codes) for a, f in zip(last, (f for c in rows.copies for f in c)))
    assert opt.flags() == 0
    opt.close()


def test_the_step_itself_is_the_same():
    plain, with_copies = Model(3), Model(3)
    a, b = plain.handle(), with_copies.handle()
    copies = mm.Mx4Copies(with_copies.params)
    b.set_mx4_weights(copies)
    b.set_max_grad_norm(1.0), a.set_max_grad_norm(1.0)
    for _ in range(3):
        a.step(), b.step()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(plain.params + plain.keep, with_copies.params + with_copies.keep))
    check(copies)
    a.close(), b.close()


def test_phases():
    model = Model(1, 2)
    opt = model.handle()
    copies = mm.Mx4Copies(model.params)
    names = [n for n, _ in opt.step_timed()]
    opt.set_mx4_weights(copies)
    timed = opt.step_timed()
    assert [n for n, _ in timed] == names + ["mx4_weights"] and timed[-1][1] > 0
    check(copies)
    opt.set_max_grad_norm(1.0)
    assert [n for n, _ in opt.step_timed()] == ["grad_norm"] + names + ["mx4_weights"]
    opt.set_mx4_weights(None)
    assert [n for n, _ in opt.step_timed()] == ["grad_norm"] + names
    opt.close()


@pytest.mark.parametrize("static", [False, True])
def test_captured_and_replayed(static):
    """Replays renew them too, the ones that the step was captured with."""
    model = Model(2, 3)
    opt = model.handle(static_scratch=static)
    copies, later = mm.Mx4Copies(model.params), mm.Mx4Copies(model.params, axis=0)
    opt.set_mx4_weights(copies)
    opt.step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        opt.step()
    opt.set_mx4_weights(later)
    for _ in range(3):
        for w in model.params:
            w.mul_(1.01)
        g.replay()
        torch.cuda.synchronize()
        check(copies)
        opt.step()
        check(later)
    opt.close()


def test_refusals():
    model = Model(4, 1)
    opt = model.handle()
    w = model.params[0]
    good = mm.Mx4Copies([w])
    for tensors in ([w.clone()], [w[1:]], [w[:, 1:]], [w, w.view(torch.int16).view(torch.bfloat16)[:255]]):
        with pytest.raises(mm.MuonError):
            opt.set_mx4_weights(mm.Mx4Copies(tensors))
    lib, err = opt._lib, mm.binding.STATUS_NAMES

    def status(**changes):
        d, _ = mm.binding._array([good._descs[0]], mm.MuonMx4)
        for k, v in changes.items():
            setattr(d[0], k, v)
        return err[lib.muon_set_mx4_weights(opt._h, d, 1)]
    grad = model.keep[0]
    ws = opt.workspace.data_ptr()
    assert status(row_codes=grad.data_ptr()) == status(col_scales=w.data_ptr()) == "MUON_ERR_ALIASING"
    assert status(col_codes=ws + 4096) == status(row_scales=ws) == "MUON_ERR_ALIASING"
    assert status(ld=w.stride(0) + 1) == status(rows=255) == status(dtype=0) == "MUON_ERR_BAD_ARG"
    assert status(row_codes=None) == "MUON_ERR_NULL_ARG"
    assert err[lib.muon_set_mx4_weights(None, good._descs, 1)] == "MUON_ERR_NULL_ARG"
    opt.set_mx4_weights(good)
    assert status(cols=7) != "MUON_OK"          # a refused list leaves the one that was set
    opt.step()
    check(good)
    opt.close()
