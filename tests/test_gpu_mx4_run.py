"""GPU tests of the operators on microscaled 4-bit floats together, as a training
run uses them: a layer's input is rounded along the samples and held, its second
moment taken from what is held, the preconditioner refreshed from the sums, the
weights stepped, their 4-bit copies renewed by the step and read back.

The activations are numbers of the format, so holding them is without loss, and
their sums are exact in float32 (products are multiples of 1/4 of at most 36,
halved twice: 2^24 / 16 / 36 = 29127 samples): a run that is given the same
activations in float32 takes the same steps, bit for bit."""

import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from oracle import mx4 as orc
from tests.parity_common import say
from tests.test_gpu_mx4 import check_form, same_values

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DS = (200, 768)                # inputs of the two kinds of layers
SAMPLES = 1111


def activations(step, d, n=SAMPLES):
    gen = torch.Generator(device="cuda").manual_seed(step * 1009 + d)
    grid = torch.tensor(orc.MAGNITUDES, device="cuda", dtype=torch.float32)
    x = grid[torch.randint(0, 8, (n, d), generator=gen, device="cuda")]
    return x * (torch.randint(0, 2, (n, d), generator=gen, device="cuda") * 2 - 1)


class Run:
    """Layers of both kinds with a slot each, an embedding under AdamW, their copies; 40 of each kind make lists that
    take several launches."""

    def __init__(self, layers=2):
        gen = torch.Generator(device="cuda").manual_seed(5)
        self.params, descs, self.keep = [], [], []
        for k in range(layers):
            for slot, d in enumerate(DS):
                w, g = (torch.randn(96 + 16 * slot, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
                m = torch.zeros(w.shape, device="cuda")
                descs.append(mm.tensor_desc(w, g, m, precond=slot))
                self.params.append(w)
                self.keep += [g, m]
        w, g = (torch.randn(515, 72, generator=gen, device="cuda") for _ in range(2))
        moments = [mm.packed_moment(w) for _ in range(2)]
        descs.append(mm.adam_tensor_desc(w, g, *moments))
        self.params.append(w)
        self.keep += [g] + moments
        self.opt = mm.MuonStep(descs, mm.default_hparams(), preconds=[mm.MuonPrecond(d, 1, 0) for d in DS],
                               keepalive=self.keep)
        self.opt.set_rounding_seed(3)
        self.copies = mm.Mx4Copies(self.params)
        self.opt.set_mx4_weights(self.copies)
        self.values = torch.empty(self.copies.elements, device="cuda")
        self.held = [mm.mx4_empty(SAMPLES, d, axis=0) for d in DS]

    def step(self, acts, in_4_bits=True):
        """`acts`: two micro-batches of each kind."""
        for k, batch in enumerate(acts):
            for slot, x in enumerate(batch):
                if in_4_bits:
                    x = mm.mx4_quantize(x, out=self.held[slot])
                self.opt.precond_accumulate(slot, 0, x, beta=0.5 if k == 0 else 1.0)
        for slot in range(len(DS)):
            self.opt.precond_refresh_accumulated(slot, 0, damping=0.5, reset=False)
        self.opt.step()
        self.copies.dequantize(axis=0, out=self.values)

    def state(self):
        sums = [t.clone() for slot in range(len(DS)) for t in self.opt.precond_sums(slot, 0)]
        return [t.clone() for t in self.params + self.keep] + sums


def batches(step):
    return [[activations(2 * step + k, d) for d in DS] for k in range(2)]


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_held_activations_step_as_the_others():
    held, plain = Run(), Run()
    for step in range(3):
        acts = batches(step)
        held.step(acts), plain.step(acts, in_4_bits=False)
        torch.cuda.synchronize()
        assert same(held.state(), plain.state()), step
        # every step halves the sums before it
        want = sum(0.5 ** (step - k) * x.double().t().contiguous() @ x.double() for k in range(step + 1)
                   for x, _ in batches(k))
        sums, count = held.opt.precond_sums(0, 0)
        assert torch.equal(sums.double(), want)
        assert float(count) == sum(0.5 ** (step - k) * 2 * SAMPLES for k in range(step + 1))
        for w, forms, v in zip(held.copies.tensors, held.copies.copies, held.copies.split(held.values)):
            dec = [check_form(f, w) for f in forms]
            same_values(v, dec[1])
    assert held.opt.flags() == 0
    held.opt.close(), plain.opt.close()


@pytest.mark.parametrize("layers", [1, 40])
def test_captured_and_replayed(layers):
    """The whole of it in one graph, replayed with other work between; lists of one launch and of several, whose
    descriptions are the launches' arguments."""
    say(f"case: {2 * layers + 1} weights")
    graphed, eager = Run(layers), Run(layers)
    acts = batches(0)
    graphed.step(acts), eager.step(acts)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graphed.step(acts)
    for step in range(1, 4):
        for old, new in zip(acts, batches(step)):
            for x, y in zip(old, new):
                x.copy_(y)
        g.replay()
        eager.step(acts)
        torch.cuda.synchronize()
        assert same(graphed.state(), eager.state()), step
        assert torch.equal(graphed.values, eager.values), step
        for a, b in zip(graphed.copies.copies, eager.copies.copies):
            for x, y in zip(a, b):
                assert torch.equal(x.codes, y.codes)
        _ = torch.ones(1 << 20, device="cuda").sum().item()
    assert graphed.opt.flags() == 0
    graphed.opt.close(), eager.opt.close()


def test_two_handles_on_two_streams_at_once():
    """Each with its own workspace; neither's sums, weights or copies show the other."""
    runs, alone = [Run(), Run()], [Run(), Run()]
    acts = [batches(10), batches(20)]
    for r, a in zip(alone, acts):
        r.step(a), r.step(a)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(2):
        for r, a, s in zip(runs, acts, streams):
            with torch.cuda.stream(s):
                r.step(a)
    torch.cuda.synchronize()
    for r, want in zip(runs, alone):
        assert same(r.state(), want.state()) and torch.equal(r.values, want.values)
        assert r.opt.flags() == 0
    for r in runs + alone:
        r.opt.close()


def test_the_same_held_activations_twice():
    """A layer's input that is counted twice."""
    run = Run()
    q = mm.mx4_quantize(activations(0, DS[0]), axis=0)
    x = mm.mx4_dequantize(q).double()
    want = x.t().contiguous() @ x
    for _ in range(2):
        run.opt.precond_accumulate(0, 0, q)
    sums, count = run.opt.precond_sums(0, 0)
    assert torch.equal(sums.double(), 2 * want) and float(count) == 2 * SAMPLES
    run.opt.close()


def test_copies_share_tensors():
    """One tensor twice in a list: each of its copies is written."""
    w = torch.randn(300, 200, device="cuda")
    copies = mm.Mx4Copies([w, w])
    copies.quantize("random", seed=4)
    for k, forms in enumerate(copies.copies):
        for f in forms:
            check_form(f, w, orc.words(4, k, *w.shape))
