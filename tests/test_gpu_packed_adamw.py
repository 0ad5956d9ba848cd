"""AdamW with packed (8-bit) moments on the GPU against the oracle.

Bytes and scales are compared for equality: the moments are float32 with
every operation rounded by itself, and the random words are given.

Weights are compared with the float64 formula on the same moments m', v'
(their float32 values).  Of the update term the kernel rounds: the square
root, its product with 1/sqrt(1-b2^t) and that number, the sum with eps, the
product with 1/(1-b1^t) and that number, the quotient, and the two products
that make lr * term, each by at most one unit in the last place (2^-23): 10
units.  The weight takes the product lr*wd*w (2 roundings of a term below
|w| / 8) and two subtractions: 2.5 half units (2^-24) of |w| + |term|.
A bf16 weight is then rounded by half a step, 2^-8 of itself; a float32 one
by nothing more.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from oracle import muon_oracle as orc
from oracle import packed_moments as pm
from tests.parity_common import from_device, say, to_device

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

CANARY = 0xA5


def _rng(*key):
    return np.random.Generator(np.random.PCG64(np.random.SeedSequence([9300, *key])))


def _store(x, dtype):
    return orc.f64_to_bf16_bits(x) if dtype == "bf16" else np.asarray(x, np.float32)


def _decode(a, dtype):
    return orc.bf16_bits_to_f64(a) if dtype == "bf16" else np.asarray(a, np.float64)


def _betas(hp):
    return float(np.float32(hp.adam_beta1)), float(np.float32(hp.adam_beta2))


def _same_bytes(got, ref, n, first):
    """Equal but for the sign of a first moment's NaN, which IEEE 754 leaves open."""
    got, ref = got.copy(), ref.copy()
    if first:
        for b in (got, ref):
            codes = b[:-(-n // pm.BLOCK) * pm.BLOCK]
            codes[codes == 0xFF] = 0x7F
    return np.array_equal(got, ref)


class Packed:
    """One tensor: its buffers on the GPU, inside larger ones whose other
    bytes must stay as they are, and its state on the oracle's side.  `ld`:
    leading dimension of param and grad, `offset`: elements by which param and
    grad start behind a 16-byte boundary."""

    def __init__(self, key, shape, dtype, ld=None, offset=0, lr_mult=1.0):
        self.key, self.shape, self.dtype, self.lr_mult = key, shape, dtype, lr_mult
        self.n = int(np.prod(shape))
        rows, cols = (1, self.n) if len(shape) == 1 else (shape[0], self.n // shape[0])
        ld = ld or cols
        tt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.bufs = [torch.zeros(offset + rows * ld + 64, dtype=tt, device="cuda") for _ in range(2)]
        self.dW, self.dG = (b[offset:offset + rows * ld].view(rows, ld)[:, :cols] for b in self.bufs)
        if ld == cols:
            self.dW, self.dG = self.dW.reshape(shape), self.dG.reshape(shape)
        nb = pm.moment_bytes(self.n)
        self.state = [torch.full((nb + 96,), CANARY, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.dM, self.dV = (s[32:32 + nb] for s in self.state)
        self.dM.zero_()
        self.dV.zero_()
        self.w = _store(_rng(*key, 1).normal(0, 0.02, (rows, cols)), dtype)
        self.dW.copy_(to_device(torch, self.w, dtype).view(self.dW.shape))
        self.mem = (np.zeros(nb, np.uint8), np.zeros(nb, np.uint8))

    def desc(self):
        return mm.adam_tensor_desc(self.dW, self.dG, self.dM, self.dV, lr_mult=self.lr_mult)

    def grad(self, step, scale=None):
        rng = _rng(*self.key, 2, step)
        g = rng.normal(0, 1e-2, self.w.shape) * 10.0 ** rng.uniform(-3, 1, self.w.shape)
        if scale is not None:
            g = g * scale
        g[rng.random(self.w.shape) < 0.1] = 0.0
        self.set_grad(g)

    def set_grad(self, g):
        self.g = _store(g, self.dtype)
        self.dG.copy_(to_device(torch, self.g, self.dtype).view(self.dG.shape))
        self.ring = [b.clone() for b in self.bufs]

    def check(self, t, tensor, hp, seed=0, factor=1.0, label=""):
        """Advance the oracle by step t and compare everything with the GPU's state."""
        label = f"{label} {self.shape} {self.dtype}"
        betas = _betas(hp)
        m0, v0 = pm.decode(*self.mem, self.n)
        m1, v1 = pm.moments_f32(_decode(self.g, self.dtype).reshape(-1), m0, v0, betas, factor)
        self.mem = pm.encode(m1, v1, pm.words(seed, t, tensor, self.n))
        for name, dev, ref in (("first", self.dM, self.mem[0]), ("second", self.dV, self.mem[1])):
            got = dev.cpu().numpy()
            assert _same_bytes(got, ref, self.n, name == "first"), f"{label}: {name} moment, {(got != ref).sum()} of {ref.size} bytes differ"
        for s, d in zip(self.state, (self.dM, self.dV)):
            assert bool((s[:32] == CANARY).all()) and bool((s[32 + d.numel():] == CANARY).all()), label
        lr = float(np.float32(hp.adam_lr) * np.float32(self.lr_mult))
        wd, eps = float(np.float32(hp.adam_weight_decay)), float(np.float32(hp.adam_eps))
        w0 = _decode(self.w, self.dtype).reshape(-1)
        ref, term = pm.update(w0, m1, v1, t, lr, betas, eps, wd)
        got = from_device(torch, self.dW.contiguous(), self.dtype).reshape(-1)
        self.w = got.reshape(self.w.shape)
        got = _decode(got, self.dtype)
        fine = np.isfinite(ref)
        assert np.array_equal(np.isnan(got), np.isnan(ref)), label
        tol = 10 * 2.0 ** -23 * term + 2.5 * 2.0 ** -24 * (np.abs(w0) + term)
        if self.dtype == "bf16":
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        err = np.abs(got - ref)[fine]
        assert (err <= tol[fine]).all(), f"{label}: weight off by {(err / tol[fine]).max():.2f} of its bound"
        # what lies between and behind the rows is untouched, the gradient too
        self.ring[0].as_strided(self.dW.shape, self.dW.stride(), self.dW.storage_offset()).copy_(self.dW)
        for p, q in zip(self.ring, self.bufs):     # as bytes: a NaN equals itself
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8)), label


SHAPES = [(1,), (2,), (255,), (256,), (257,), (4095,), (4096,), (4097,), (300, 64), (4, 5, 6), (1001, 1), (1, 1001),
          (130, 513)]
STRIDED = [((37, 50), 56), ((37, 48), 64), ((64, 1), 3), ((5, 300), 301), ((3, 4096), 4112)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_match_bytes_and_weights(dtype):
    say(f"case: packed AdamW, {dtype}, many shapes in one handle, 4 steps from zero")
    hp = mm.default_hparams()
    ts = [Packed((k, dtype == "f32"), s, dtype, lr_mult=1.0 + 0.25 * (k % 3)) for k, s in enumerate(SHAPES)]
    ts += [Packed((50 + k, dtype == "f32"), s, dtype, ld=ld) for k, (s, ld) in enumerate(STRIDED)]
    ts += [Packed((70 + k, dtype == "f32"), s, dtype, offset=o) for k, (s, o) in
           enumerate([((1000,), 1), ((40, 80), 3), ((257,), 4)])]
    st = mm.MuonStep([t.desc() for t in ts], hp)
    for t in (1, 2, 3, 4):
        for x in ts:
            x.grad(t)
        st.step()
        for k, x in enumerate(ts):
            x.check(t, k, hp, label=f"step {t}")
    assert st.flags() == 0 and st.adam_step() == 4
    st.close()


@pytest.mark.parametrize("beta1,beta2,eps,wd", [(0.0, 0.0, 1e-8, 0.0), (0.95, 0.999, 1e-15, 0.1), (0.3, 0.2, 0.1, 0.01)])
def test_hyperparameters_seed_and_late_steps(beta1, beta2, eps, wd):
    say(f"case: packed AdamW, betas ({beta1}, {beta2}), a 64-bit seed, from step 70000")
    hp = mm.default_hparams(adam_beta1=beta1, adam_beta2=beta2, adam_eps=eps, adam_weight_decay=wd, adam_lr=2e-3)
    ts = [Packed((100, k), (40, 130), d) for k, d in enumerate(("bf16", "f32"))]
    st = mm.MuonStep([t.desc() for t in ts], hp)
    seed = 0x123456789ABCDEF0
    st.set_rounding_seed(seed)
    st.set_adam_step(70000)
    for t in (70001, 70002, 70003):
        for x in ts:
            x.grad(t)
        st.step()
        for k, x in enumerate(ts):
            x.check(t, k, hp, seed=seed, label=f"step {t}")
    st.close()


@pytest.mark.parametrize("scale", [1e-33, 1e-20, 1e-12, 1e12, 1e17])
def test_gradients_of_any_size(scale):
    say(f"case: packed AdamW, gradients times {scale}")
    hp = mm.default_hparams(adam_eps=1e-8)
    ts = [Packed((110, k), (3000,), d) for k, d in enumerate(("bf16", "f32"))]
    st = mm.MuonStep([t.desc() for t in ts], hp)
    for t in (1, 2):
        for x in ts:
            x.grad(t, scale)
        st.step()
        for k, x in enumerate(ts):
            x.check(t, k, hp, label=f"step {t}")
    assert st.flags() == 0
    st.close()


def test_zero_gradients_and_single_elements():
    say("case: packed AdamW, zero gradients, blocks with one element that is not zero, vanished gradients")
    hp = mm.default_hparams()
    x = Packed((120,), (2048,), "f32")
    st = mm.MuonStep([x.desc()], hp)
    x.set_grad(np.zeros((1, 2048)))
    st.step()
    x.check(1, 0, hp)
    assert not x.dM.bool()[:2048].any() and not x.dV.bool()[:2048].any()
    g = np.zeros((1, 2048))
    g[0, 5], g[0, 255], g[0, 256], g[0, 2047] = 1e-3, -2.0, 1e-30, 7e4
    x.set_grad(g)
    st.step()
    x.check(2, 0, hp)
    x.set_grad(np.zeros((1, 2048)))
    for t in range(3, 9):
        st.step()
        x.check(t, 0, hp)
    st.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("at", [5, 300, 999])      # either half of a wave, the last element
def test_nonfinite_gradient_stays_in_its_element(dtype, bad, at):
    say(f"case: packed AdamW, gradient element {at} {bad}")
    hp = mm.default_hparams()
    x = Packed((130,), (1000,), dtype)
    st = mm.MuonStep([x.desc()], hp)
    x.grad(1)
    st.step()
    x.check(1, 0, hp)
    assert st.flags() == 0
    x.grad(2)
    g = _decode(x.g, dtype)
    g[0, at] = bad
    x.set_grad(g)
    st.step()
    # the oracle's weight of the element is NaN as well: m' / sqrt(v') of inf / inf or NaN
    x.check(2, 0, hp)
    assert st.flags(reset=True) & 1
    m, _ = pm.decode(*x.mem, 1000)
    assert np.isnan(m[at]) and np.isfinite(np.delete(m, at)).all()
    st.close()


def test_second_moment_overflow():
    say("case: packed AdamW, a gradient whose square overflows float32")
    hp = mm.default_hparams()
    x = Packed((140,), (512,), "f32")
    st = mm.MuonStep([x.desc()], hp)
    x.grad(1)
    g = np.asarray(x.g, np.float64)
    g[0, 100] = 1e25
    x.set_grad(g)
    st.step()
    x.check(1, 0, hp)
    _, v = pm.decode(*x.mem, 512)
    assert v[100] == 1.875 * 2.0 ** 127
    st.close()


def test_beside_the_other_kinds():
    say("case: packed tensors beside Muon matrices and float32-moment AdamW tensors, bitwise as without them")
    hp = mm.default_hparams()

    def others():
        w = to_device(torch, orc.f64_to_bf16_bits(_rng(150, 1).normal(0, 0.02, (256, 384))), "bf16")
        g = to_device(torch, orc.f64_to_bf16_bits(_rng(150, 2).normal(0, 0.02, (256, 384))), "bf16")
        aw, ag = (torch.from_numpy(_rng(150, k).normal(0, 1, 700).astype(np.float32)).cuda() for k in (3, 4))
        return [w, g, torch.zeros(256, 384, device="cuda"), aw, ag, torch.zeros(700, device="cuda"),
                torch.zeros(700, device="cuda")]

    def descs(o):
        return mm.tensor_desc(*o[:3]), mm.adam_tensor_desc(*o[3:])
    a, b = others(), others()
    x, y = Packed((151,), (90, 70), "bf16"), Packed((152,), (333,), "f32")
    mu, ad = descs(a)
    both = mm.MuonStep([mu, x.desc(), ad, y.desc()], hp)
    alone = mm.MuonStep(list(descs(b)), hp)
    assert both.packed_elements() == 90 * 70 + 333
    for t in (1, 2, 3):
        x.grad(t)
        y.grad(t)
        both.step()
        alone.step()
        x.check(t, 1, hp)
        y.check(t, 3, hp)
        for p, q in zip(a, b):
            assert torch.equal(p, q)
    names = [n for n, _ in both.step_timed()]
    assert names[0] == "adamw" and sum(n.startswith("bx") for n in names) == 5
    both.close()
    alone.close()


def test_graph_replays_match_eager_and_streams():
    say("case: packed AdamW captured in a graph, replayed with new gradients and eager work between")
    hp = mm.default_hparams()
    a, b = Packed((160,), (77, 100), "bf16"), Packed((160,), (77, 100), "bf16")
    eager = mm.MuonStep([a.desc()], hp)
    st = mm.MuonStep([b.desc()], hp)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.grad(0)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            st.step()
            values = st.unpack_moments()
    torch.cuda.current_stream().wait_stream(side)
    for t in range(1, 6):
        a.grad(t)
        b.grad(t)
        torch.cuda.synchronize()
        if t == 3:          # one ordinary step of the captured handle among the replays
            st.step()
        else:
            graph.replay()
        eager.step()
        a.check(t, 0, hp)
        b.check(t, 0, hp)
        if t != 3:
            m, v = pm.decode(*b.mem, b.n)
            assert np.array_equal(values.cpu().numpy().astype(np.float64), np.stack([m, v]))
        torch.randn(1 << 20, device="cuda").sum().item()
    eager.close()
    st.close()


def test_two_handles_on_two_streams():
    say("case: two packed handles stepping on two streams at once")
    hp = mm.default_hparams()
    xs = [Packed((170, k), (1500, 100), "bf16") for k in range(2)]
    sts = [mm.MuonStep([x.desc()], hp) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for t in (1, 2, 3):
        for x in xs:
            x.grad(t)
        torch.cuda.synchronize()
        for s, st in zip(streams, sts):
            st.step(stream=s)
        torch.cuda.synchronize()
        for x in xs:
            x.check(t, 0, hp)
    for st in sts:
        st.close()


def test_resumed_run_repeats_the_bytes():
    say("case: packed AdamW resumed from its buffers and step count")
    hp = mm.default_hparams()
    a, b = Packed((180,), (5000,), "f32"), Packed((180,), (5000,), "f32")
    st = mm.MuonStep([a.desc()], hp)
    st.set_rounding_seed(9)
    for t in (1, 2):
        a.grad(t)
        st.step()
    for dst, src in ((b.dW, a.dW), (b.dM, a.dM), (b.dV, a.dV)):
        dst.copy_(src)
    st2 = mm.MuonStep([b.desc()], hp)
    st2.set_rounding_seed(9)
    st2.set_adam_step(2)
    for x, s in ((a, st), (b, st2)):
        x.grad(3)
        s.step()
    assert torch.equal(a.dW, b.dW) and torch.equal(a.dM, b.dM) and torch.equal(a.dV, b.dV)
    st.close()
    st2.close()


SIZES = [(1,), (255,), (4097,), (3, 1000), (64, 256), (31,)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pack_and_unpack(dtype):
    say(f"case: pack and unpack, {dtype} values")
    tt = torch.float32 if dtype == "f32" else torch.bfloat16
    xs = [Packed((200, k), s, "bf16") for k, s in enumerate(SIZES)]
    st = mm.MuonStep([x.desc() for x in xs])
    n = st.packed_elements()
    assert n == sum(x.n for x in xs)
    rng = _rng(201)
    m = _store(rng.normal(0, 1e-3, n) * 10.0 ** rng.uniform(-3, 1, n), dtype)
    v = _store((rng.normal(0, 1e-3, n) * 10.0 ** rng.uniform(-3, 1, n)) ** 2, dtype)
    v[::7] = 0
    vals = torch.stack([to_device(torch, m, dtype), to_device(torch, v, dtype)])
    st.pack_moments(vals)
    at = 0
    out = st.unpack_moments(tt)
    assert out.dtype == tt
    pairs = st.split_moments(out)
    for x, (p, q) in zip(xs, pairs):
        mk, vk = (_decode(a[at:at + x.n], dtype) for a in (m, v))
        x.mem = pm.encode(mk.astype(np.float32), vk.astype(np.float32))
        assert np.array_equal(x.dM.cpu().numpy(), x.mem[0]) and np.array_equal(x.dV.cpu().numpy(), x.mem[1]), x.shape
        dm, dv = pm.decode(*x.mem, x.n)
        assert np.array_equal(p.double().cpu().numpy().reshape(-1), dm), x.shape       # exact in either dtype
        assert np.array_equal(q.double().cpu().numpy().reshape(-1), dv), x.shape
        for s, d in zip(x.state, (x.dM, x.dV)):
            assert bool((s[:32] == CANARY).all()) and bool((s[32 + d.numel():] == CANARY).all())
        at += x.n
    # what was unpacked packs to the same values.  Not always to the same bytes: where a block's largest was
    # rounded down its new scale is one lower, which holds every value that the old one held.
    st.pack_moments(out)
    assert torch.equal(st.unpack_moments(tt), out)
    before = [(x.dM.clone(), x.dV.clone()) for x in xs]
    # into the middle of a caller's buffer, misaligned for vectors; nothing beside it changes
    room = torch.full((2 * n + 21,), 7.0, dtype=tt, device="cuda")
    st.unpack_moments(out=room[5:5 + 2 * n].view(2, n))
    assert torch.equal(room[5:5 + 2 * n].view(2, n), out)
    assert bool((room[:5] == 7).all()) and bool((room[5 + 2 * n:] == 7).all())
    st.pack_moments(room[5:5 + 2 * n].view(2, n))
    for x, (p, q) in zip(xs, before):
        assert torch.equal(x.dM, p) and torch.equal(x.dV, q)
    assert st.flags() == 0
    st.close()


def test_pack_values_that_are_not_numbers():
    say("case: pack NaN, infinite, negative and denormal values")
    x = Packed((210,), (512,), "f32")
    st = mm.MuonStep([x.desc()])
    vals = torch.zeros(2, 512, device="cuda")
    vals[0, ::2] = 1e-4
    vals[1] = 1e-8
    vals[0, 300], vals[0, 301], vals[1, 302], vals[1, 303], vals[1, 304] = \
        float("nan"), float("-inf"), float("nan"), -1.0, float("inf")
    vals[1, 305], vals[1, 306] = -0.0, 1e-42
    st.pack_moments(vals)
    m, v = vals.cpu().numpy()
    m[302] = m[303] = np.nan
    ref = pm.encode(m, np.abs(v))
    keep = np.ones(512, bool)
    keep[300:304] = False          # the byte of a second moment without a meaning
    assert _same_bytes(x.dM.cpu().numpy(), ref[0], 512, True)
    assert np.array_equal(x.dV.cpu().numpy()[:512][keep], ref[1][:512][keep])
    assert np.array_equal(x.dV.cpu().numpy()[512:], ref[1][512:])
    assert st.flags() & 1
    out = st.unpack_moments()
    assert bool(out[0, 300:304].isnan().all()) and not bool(out[0, 304:].isnan().any())
    st.close()


def test_conversion_calls_refuse_and_without_packed_tensors_do_nothing():
    say("case: refusals of pack and unpack")
    x = Packed((220,), (300,), "f32")
    st = mm.MuonStep([x.desc()])
    for bad in (torch.zeros(2, 299, device="cuda"), torch.zeros(2, 300), torch.zeros(300, 2, device="cuda").t(),
                torch.zeros(2, 300, device="cuda", dtype=torch.float16)):
        with pytest.raises(ValueError):
            st.pack_moments(bad)
        with pytest.raises(ValueError):
            st.unpack_moments(out=bad)
    with pytest.raises(ValueError):
        st.unpack_moments(torch.bfloat16, out=torch.zeros(2, 300, device="cuda"))
    lib = st._lib
    for call in (lib.muon_pack_moments, lib.muon_unpack_moments):
        assert call(st._h, None, 0, None) == 1                                   # NULL
        assert call(st._h, x.dW.data_ptr(), 7, None) == 3                        # dtype
        assert call(st._h, x.dW.data_ptr() + 2, 0, None) == 4                    # alignment
        assert call(st._h, x.dW.data_ptr(), 0, None) == 5                        # a registered tensor
        assert call(st._h, st.workspace.data_ptr(), 0, None) == 5                # the workspace
    st.close()
    f = [torch.zeros(10, device="cuda") for _ in range(4)]
    plain = mm.MuonStep([mm.adam_tensor_desc(*f)])
    assert plain.unpack_moments().shape == (2, 0) and plain.split_moments(plain.unpack_moments()) == []
    plain.pack_moments(torch.zeros(2, 0, device="cuda"))
    plain.close()


def test_static_scratch():
    say("case: packed AdamW on a static handle")
    hp = mm.default_hparams()
    x = Packed((230,), (123, 45), "bf16")
    st = mm.MuonStep([x.desc()], hp, static_scratch=True)
    st.set_max_grad_norm(float("inf"))
    for t in (1, 2):
        x.grad(t)
        st.step()
        x.check(t, 0, hp)
    assert st.grad_norm[1].item() == 1.0
    st.close()


def test_unpack_on_another_stream_takes_that_streams_memory():
    say("case: unpacking on a side stream while the current stream still uses a freed block")
    x = Packed((330,), (64, 4096), "bf16")
    st = mm.MuonStep([x.desc()])
    x.grad(1)
    st.step()
    want = st.unpack_moments().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    block = torch.zeros_like(want)
    place = block.data_ptr()
    del block                                    # the current stream may hand it out again, another one not
    got = st.unpack_moments(stream=side)
    assert got.data_ptr() != place
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    st.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_largest_first_moments_stay_finite(dtype):
    say(f"case: {dtype} first moments up to the type's largest, packed and stepped, against the oracle")
    tt = torch.float32 if dtype == "f32" else torch.bfloat16
    most, top = 1.875 * 2.0 ** 127, torch.finfo(tt).max
    x = Packed((360,), (1000,), dtype)
    hp = mm.default_hparams(adam_beta1=0.0, adam_beta2=0.5)       # the first moment is the gradient
    st = mm.MuonStep([x.desc()], hp)
    big = _rng(361).uniform(1.7 * 2.0 ** 127, top, 1000) * _rng(362).choice([-1, 1], 1000)
    big[:6] = most, -top, top, 1.9375 * 2.0 ** 127, 1e30, 0.0
    m = _store(big, dtype)
    m64 = _decode(m, dtype)
    v = _store(np.full(1000, 1e-8), dtype)
    st.pack_moments(torch.stack([to_device(torch, m, dtype), to_device(torch, v, dtype)]))
    x.mem = pm.encode(m64.astype(np.float32), _decode(v, dtype).astype(np.float32))
    assert _same_bytes(x.dM.cpu().numpy(), x.mem[0], 1000, True)
    out = st.unpack_moments(tt)[0].double().cpu().numpy()
    assert np.array_equal(out, pm.decode(*x.mem, 1000)[0]) and np.abs(out).max() == most
    # gradients of that size step the same way: random rounding, the second moments overflow
    x.set_grad(m64.reshape(1, 1000))
    st.step()
    x.check(1, 0, hp)
    out = st.unpack_moments(torch.float32)
    assert bool(out.isfinite().all()) and out[0].abs().max().item() == most
    assert out[1].max().item() == most and st.flags() == 0
    st.close()
