"""Packed moments, clipping and conversion as a training run uses them
together, and at the ends of their range: a run with Muon matrices, AdamW
tensors of both kinds of moments and a clipping norm, checkpointed in the
middle; tensors of more than 2^31 elements; a static handle whose scratch has
no room for the norm's sums."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from oracle import muon_oracle as orc
from oracle import packed_moments as pm
from tests.parity_common import decode, from_device, rel_f, say, to_device
from tests.test_gpu_packed_adamw import Packed, _rng

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

MUON_SHAPES = [(256, 384), (130, 70)]


class Run:
    """One run's tensors and handle."""

    def __init__(self, hp):
        self.hp = hp
        self.W, self.G, self.M = [], [], []
        for k, (r, c) in enumerate(MUON_SHAPES):
            self.W.append(to_device(torch, orc.f64_to_bf16_bits(_rng(400, k, 1).normal(0, 0.02, (r, c))), "bf16"))
            self.G.append(torch.empty(r, c, dtype=torch.bfloat16, device="cuda"))
            self.M.append(torch.zeros(r, c, device="cuda"))
        self.packed = [Packed((401, 0), (300, 64), "bf16"), Packed((401, 1), (768,), "f32"),
                       Packed((401, 2), (37, 50), "bf16", ld=56)]
        self.a = [torch.from_numpy(_rng(402, k).normal(0, 0.02, 333).astype(np.float32)).cuda() for k in range(2)]
        self.a += [torch.zeros(333, device="cuda") for _ in range(2)]
        self.start()

    def start(self, steps=0):
        descs = [mm.tensor_desc(*x) for x in zip(self.W, self.G, self.M)]
        descs += [x.desc() for x in self.packed] + [mm.adam_tensor_desc(*self.a)]
        self.opt = mm.MuonStep(descs, self.hp)
        self.opt.set_adam_step(steps)
        self.opt.set_rounding_seed(77)
        self.opt.set_max_grad_norm(0.5)

    def grads(self, t):
        for k, g in enumerate(self.G):
            g.copy_(to_device(torch, orc.f64_to_bf16_bits(_rng(403, k, t).normal(0, 1e-2, g.shape)), "bf16"))
        for x in self.packed:
            x.grad(t)
        self.a[1].copy_(torch.from_numpy(_rng(404, t).normal(0, 1e-2, 333).astype(np.float32)))

    def all_grads(self):
        return self.G + [x.dG for x in self.packed] + [self.a[1]]

    def state(self):
        return self.W + self.M + self.a + [y for x in self.packed for y in (x.dW, x.dM, x.dV)]


def test_run_with_checkpoint():
    say("case: 6 clipped steps over Muon, packed and float32-moment tensors; checkpoint by values after 3")
    hp = mm.default_hparams()
    a, b = Run(hp), Run(hp)
    for t in range(1, 7):
        a.grads(t)
        b.grads(t)
        M0 = [m.double().cpu().numpy() for m in a.M]
        a.opt.step()
        b.opt.step()
        norm, factor = (float(x) for x in a.opt.grad_norm)
        ref = pm.clip([g.double().cpu().numpy() for g in a.all_grads()], 0.5)
        assert abs(norm - ref[0]) <= 2 * 2.0 ** -24 * ref[0] and abs(factor - ref[1]) <= 2 * 2.0 ** -24 * ref[1]
        assert factor < 1
        for k, x in enumerate(a.packed):
            x.check(t, 2 + k, hp, seed=77, factor=factor, label=f"step {t}")
        mu = float(np.float32(hp.momentum))
        for M, G, m0 in zip(a.M, a.G, M0):       # EMA of the clipped gradient: three float32 roundings
            g = decode(from_device(torch, G, "bf16"), "bf16") * factor
            want = mu * m0 + (1 - mu) * g
            err = np.abs(M.double().cpu().numpy() - want)
            assert (err <= 4 * 2.0 ** -24 * (np.abs(mu * m0) + np.abs((1 - mu) * g))).all()
        for p, q in zip(a.state(), b.state()):
            if p.dtype != torch.uint8:
                assert torch.equal(p, q), t
        assert torch.equal(a.opt.unpack_moments(), b.opt.unpack_moments())
        if t == 3:          # b goes on from a file: values, count and a new handle over new buffers
            values, steps = b.opt.unpack_moments().cpu(), b.opt.adam_step()
            b.opt.close()
            for x in b.packed:
                x.dM.fill_(0x55)
                x.dV.fill_(0x55)
            b.start(steps)
            b.opt.pack_moments(values.cuda())
    assert a.opt.flags() == 0 and b.opt.flags() == 0 and a.opt.adam_step() == 6
    a.opt.close()
    b.opt.close()


def test_more_than_two_to_the_31_elements():
    rows, cols = 1 << 20, 2176
    n = rows * cols
    say(f"case: one packed tensor of {n} bf16 elements, clipped; windows against the oracle")
    hp = mm.default_hparams()
    p = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros_like(p)
    m, v = mm.packed_moment(p), mm.packed_moment(p)
    # windows of whole blocks: the start, round 2^31 and 2^32 bytes, the end
    size = 4096
    starts = [0, (1 << 31) - 2048, (1 << 31) // 2 - 2048, n - size]
    w0, g0 = {}, {}
    for k, s in enumerate(starts):
        w0[s] = orc.f64_to_bf16_bits(_rng(410, k).normal(0, 0.02, size))
        g0[s] = orc.f64_to_bf16_bits(_rng(411, k).normal(0, 1e-2, size))
        p.view(-1)[s:s + size] = to_device(torch, w0[s], "bf16")
        g.view(-1)[s:s + size] = to_device(torch, g0[s], "bf16")
    st = mm.MuonStep([mm.adam_tensor_desc(p, g, m, v)], hp, keepalive=[p, g, m, v])
    st.set_max_grad_norm(0.5)
    st.step()
    ref = pm.clip([orc.bf16_bits_to_f64(x) for x in g0.values()], 0.5)
    norm, factor = (float(x) for x in st.grad_norm)
    assert abs(norm - ref[0]) <= 2 * 2.0 ** -24 * ref[0] and abs(factor - ref[1]) <= 2 * 2.0 ** -24 * ref[1]
    betas = (float(np.float32(hp.adam_beta1)), float(np.float32(hp.adam_beta2)))
    nb = n // pm.BLOCK
    values = st.unpack_moments(torch.bfloat16)
    for s in starts:
        m1, v1 = pm.moments_f32(orc.bf16_bits_to_f64(g0[s]), np.zeros(size), np.zeros(size), betas, factor)
        # the window's words: those of its place in the tensor
        first = s // 16
        with np.errstate(over="ignore"):
            u = lambda x: np.array([x & 0xFFFFFFFF], np.uint32)  # noqa: E731
            key = pm._mix(pm._mix(pm._mix(pm._mix(u(0)) + u(0)) + u(1)) + u(0))
            word = (pm._mix(key + np.arange(first, first + size // 16, dtype=np.uint32))[:, None]
                    + np.arange(16, dtype=np.uint32) * pm.GOLDEN).reshape(-1)
        mem = pm.encode(m1, v1, word)
        b0, b1 = s // pm.BLOCK, (s + size) // pm.BLOCK
        for dev, want in ((m, mem[0]), (v, mem[1])):
            got = np.concatenate([dev[s:s + size].cpu().numpy(),
                                  dev[nb * pm.BLOCK:].view(-1, 2)[b0:b1].reshape(-1).cpu().numpy()])
            assert np.array_equal(got, want), s
        dm, dv = pm.decode(*mem, size)
        assert np.array_equal(values[0, s:s + size].double().cpu().numpy(), dm)
        assert np.array_equal(values[1, s:s + size].double().cpu().numpy(), dv)
        want, term = pm.update(orc.bf16_bits_to_f64(w0[s]), m1, v1, 1, float(np.float32(hp.adam_lr)), betas,
                               float(np.float32(hp.adam_eps)), float(np.float32(hp.adam_weight_decay)))
        got = p.view(-1)[s:s + size].double().cpu().numpy()
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * (term + np.abs(want))).all(), s
    # everything else is as it was: zero
    for s in starts:
        p.view(-1)[s:s + size] = 0
        for t in (m, v):
            t[s:s + size] = 0
    assert not bool(p.any())
    for t in (m, v):
        for part in t[:n].split(1 << 30):
            assert not bool(part.any())
    st.pack_moments(values)
    again = st.unpack_moments(torch.bfloat16)
    assert torch.equal(again.view(torch.int16), values.view(torch.int16))
    st.close()


def test_rows_with_gaps_past_two_to_the_31():
    say("case: packed rows of 2 in a buffer of 2^31 + elements (leading dimension 2100)")
    rows, cols, ld = 1 << 20, 2, 2100
    hp = mm.default_hparams()
    wide = torch.zeros(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)
    p = wide[:, :cols]
    g = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    g[-1, 1], g[0, 0], g[rows // 2, 0] = 1e-2, -2e-2, 3e-2
    m, v = mm.packed_moment(p), mm.packed_moment(p)
    st = mm.MuonStep([mm.adam_tensor_desc(p, g, m, v)], hp, keepalive=[wide, g, m, v])
    st.step()
    # the first step moves a weight by lr (against its gradient's sign) up to eps / |g|
    lr = float(np.float32(hp.adam_lr))
    got = p[g != 0].double().cpu().numpy() * np.sign(g[g != 0].double().cpu().numpy())
    assert (np.abs(got + lr) <= lr * (2.0 ** -8 + 1e-5)).all()
    p[-1, 1] = p[0, 0] = p[rows // 2, 0] = 0
    for part in wide.view(-1).split(1 << 30):
        assert not bool(part.any())
    st.close()


def test_static_scratch_without_room_for_the_norm():
    say("case: a static handle that fits only without the norm's sums")
    hp = mm.default_hparams()
    w = [torch.zeros(2048, 2304, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    mom = torch.zeros(2048, 2304, device="cuda")
    descs = [mm.tensor_desc(*w, mom)]
    limit = 64 << 20
    # small float32 matrices, then AdamW vectors a few at a time, until the sums no longer fit (a static handle's
    # plan has one lane, so its size is not workspace_size's to the byte)
    keep = []
    while mm.workspace_size(descs, hp) + (160 << 10) < limit:
        t = [torch.zeros(64, 64, device="cuda") for _ in range(3)]
        keep += t
        descs.append(mm.tensor_desc(*t))
    for _ in range(200):
        st = mm.MuonStep(descs, hp, static_scratch=True)
        try:
            st.set_max_grad_norm(1.0)
        except mm.MuonError as err:
            e = err
            break
        st.close()
        for _ in range(16):
            t = [torch.zeros(1, device="cuda") for _ in range(4)]
            keep += t
            descs.append(mm.adam_tensor_desc(*t))
    else:
        raise AssertionError("the norm's sums always fitted")
    assert "WORKSPACE_TOO_SMALL" in str(e) and st.grad_norm is None
    st.set_max_grad_norm(0.0)
    st.step()
    assert st.flags() == 0
    st.close()


def test_tensors_of_another_device_are_refused():
    say("case: a packed tensor that is not on the handle's device")
    p = torch.zeros(100)
    with pytest.raises(ValueError):
        mm.MuonStep([mm.adam_tensor_desc(p, p.clone(), mm.packed_moment(p), mm.packed_moment(p))])


def test_clipping_before_the_preconditioner():
    say("case: clipped Newton-Muon step against one on gradients scaled beforehand")
    hp = mm.default_hparams()
    pc = mm.MuonPrecond()
    pc.d, pc.nblocks = 128, 1
    gen = torch.Generator(device="cuda").manual_seed(5)
    acts = torch.randn(2048, 128, device="cuda", generator=gen)
    w = torch.randn(256, 128, device="cuda", generator=gen) * 0.02
    g = torch.randn(256, 128, device="cuda", generator=gen) * 1e-2
    out = []
    factor = None
    for clipped in (True, False):
        p, gg, m = w.clone(), g.clone(), torch.zeros_like(w)
        if not clipped:
            gg *= factor
        st = mm.MuonStep([mm.tensor_desc(p, gg, m, precond=0)], hp, [pc], keepalive=[p, gg, m])
        st.precond_refresh(0, 0, acts)
        if clipped:
            st.set_max_grad_norm(0.25)
        st.step()
        if clipped:
            factor = st.grad_norm[1].clone()
            assert 0 < factor.item() < 1
        out.append((m.cpu().numpy(), p.cpu().numpy()))
        assert st.flags() == 0
        st.close()
    # (f G) S^-1 and f (G S^-1): float32 sums of 128 products of either, each rounded 128 times at most
    assert rel_f(out[0][0], out[1][0]) <= 128 * 2.0 ** -24
    # float32 Newton-Schulz of two momenta that close: its own parity bar, 1e-5, on the update lr * O; the
    # weights are larger than the update
    assert rel_f(out[0][1], out[1][1]) <= 1e-5


def test_debug_build_matches():
    say("case: the bounds-checking build, packed and clipped, bitwise as the release build")
    from matrix_aware_optimizer_muon_amd import build as BLD
    hp = mm.default_hparams()
    states = []
    for library in (None, BLD.DEBUG_LIB):
        xs = [Packed((420, k), s, d) for k, (s, d) in enumerate([((300, 64), "bf16"), ((5001,), "f32")])]
        st = mm.MuonStep([x.desc() for x in xs], hp, library=library)
        for t in (1, 2, 3):
            if t == 2:
                st.set_max_grad_norm(0.25)
            for x in xs:
                x.grad(t)
            st.step()
        states.append([y.clone() for x in xs for y in (x.dW, x.dM, x.dV)] + [st.grad_norm.clone(), st.unpack_moments()])
        assert st.flags() == 0
        st.close()
    for a, b in zip(*states):
        assert torch.equal(a, b)


def test_run_moves_from_float32_moments_to_packed_ones():
    say("case: three steps with float32 moments, then packed ones from them, against the oracle")
    hp = mm.default_hparams()
    xs = [Packed((430, k), s, d, ld=ld) for k, (s, d, ld) in enumerate(
        [((300, 64), "bf16", None), ((777,), "f32", None), ((37, 50), "bf16", 56)])]
    old = [tuple(torch.zeros(x.shape, device="cuda") for _ in range(2)) for x in xs]
    st = mm.MuonStep([mm.adam_tensor_desc(x.dW, x.dG, *mv) for x, mv in zip(xs, old)], hp)
    for t in (1, 2, 3):
        for x in xs:
            x.grad(t)
        st.step()
    steps = st.adam_step()
    st.close()
    opt = mm.MuonStep([x.desc() for x in xs], hp)
    values = torch.empty(2, opt.packed_elements(), device="cuda")
    for (first, second), (m, v) in zip(opt.split_moments(values), old):
        first.copy_(m.reshape(first.shape)), second.copy_(v.reshape(second.shape))
    opt.pack_moments(values)
    opt.set_adam_step(steps)
    for x, (m, v) in zip(xs, old):
        x.mem = pm.encode(m.cpu().numpy().reshape(-1), v.cpu().numpy().reshape(-1))
        assert np.array_equal(x.dM.cpu().numpy(), x.mem[0]) and np.array_equal(x.dV.cpu().numpy(), x.mem[1])
        x.w = from_device(torch, x.dW.contiguous(), x.dtype).reshape(x.w.shape)
        x.ring = [b.clone() for b in x.bufs]
    for t in (4, 5):
        for x in xs:
            x.grad(t)
        opt.step()
        for k, x in enumerate(xs):
            x.check(t, k, hp, label=f"step {t}")
    assert opt.flags() == 0 and opt.adam_step() == 5
    opt.close()
