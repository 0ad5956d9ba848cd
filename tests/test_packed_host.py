"""Host-only checks of packed moments and gradient clipping (no GPU): sizes,
refusals, plans.  Pointers are fake addresses the library only compares."""

import ctypes

import pytest

import matrix_aware_optimizer_muon_amd as mm
from matrix_aware_optimizer_muon_amd import binding as B

torch = pytest.importorskip("torch")
lib = B.load_library()
BASE = 1 << 36


def packed(rows, cols, base=BASE, dtype=B.MUON_BF16, ld=None):
    """An AdamW tensor with packed moments, and the address behind it."""
    es = 4 if dtype == B.MUON_F32 else 2
    up = lambda b: (b + 4095) // 4096 * 4096 + 4096  # noqa: E731
    span, moment = up(rows * (ld or cols) * es), up(mm.packed_moment_bytes(rows * cols))
    t = B.MuonTensor()
    t.param, t.grad = base, base + span
    t.momentum, t.exp_avg_sq = base + 2 * span, base + 2 * span + moment
    t.rows, t.cols = rows, cols
    t.ld_param = t.ld_grad = ld or cols
    t.ld_momentum = cols
    t.dtype, t.precond, t.lr_mult, t.kind, t.state_bits = dtype, -1, 1.0, B.KIND_ADAMW, 8
    return t, base + 2 * span + 2 * moment


def status(*tensors):
    ta, n = B._array(list(tensors), B.MuonTensor)
    pa, npc = B._array([], B.MuonPrecond)
    out = ctypes.c_size_t(0)
    st = lib.muon_workspace_size(ta, n, pa, npc, ctypes.byref(mm.default_hparams()), ctypes.byref(out))
    return B.STATUS_NAMES[st]


@pytest.mark.parametrize("n,blocks", [(1, 1), (255, 1), (256, 1), (257, 2), (50257 * 768, 150771), (1 << 35, 1 << 27)])
def test_moment_bytes(n, blocks):
    assert mm.packed_moment_bytes(n) == 258 * blocks


@pytest.mark.parametrize("n", [0, -1, (1 << 35) + 1])
def test_moment_bytes_refusals(n):
    assert lib.muon_packed_moment_bytes(n) == 0
    with pytest.raises(ValueError):
        mm.packed_moment_bytes(n)


def test_accepts_and_plans():
    a, end = packed(300, 64)
    b, end = packed(1, 9000, end, B.MUON_F32)
    c, end = packed(37, 48, end, ld=56)
    assert status(a, b, c) == "MUON_OK"
    f = B.MuonTensor.from_buffer_copy(a)       # the same beside it with float32 moments
    f.param, f.grad, f.momentum, f.exp_avg_sq = (end + k * (1 << 20) for k in range(4))
    f.state_bits = 32
    plan = mm.plan_describe([a, f, b, c], mm.default_hparams())
    assert plan["packed_tensors"] == 3 and plan["packed_tasks"] == 10 + 5 + 1
    assert plan["adamw_tensors"] == 1
    assert plan["launch_order"] == ["adam_tick", "adamw", "adamw_packed"]
    # few packed chunks alone: no launch for the count before theirs
    order = lambda *ts: mm.plan_describe(list(ts), mm.default_hparams())["launch_order"]  # noqa: E731
    assert order(a) == order(a, b, c) == order(packed(2048, 2048)[0]) == ["adamw_packed"]
    assert order(packed(2049, 2048)[0]) == ["adam_tick", "adamw_packed"]
    assert mm.plan_describe([f], mm.default_hparams())["launch_order"] == ["adam_tick", "adamw"]


def test_refusals():
    def bad(**changes):
        t, _ = packed(300, 64)
        for k, v in changes.items():
            setattr(t, k, v)
        return status(t)
    assert bad() == "MUON_OK"
    assert bad(state_bits=4) == "MUON_ERR_BAD_ARG"
    assert bad(state_bits=-8) == "MUON_ERR_BAD_ARG"
    assert bad(ld_momentum=65) == "MUON_ERR_BAD_SHAPE"
    assert bad(exp_avg_sq=None) == "MUON_ERR_NULL_ARG"
    assert bad(momentum=None) == "MUON_ERR_NULL_ARG"
    assert bad(split_rows=100) == "MUON_ERR_BAD_ARG"
    t, _ = packed(300, 64)
    assert bad(momentum=t.momentum + 8) == "MUON_ERR_ALIGNMENT"
    assert bad(exp_avg_sq=t.exp_avg_sq + 4) == "MUON_ERR_ALIGNMENT"
    assert bad(exp_avg_sq=t.momentum) == "MUON_ERR_ALIASING"
    # the buffer reaches to the last scale: 75 blocks of 258 bytes
    assert bad(exp_avg_sq=t.momentum + 75 * 258 - 6) == "MUON_ERR_ALIASING"     # 16-byte aligned
    assert bad(exp_avg_sq=t.momentum + (75 * 258 + 15) // 16 * 16) == "MUON_OK"
    # packed moments are AdamW's alone
    assert bad(kind=B.KIND_MUON, exp_avg_sq=None) == "MUON_ERR_UNSUPPORTED"
    big, _ = packed(1 << 15, 1 << 20)
    assert status(big) == "MUON_ERR_UNSUPPORTED"            # 2^35 elements: 2^32 threads
    big.rows += 1
    assert status(big) == "MUON_ERR_UNSUPPORTED"
    half, end = packed(1 << 14, 1 << 20)
    assert status(half, packed(1 << 14, 1 << 20, end)[0]) == "MUON_ERR_UNSUPPORTED"


def test_calls_without_a_handle():
    names = [lib.muon_set_rounding_seed(None, 1), lib.muon_set_max_grad_norm(None, 1.0, None),
             lib.muon_pack_moments(None, None, 0, None), lib.muon_unpack_moments(None, None, 0, None)]
    assert [B.STATUS_NAMES[s] for s in names] == ["MUON_ERR_NULL_ARG"] * 4


def test_descriptor_from_tensors():
    p = torch.zeros(30, 20, dtype=torch.bfloat16)
    g = torch.zeros_like(p)
    m, v = mm.packed_moment(p), mm.packed_moment(p)
    assert m.dtype == torch.uint8 and m.numel() == 3 * 258 and not m.any()
    d = mm.adam_tensor_desc(p, g, m, v, lr_mult=0.5)
    assert (d.rows, d.cols, d.ld_param, d.ld_momentum, d.state_bits, d.reserved, d.kind) == (30, 20, 20, 20, 8, 8, 1)
    assert d.momentum == m.data_ptr() and d.exp_avg_sq == v.data_ptr() and d.lr_mult == 0.5
    wide = torch.zeros(30, 32, dtype=torch.bfloat16)
    assert mm.adam_tensor_desc(wide[:, :20], g, m, v).ld_param == 32
    vec = torch.zeros(600)
    assert mm.adam_tensor_desc(vec, torch.zeros(600), m, v).rows == 1
    for bad in ((p, g[:, :10], m, v), (p, g.float(), m, v), (p, g, m[:-1], v), (p, g, m, v.float()),
                (p, g, m, torch.zeros_like(p, dtype=torch.float32)), (p.t(), g.t(), m, v),
                (p.half(), g.half(), m, v), (p, g, m.view(3, 258), v)):
        with pytest.raises(ValueError):
            mm.adam_tensor_desc(*bad)
    f = torch.zeros(30, 20)
    assert mm.adam_tensor_desc(p, g, f, f.clone()).state_bits == 0


MOST_CHUNKS = (1 << 24) - 1          # 2^24 blocks of 256 threads are 2^32, one launch's limit
LARGE = ((1 << 20) - 1, 1 << 15)     # 2^24 - 16 chunks


def many(shapes):
    ts, end = [], BASE
    for r, c in shapes:
        t, end = packed(r, c, end)
        ts.append(t)
    return ts


@pytest.mark.parametrize("shapes", [[LARGE, (15, 2048)], [LARGE, (13, 2048), (1, 1), (1, 2047)]])
def test_most_chunks_of_a_handle(shapes):
    assert sum(-(-r * c // 2048) for r, c in shapes) == MOST_CHUNKS
    assert status(*many(shapes)) == "MUON_OK"


@pytest.mark.parametrize("shapes", [
    [LARGE, (1, (1 << 15) - 1)],                              # 2^35 - 1 elements, 2^24 chunks
    [LARGE, (15, 2048), (1, 1)],                              # a chunk for one element
    [LARGE, (12, 2048), *[(1, k) for k in (1, 2, 255, 2047)]],
])
def test_too_many_chunks_are_refused(shapes):
    assert sum(r * c for r, c in shapes) < 1 << 35
    assert sum(-(-r * c // 2048) for r, c in shapes) > MOST_CHUNKS
    assert status(*many(shapes)) == "MUON_ERR_UNSUPPORTED"
