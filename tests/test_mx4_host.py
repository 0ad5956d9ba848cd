"""Host-only checks of microscaled 4-bit floats (no GPU): every refusal of the
list calls and of the binding.  Pointers are fake addresses the library only
compares; no call here passes its checks."""

import ctypes

import pytest

import matrix_aware_optimizer_muon_amd as mm
from matrix_aware_optimizer_muon_amd import binding as B
from tests.test_binding_device_host import World

torch = pytest.importorskip("torch")
lib = B.load_library()
BASE = 1 << 36


def matrix(k=0, rows=100, cols=70, dtype=B.MUON_BF16, row=True, col=True):
    """The k-th matrix of a list, its buffers apart from the others'."""
    at = BASE + k * (1 << 30)
    d = mm.MuonMx4()
    d.values, d.rows, d.cols, d.ld, d.dtype = at, rows, cols, cols, dtype
    if row:
        d.row_codes, d.row_scales = at + (1 << 26), at + (2 << 26)
        d.ld_row_codes, d.ld_row_scales = 16 * -(-cols // 32), 4 * -(-cols // 128)
    if col:
        d.col_codes, d.col_scales = at + (3 << 26), at + (4 << 26)
        d.ld_col_codes, d.ld_col_scales = 16 * -(-rows // 32), 4 * -(-rows // 128)
    return d


def refused(*ms, axis=None, rounding=0, n=None):
    """The name of the status, and the text, of a list that does not pass."""
    arr, count = B._array(list(ms), mm.MuonMx4)
    n = count if n is None else n
    if axis is None:
        st = lib.muon_mx4_quantize(arr, n, rounding, 0, None)
    else:
        st = lib.muon_mx4_dequantize(arr, n, axis, None)
    assert st != 0
    return B.STATUS_NAMES[st], lib.muon_last_error().decode()


def sentinel():
    d = matrix(50)
    d.values = None
    return d


def passes(*ms, axis=None):
    """Whether all is found right up to the sentinel's missing values."""
    status, text = refused(*ms, sentinel(), axis=axis)
    return status == "MUON_ERR_NULL_ARG" and text == f"matrix {len(ms)}: values is NULL"


def test_lists_pass_up_to_the_sentinel():
    assert passes(matrix(0), matrix(1, row=False), matrix(2, col=False), matrix(3, 1, 1, B.MUON_F32))
    assert passes(matrix(0), axis=0) and passes(matrix(0, col=False), axis=1)


@pytest.mark.parametrize("field,value,status", [
    ("rows", 0, "BAD_SHAPE"), ("cols", 0, "BAD_SHAPE"), ("rows", (1 << 30) + 1, "BAD_SHAPE"), ("cols", -5, "BAD_SHAPE"),
    ("ld", 69, "BAD_SHAPE"), ("dtype", 2, "BAD_DTYPE"), ("dtype", -1, "BAD_DTYPE"), ("reserved", 1, "BAD_ARG"),
    ("values", None, "NULL_ARG"), ("values", BASE + 1, "ALIGNMENT"),
    ("row_codes", None, "NULL_ARG"), ("row_scales", None, "NULL_ARG"), ("col_codes", None, "NULL_ARG"),
    ("col_scales", None, "NULL_ARG"), ("row_codes", BASE + (1 << 26) + 8, "ALIGNMENT"),
    ("row_scales", BASE + (2 << 26) + 2, "ALIGNMENT"), ("col_codes", BASE + (3 << 26) + 4, "ALIGNMENT"),
    ("col_scales", BASE + (4 << 26) + 1, "ALIGNMENT"), ("ld_row_codes", 32, "BAD_SHAPE"), ("ld_row_codes", 56, "ALIGNMENT"),
    ("ld_row_scales", 2, "BAD_SHAPE"), ("ld_row_scales", 6, "ALIGNMENT"), ("ld_col_codes", 48, "BAD_SHAPE"),
    ("ld_col_codes", 72, "ALIGNMENT"), ("ld_col_scales", 3, "BAD_SHAPE"), ("ld_col_scales", 5, "ALIGNMENT"),
    ("ld_row_codes", 1 << 40, "BAD_SHAPE"), ("ld_col_scales", 1 << 40, "BAD_SHAPE")])
def test_refusals_of_one_matrix(field, value, status):
    d = matrix(1)
    setattr(d, field, value)
    for ms in ([d], [matrix(0), d]):
        assert refused(*ms)[0] == "MUON_ERR_" + status
    row, col = "row_" in field, "col_" in field
    if not col:
        assert refused(d, axis=1)[0] == "MUON_ERR_" + status
    if not row:
        assert refused(d, axis=0)[0] == "MUON_ERR_" + status
    # the form that is not read does not matter
    if row:
        assert passes(d, axis=0)
    if col:
        assert passes(d, axis=1)


def test_refusals_of_a_call():
    assert refused(matrix(0), rounding=2)[0] == refused(matrix(0), rounding=-1)[0] == "MUON_ERR_BAD_ARG"
    assert refused(matrix(0), axis=2)[0] == refused(matrix(0), axis=-1)[0] == "MUON_ERR_BAD_ARG"
    assert refused(matrix(0), n=-1)[0] == "MUON_ERR_BAD_ARG"
    assert refused(matrix(0, row=False, col=False))[0] == "MUON_ERR_NULL_ARG"
    assert refused(matrix(0, col=False), axis=0)[0] == refused(matrix(0, row=False), axis=1)[0] == "MUON_ERR_NULL_ARG"
    assert lib.muon_mx4_quantize(None, 1, 0, 0, None) == 1
    big = matrix(0, 1 << 30, 1 << 14)
    big.ld_col_codes, big.ld_col_scales = 1 << 29, 1 << 25
    assert refused(big)[0] == "MUON_ERR_UNSUPPORTED"


def test_overlaps():
    def moved(**at):
        d = matrix(1)
        for k, v in at.items():
            setattr(d, k, v)
        return refused(matrix(0), d)[0]
    last = BASE + 100 * 70 * 2                      # behind the first matrix's values
    assert moved(row_codes=BASE + 96) == "MUON_ERR_ALIASING"                    # codes over values
    assert moved(col_scales=last // 4 * 4 - 4) == "MUON_ERR_ALIASING"
    assert moved(row_scales=BASE + (2 << 26) + 4 * 99) == "MUON_ERR_ALIASING"   # scales over scales
    assert moved(col_codes=matrix(1).row_codes + 16) == "MUON_ERR_ALIASING"     # a matrix's two forms
    assert moved(values=BASE + (1 << 26)) == "MUON_ERR_ALIASING"                # values over another's codes
    # read by both, written by none: allowed, and a form just behind the values
    both, behind = matrix(1), matrix(2)
    both.values = BASE
    behind.row_codes = -(-last // 16) * 16
    assert passes(matrix(0), both, behind)
    # reading back, the values are what is written
    assert refused(matrix(0), both, axis=1)[0] == "MUON_ERR_ALIASING"
    shared = matrix(1)
    shared.row_codes, shared.row_scales = matrix(0).row_codes, matrix(0).row_scales
    assert passes(matrix(0), shared, axis=1) and refused(matrix(0), shared)[0] == "MUON_ERR_ALIASING"
    inside = matrix(1)                              # a written span around a read one around another
    inside.row_codes, inside.ld_row_codes = BASE - 4096, 1 << 16
    assert refused(inside, matrix(0))[0] == "MUON_ERR_ALIASING"


def test_binding_refusals():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    for codes, scales, rows, cols, axis in ((u8(4, 16), u8(4, 1), 4, 33, 1), (u8(4, 32), u8(4, 1), 4, 33, 1),
                                            (u8(4, 32), u8(3, 4), 4, 33, 1), (u8(4, 32), u8(4, 4), 4, 33, 0),
                                            (u8(4, 32), u8(4, 4), 4, 33, 2), (u8(128), u8(4, 4), 4, 33, 1),
                                            (u8(4, 32).float(), u8(4, 4), 4, 33, 1), (u8(32, 4).t(), u8(4, 4), 4, 33, 1),
                                            (u8(1, 32).expand(4, 32), u8(4, 4), 4, 33, 1)):
        with pytest.raises(ValueError):
            mm.Mx4(codes, scales, rows, cols, axis)
    form = mm.Mx4(u8(4, 32), u8(4, 4), 4, 33)
    for shape in ((), (0,), (0, 4), (4, 0), (0, 3, 4)):
        with pytest.raises(ValueError):
            mm.mx4_quantize(torch.zeros(shape))
        with pytest.raises(ValueError):
            mm.Mx4Copies([torch.zeros(shape)])
    with pytest.raises(ValueError):
        mm.mx4_desc(torch.zeros(5, 33), form)
    with pytest.raises(ValueError):
        mm.mx4_desc(torch.zeros(4, 33, dtype=torch.float16), form)
    with pytest.raises(ValueError):
        mm.mx4_desc(torch.zeros(33, 4).t(), form)
    with pytest.raises(ValueError):
        mm.mx4_quantize(torch.zeros(4, 33), rounding="up")
    for bad in ((), (1, 1), 2, (0, 2)):
        with pytest.raises(ValueError):
            mm.Mx4Copies([torch.zeros(4, 33)], axis=bad)
    with pytest.raises(ValueError):
        mm.Mx4Copies([])
    for call in (lambda: mm.mx4_quantize(torch.zeros(4, 33)), lambda: mm.mx4_dequantize(form),
                 lambda: mm.Mx4Copies([torch.zeros(4, 33)]).quantize(),
                 lambda: mm.Mx4Copies([torch.zeros(4, 33)]).dequantize()):       # host memory
        with pytest.raises(ValueError):
            call()
    copies = mm.Mx4Copies([torch.zeros(4, 33), torch.zeros(7)], axis=1)
    for axis, dtype, out in ((0, None, None), (1, torch.float16, None), (1, torch.float32, torch.zeros(139).bfloat16()),
                             (1, None, torch.zeros(138)), (1, None, torch.zeros(278)[::2])):
        with pytest.raises(ValueError):
            copies.dequantize(axis=axis, dtype=dtype, out=out)


def test_descriptions():
    """What the binding hands over, for lines with gaps, one line and both forms."""
    x = torch.zeros(6, 80)[:, :70]
    codes, scales = torch.zeros(6, 64, dtype=torch.uint8), torch.zeros(6, 8, dtype=torch.uint8)
    d = mm.mx4_desc(x, mm.Mx4(codes[:, :48], scales[:, :3], 6, 70))
    assert (d.rows, d.cols, d.ld, d.ld_row_codes, d.ld_row_scales, d.dtype) == (6, 70, 80, 64, 8, 0)
    assert d.col_codes is None and d.col_scales is None
    one = mm.mx4_desc(torch.zeros(70), mm.Mx4(codes[:1, :48], scales[:1, :3], 1, 70))
    assert (one.rows, one.cols, one.ld, one.ld_row_codes, one.ld_row_scales) == (1, 70, 70, 48, 4)
    copies = mm.Mx4Copies([torch.zeros(6, 70), torch.zeros(3, 2, 2)])
    assert copies.elements == 432 and [tuple(v.shape) for v in copies.split(torch.zeros(432))] == [(6, 70), (3, 4)]
    assert [[f.axis for f in c] for c in copies.copies] == [[1, 0], [1, 0]]
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel()) for c in copies.copies for f in c for t in (f.codes, f.scales))
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    assert all(f.codes.data_ptr() % 16 == 0 and f.scales.data_ptr() % 4 == 0 for c in copies.copies for f in c)


def test_exported_and_declared():
    assert {"muon_mx4_quantize", "muon_mx4_dequantize"} <= set(mm.header_functions())
    assert ctypes.sizeof(mm.MuonMx4) == 104


@pytest.mark.parametrize("index", [0, 1])
def test_calls_run_on_the_tensors_device(monkeypatch, index):
    """As a handle's do: the library is called with the tensors' device the current one, and its stream."""
    world = World()
    monkeypatch.setattr(B, "_torch", lambda: world)
    B._launch_on(torch.device("cuda", index), world.muon_mx4_quantize, None, 0, 0, 0, None)
    assert world.calls == [("muon_mx4_quantize", index)] and world.current == 0
