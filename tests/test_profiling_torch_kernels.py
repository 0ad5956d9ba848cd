"""Torch's own kernels, which run around a step (buffers made and filled), are
no phase of it: they are told apart, and the traffic summary has none (CPU only)."""

from matrix_aware_optimizer_muon_amd import profiling as P
from tests.test_profiling_host import BX, COPY, _write

FILL = ("void at::native::vectorized_elementwise_kernel<4, at::native::FillFunctor<float>, std::array<char*, 1ul> >"
        "(int, at::native::FillFunctor<float>, std::array<char*, 1ul>)")
MANGLED = "_ZN2at6native29vectorized_elementwise_kernelILi4ENS0_11FillFunctorIfEESt5arrayIPcLm1EEEEviT0_T1_"


def test_kinds():
    assert P.kernel_kind(FILL) == P.kernel_kind(MANGLED) == "torch"
    assert P.kernel_kind("void muon::(anonymous namespace)::quantize_kernel<true, true>(...)") == "quantize_kernel"


def test_traffic_leaves_them_out(tmp_path):
    fields = ["Dispatch_Id", "Kernel_Name", "Counter_Name", "Counter_Value"]
    for d, name, rows in (("f", "FETCH_SIZE", [(1, BX, 100.0), (2, FILL, 3.0), (3, MANGLED, 5.0)]),
                          ("w", "WRITE_SIZE", [(1, BX, 50.0), (2, FILL, 7.0), (3, MANGLED, 9.0)]),
                          ("cf", "FETCH_SIZE", [(1, COPY, 1024.0)]), ("cw", "WRITE_SIZE", [(1, COPY, 1024.0)])):
        _write(str(tmp_path / d / "run_counter_collection.csv"), fields,
               [{"Dispatch_Id": i, "Kernel_Name": k, "Counter_Name": name, "Counter_Value": v} for i, k, v in rows])
    got = P.traffic(*(str(tmp_path / d) for d in ("f", "w", "cf", "cw")), 1 << 20, ["cmd"])
    for part in ("per_launch_bytes", "per_launch_read_bytes", "per_launch_write_bytes"):
        assert set(got[part]) == {"bx"}, part
    assert got["per_launch_bytes"]["bx"] == 150 * 1024
