"""MI355X-native Muon optimizer step: a C-ABI library (libmuon.so, HIP for
gfx950) and its thin ctypes binding.  See include/muon.h for the ABI."""

from matrix_aware_optimizer_muon_amd.binding import (  # noqa: F401
    LIB_PATH, MuonError, MuonHparams, MuonMx4, MuonPrecond, MuonStep, MuonTensor, Mx4, Mx4Copies,
    adam_tensor_desc, default_hparams, header_functions, load_library, mx4_dequantize, mx4_desc,
    mx4_empty, mx4_quantize, packed_moment, packed_moment_bytes, plan_describe, tensor_desc, workspace_size,
)
