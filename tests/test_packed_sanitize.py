"""The planner's part in packed moments and the gradient norm under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only), with the driver
of test_host_sanitize: packed tensors of every kind, beside the others and
refused ones; statuses, sizes and plans must equal the shipped library's."""

import json
import os
import subprocess

import pytest

import matrix_aware_optimizer_muon_amd as mm
from matrix_aware_optimizer_muon_amd import binding as B
from tests.test_packed_host import packed

host = pytest.importorskip("tests.test_host_sanitize")
driver = host.driver


def _requests():
    shapes = [(1, 1, B.MUON_BF16, None), (1, 257, B.MUON_F32, None), (300, 64, B.MUON_BF16, None),
              (37, 48, B.MUON_F32, 56), (37, 50, B.MUON_BF16, 51), (50257, 768, B.MUON_BF16, None), (1 << 20, 1, B.MUON_F32, 3)]
    ts, end = [], 1 << 36
    for r, c, dt, ld in shapes:
        t, end = packed(r, c, end, dt, ld)
        ts.append(t)
    out = [("all", (ts, [], mm.default_hparams()))] + [("alone", ([t], [], mm.default_hparams())) for t in ts]
    mixed, _, hp = host.workload_request("gpt2s_aux")
    more, at = [], 1 << 44
    for r, c, dt, ld in shapes:
        t, at = packed(r, c, at, dt, ld)
        more.append(t)
    out.append(("beside", (mixed + more, [], hp)))
    refused = []
    for field, value in (("state_bits", 4), ("ld_momentum", 65), ("momentum", (1 << 36) + 8), ("kind", 0)):
        t, _ = packed(300, 64)
        setattr(t, field, value)
        refused.append((field, ([t], [], mm.default_hparams())))
    return out + refused, len(refused)


def test_packed_requests_under_sanitizers(driver, tmp_path):
    reqs, n_refused = _requests()
    path = tmp_path / "requests.bin"
    path.write_bytes(b"".join(host._serialise(*r) for _, r in reqs))
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([driver, str(path)], stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True, env=env,
                       timeout=600)
    assert r.returncode == 0 and "Sanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[-6000:]
    lines = r.stdout.splitlines()
    assert len(lines) == 2 * len(reqs)
    refused = 0
    for (label, req), head, body in zip(reqs, lines[::2], lines[1::2]):
        _, _, _, st, _, nbytes = head.split()
        plan = json.loads(body[len("plan "):]) if body.startswith("plan ") else None
        assert (st, int(nbytes), plan) == host._library_result(*req), label
        refused += st != "MUON_OK"
    assert refused == n_refused
