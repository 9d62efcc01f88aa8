"""The kernels' index arithmetic at sizes near 2^31, on the host under UndefinedBehaviorSanitizer
(tests/sanitize/kla_index_sanitize.hip; no GPU needed): a device store at a wrapped index would be
one out of range, which no test on a GPU may show."""

import os
import subprocess

import pytest

import test_abi_sanitized as base
from gated_delta_rule_kla_amd import build as libbuild

SOURCE = os.path.join(base.ROOT, "tests", "sanitize", "kla_index_sanitize.hip")


@pytest.mark.timeout(600)
def test_index_arithmetic_on_the_host(tmp_path):
    hipcc = base._hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "index")
    r = subprocess.run([hipcc, *libbuild._flags(), *base.SAN, "-x", "hip", SOURCE, "-o", exe], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    log = r.stdout + r.stderr
    assert "AddressSanitizer" not in log and "runtime error" not in log, log[-3000:]
    assert r.returncode == 0 and "ok: 0 failure(s)" in r.stdout, log[-3000:]
