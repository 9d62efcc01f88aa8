"""The host code of linear attention and of the later 4-bit cache entry points under the sanitizers
(no GPU needed): the objects that tests/test_abi_sanitized.py builds, with a driver of their own
(tests/sanitize/kla_more_operators_sanitize.c)."""

import glob
import os
import subprocess

import pytest

import test_abi_sanitized as base
from gated_delta_rule_kla_amd import build as libbuild

DRIVER = os.path.join(base.ROOT, "tests", "sanitize", "kla_more_operators_sanitize.c")


@pytest.mark.timeout(900)
def test_more_operators_host_code_under_the_sanitizers(tmp_path):
    hipcc = base._hipcc()
    if hipcc is None or base._clang(hipcc) is None:
        pytest.skip("hipcc or its clang not available")
    out = os.path.dirname(base._build(hipcc))
    objs = [o for o in glob.glob(os.path.join(out, "*.o")) if not o.endswith("_driver.o")]
    assert len(objs) == len(libbuild.SOURCES)
    driver, exe = str(tmp_path / "driver.o"), str(tmp_path / "driver")
    host = [f for f in base.SAN if f != "-Xarch_host"]
    for cmd in ([base._clang(hipcc), "-x", "c", "-std=c11", "-O1", *host, "-I", os.path.join(base.ROOT, "include"),
                 "-c", DRIVER, "-o", driver],
                [hipcc, f"--offload-arch={libbuild.ARCH}", *base.SAN, *objs, driver, "-o", exe]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    log = r.stdout + r.stderr
    assert "AddressSanitizer" not in log and "runtime error" not in log, log
    assert r.returncode == 0 and "ok: 0 failure(s)" in r.stdout, log
