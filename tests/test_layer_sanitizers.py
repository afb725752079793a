"""The host-only tests of a layer's operators' front end once more against the AddressSanitizer and
UndefinedBehaviorSanitizer build of the host code."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_layer_abi_under_asan_ubsan():
    from matrix_orthogonalising_optimizer_muon_amd import build
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    rt = build.asan_runtime()
    if rt is None:
        pytest.skip("no AddressSanitizer runtime in the ROCm toolchain")
    lib = build.build_asan()
    env = dict(os.environ, MUON_AMD_LIB=lib, LD_PRELOAD=rt,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_layer_abi.py"), "-k", "not python"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-4000:])
    assert "passed" in r.stdout and "failed" not in r.stdout
