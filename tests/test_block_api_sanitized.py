"""The host-side tests of the operators around retention (tests/test_block_api.py) again, against
a copy of the library whose host code is built with AddressSanitizer and
UndefinedBehaviorSanitizer (device code unchanged; no GPU needed)."""
import os
import subprocess
import sys
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]
sys.path.insert(0, str(ROOT / "linear_recurrent_sequence_rn_amd"))


def test_block_api_tests_pass_under_asan_and_ubsan(tmp_path):
    import build
    if not Path(build.HIPCC).exists():
        pytest.skip("hipcc not available")
    lib = build.build(sanitize=True, lib=tmp_path / "librn_retention.so")
    env = dict(os.environ, RN_LIB_PATH=str(lib), LD_PRELOAD=build.sanitizer_runtime(),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        "-m", "not gpu", "tests/test_block_api.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = r.stdout[-3000:] + r.stderr[-3000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "failed" not in r.stdout, tail
