"""The host side of the vocabulary cross-entropy, the adapters and the orthogonalised update under AddressSanitizer and
UndefinedBehaviorSanitizer: their argument checks, sizes and scales, built with the sanitizers on host code only."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_cpu_checks_under_sanitizers(tmp_path):
    from kronecker_factored_structured_amd import build as B
    rt = B.sanitizer_runtime()
    if not rt:
        pytest.skip("no AddressSanitizer runtime in this toolchain")
    env = dict(os.environ, KRON_LIB_PATH=B.build(host_sanitize=True, out=str(tmp_path / "libkron_san.so")),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    env["LD_PRELOAD"] = rt + (":" + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    files = [os.path.join(ROOT, "tests", f) for f in ("test_finetune_cpu.py", "test_muon_scales_cpu.py")]
    # (-s: what a sanitizer prints as it ends the process is not lost with what pytest holds back)
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-s", "-p", "no:cacheprovider", *files], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
