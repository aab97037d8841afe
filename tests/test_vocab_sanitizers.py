"""The host code of the vocabulary-end calls (workspace sizes, limits, argument
checks) under AddressSanitizer and UBSan, run on the CPU by
tests/sanitize/vocab_checks.cpp.  Needs hipcc (the device code is compiled as
usual and never launched)."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from chunked_kl_loss_seq_amd import build as BLD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_vocabulary_calls_under_asan_and_ubsan(tmp_path):
    from test_host_sanitizers import SAN  # the sanitizers' flags, host side only

    try:
        cc = BLD.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    flags = [f for f in BLD.FLAGS if f != "-O3"] + ["-O1", "-g"] + SAN
    srcs = [os.path.join(BLD.CSRC, s) for s in BLD.SOURCES]
    srcs.append(os.path.join(ROOT, "tests", "sanitize", "vocab_checks.cpp"))

    def comp(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        x = ["-x", "hip"] if src.endswith(".cpp") else []
        r = subprocess.run([cc, *flags, *x, "-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]
        return obj

    with ThreadPoolExecutor(max_workers=min(6, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(comp, srcs))
    exe = str(tmp_path / "vocab_checks")
    r = subprocess.run([cc, f"--offload-arch={BLD.ARCH}", *SAN, *objs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), (r.stdout + r.stderr)[-4000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
