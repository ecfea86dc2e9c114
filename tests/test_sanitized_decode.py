"""The host code of the decode-side operators under AddressSanitizer and
UndefinedBehaviorSanitizer: the threaded table of cosines and sines, every argument
check, the workspace sizes, and the compiled calls on top of them.

Runs the operators' CPU tests against the sanitizer variant of libtq.so in a child
process, as test_sanitized_host.py does for the packers and the C ABI."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = ["test_decode_host.py", "test_decode_limits.py"]


def _built(build_lib):
    """The sanitizer variant, from the present sources."""
    sources = [os.path.join(d, f) for d in (build_lib.CSRC, build_lib.CSRC_DECODE, build_lib.INCLUDE,
                                            build_lib.PKG) for f in os.listdir(d)
               if f.endswith((".hip", ".cpp", ".h", ".py"))]
    if os.path.exists(build_lib.SAN_LIB) and os.path.getmtime(build_lib.SAN_LIB) > max(
            map(os.path.getmtime, sources)):
        return build_lib.SAN_LIB
    return build_lib.build(sanitize=True)


@pytest.mark.slow
def test_decode_host_code_under_sanitizers():
    sys.path.insert(0, ROOT)
    from bit_mixed_precision_amd import build_lib
    lib = _built(build_lib)
    env = build_lib.sanitizer_env()
    out = subprocess.run(
        [sys.executable, "-m", "pytest", "-x", "-q", "-m", "not gpu", "-p", "no:cacheprovider",
         *(os.path.join(ROOT, "tests", t) for t in TESTS)],
        env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    tail = out.stdout[-3000:] + out.stderr[-3000:]
    assert out.returncode == 0, tail
    assert "passed" in out.stdout and "ERROR: AddressSanitizer" not in out.stderr, tail
    assert "runtime error" not in out.stderr, tail  # UBSan reports
    probe = subprocess.run(
        [sys.executable, "-c", "import bit_mixed_precision_amd.binding as b; print(b._LIB_PATH)"],
        env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert probe.stdout.strip() == lib, probe.stdout + probe.stderr
