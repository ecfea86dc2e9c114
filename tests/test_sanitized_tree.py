"""The host code of the operators on drafted trees and kept caches under AddressSanitizer
and UndefinedBehaviorSanitizer: their argument checks, workspace sizes and compiled
calls, as test_sanitized_decode.py does for the operators before them."""

import os
import subprocess
import sys

import pytest

from test_sanitized_decode import ROOT, _built


@pytest.mark.slow
def test_tree_host_code_under_sanitizers():
    sys.path.insert(0, ROOT)
    from bit_mixed_precision_amd import build_lib
    _built(build_lib)
    out = subprocess.run(
        [sys.executable, "-m", "pytest", "-x", "-q", "-m", "not gpu", "-p", "no:cacheprovider",
         os.path.join(ROOT, "tests", "test_tree_limits.py")],
        env=build_lib.sanitizer_env(), cwd=ROOT, capture_output=True, text=True, timeout=900)
    tail = out.stdout[-3000:] + out.stderr[-3000:]
    assert out.returncode == 0, tail
    assert "passed" in out.stdout and "ERROR: AddressSanitizer" not in out.stderr, tail
    assert "runtime error" not in out.stderr, tail
