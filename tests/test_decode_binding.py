"""The binding of the decode-side calls on the CPU: what it needs to be imported, and
that its compiled and its Python form take and refuse the same arguments."""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = r"""
import sys, types, warnings
sys.modules["bit_mixed_precision_amd._tq_torch"] = {stand_in}
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    import bit_mixed_precision_amd.binding as tq
assert any("_tq_torch.so" in str(w.message) for w in said), [str(w.message) for w in said]
import numpy as np, torch
W = np.random.default_rng(0).normal(size=(16, 256)).astype(np.float32)
qs, scales, gamma = tq.tq_pack_tq2(W)
assert np.array_equal(tq.tq_unpack_tq2(qs, 256), tq.tq_ternarize_f32(W)[0])
assert tq.tq_rope_table(4, 8).shape == (4, 4, 2)
x, pos = torch.zeros(3, 4, 16, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
k, pool = torch.zeros(5, 16, 2, 16, dtype=torch.float16), torch.zeros(2, 5, 16, 16)
pt = torch.zeros(3, 4, dtype=torch.int32)
for call in (lambda: tq.tq_rope(x, torch.zeros(8, 8, 2), pos),
             lambda: tq.tq_rope_append(torch.cat([x, x], 1), torch.zeros(8, 8, 2), pos, pt, k, k),
             lambda: tq.tq_paged_attention(x, k, k, pt, pos),
             lambda: tq.tq_pages_fork(pool, pt, pos, pos, 16),
             lambda: tq.tq_pages_grow(pt, pos, pos, 5, 16),
             lambda: tq.tq_pages_compact(pool, pt, pos, 16)):
    try:
        call()
    except tq.TQError as e:
        assert e.status == tq.TQ_ERR_DEVICE, e
    else:
        raise AssertionError("a CPU tensor was taken")
print("fine")
"""


@pytest.mark.parametrize("stand_in", [
    "None",  # importing it raises ImportError
    "types.SimpleNamespace(torch_version='1.0')",  # built for another torch
    "types.SimpleNamespace()"])
def test_import_without_the_compiled_calls(stand_in):
    """The packers, the products and the decode-side calls do not need _tq_torch.so."""
    out = subprocess.run([sys.executable, "-c", WITHOUT.format(stand_in=stand_in)], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "fine", out.stderr[-3000:]


def test_the_compiled_calls_are_there():
    assert tq._fast.torch_version == torch.__version__


def test_build_without_headers(monkeypatch, tmp_path):
    """Without Python's headers there is no call to compile _tq_torch.so."""
    import sysconfig

    from bit_mixed_precision_amd import build_lib
    assert build_lib._torch_ext_cmd("x.so")[0] == "g++"
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(sysconfig, "get_paths", lambda: paths)
    assert build_lib._torch_ext_cmd("x.so") is None
