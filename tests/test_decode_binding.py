"""The binding of the decode-side calls on the CPU: what it needs to be imported, and
that its compiled and its Python form take and refuse the same arguments."""

import os
import subprocess
import sys

import numpy as np
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


FLAGS = [2, -1, None, "yes", [1], 0.5, 1 << 70, torch.ones(2)]


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def test_flags(device):
    """interleaved and inverse: a bool, or 0 or 1, in both forms of a call; on the CPU
    the refusal of the flag comes before that of the device."""
    h = dict(dtype=torch.float16, device=device)
    i = dict(dtype=torch.int32, device=device)
    X, pos = torch.ones(3, 8, 16, **h), torch.ones(3, **i)
    table = torch.from_numpy(tq.tq_rope_table(8, 16)).to(device)
    k, pt = torch.zeros(5, 16, 2, 16, **h), torch.zeros(3, 4, **i)
    forms = [{}] if device == "cpu" else [{}, {"stream": torch.cuda.current_stream().cuda_stream}]
    calls = [lambda f, kw: tq.tq_rope(X, table, pos, interleaved=f, **kw),
             lambda f, kw: tq.tq_rope(X, table, pos, inverse=f, **kw),
             lambda f, kw: tq.tq_rope_append(X, table, pos, pt, k, k.clone(), f, **kw)]
    for call in calls:
        for kw in forms:
            for bad in FLAGS:
                with pytest.raises(tq.TQError) as e:
                    call(bad, kw)
                assert e.value.status == tq.TQ_ERR_VALUE, bad
        if device == "cuda":
            for value in (False, True):
                want = call(value, {})
                for same in (int(value), np.bool_(value), float(value), torch.tensor(value)):
                    for kw in forms:
                        assert torch.equal(call(same, kw), want)


def test_arguments_that_are_no_tensors():
    """Every tensor argument in turn replaced by None, an array and a list: TQError, not
    whatever the first attribute access gives."""
    h, i = dict(dtype=torch.float16), dict(dtype=torch.int32)
    x, pos, pt = torch.zeros(3, 8, 16, **h), torch.zeros(3, **i), torch.zeros(3, 4, **i)
    table, k = torch.zeros(8, 8, 2), torch.zeros(5, 16, 2, 16, **h)
    pool = torch.zeros(2, 5, 16, 16, **h)
    calls = [(tq.tq_rope, (x, table, pos)), (tq.tq_rope_append, (x, table, pos, pt, k, k)),
             (tq.tq_paged_attention, (x, k, k, pt, pos)), (tq.tq_pages_fork, (pool, pt, pos, pos)),
             (tq.tq_pages_grow, (pt, pos, pos)), (tq.tq_pages_compact, (pool, pt, pos)),
             (tq.tq_pages_copy, (pool, pos, pos))]
    rest = {tq.tq_pages_fork: (16,), tq.tq_pages_grow: (5, 16), tq.tq_pages_compact: (16,)}
    for fn, args in calls:
        for n in range(len(args)):
            for bad in (None, np.zeros((3, 4), np.int32), [1, 2]):
                with pytest.raises(tq.TQError) as e:
                    fn(*args[:n], bad, *args[n + 1:], *rest.get(fn, ()))
                assert e.value.status in (tq.TQ_ERR_VALUE, tq.TQ_ERR_SHAPE), (fn, n)
