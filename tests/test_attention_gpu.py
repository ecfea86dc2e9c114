"""Further GPU parity tests of tq_paged_attention; helpers, oracle and the
derivation of the bounds as in test_decode_gpu.py."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

from test_decode_gpu import paged, run_attention  # noqa: E402


@pytest.mark.parametrize("dtype,B,Hq,Hkv,D,longest", [
    ("f16", 4, 8, 8, 128, 512), ("bf16", 16, 64, 8, 128, 300), ("f16", 200, 8, 8, 64, 97),
    ("bf16", 30, 6, 3, 256, 200), ("f16", 1, 40, 1, 80, 33)])
def test_attention_own_workgroups_repeat(dtype, B, Hq, Hkv, D, longest):
    """Rows with a workgroup each: every wave's part is in every answer, and the bits
    are the same on every call and on another stream."""
    lens = np.random.default_rng(D + B).integers(0, longest + 1, B)
    lens[0] = longest
    q, k, v, pt, lens = paged(B, dtype, lens, Hq, Hkv, D, 16)
    pt = pt[:, :-(-longest // 16)].contiguous()
    assert tq.tq_paged_attention_workspace(B, Hq, Hkv, D, 16, pt.shape[1]) == 0
    want, lw = run_attention(q, k, v, pt, lens, dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(20):
        stream = {"stream": side.cuda_stream} if i % 2 else {}
        out, lse = tq.tq_paged_attention(q, k, v, pt, lens, return_lse=True, **stream)
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, lw), i
