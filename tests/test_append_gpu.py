"""tq_rope_append at the sizes of prompts: thousands of tokens of a few sequences."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

from oracle import rope_frequencies_ref  # noqa: E402
from test_decode_gpu import DT, check_rope, i32, randn  # noqa: E402


@pytest.mark.parametrize("dtype,interleaved,T,Hq,Hkv,D,rot,size,order", [
    ("f16", False, 4099, 64, 8, 128, 128, 16, "tokens"),   # two heads a thread
    ("bf16", True, 60000, 5, 2, 64, 64, 24, "heads"),      # the same, an odd number of heads
    ("f16", True, 30011, 6, 3, 80, 40, 1, "tokens"),       # vectors of 4
    ("bf16", False, 2500, 4, 2, 36, 12, 16, "tokens"),     # single numbers
])
def test_append_prompts(dtype, interleaved, T, Hq, Hkv, D, rot, size, order):
    rng = np.random.default_rng(T)
    ends = np.sort(rng.permutation(T - 1)[:3] + 1)  # four prompts, packed
    seq = np.searchsorted(ends, np.arange(T), side="right")
    lens = np.bincount(seq, minlength=4)
    start = [0, 7, size, 3 * size - 1]              # where each goes on
    pos = np.concatenate([s + np.arange(n) for s, n in zip(start, lens)])
    n_pos = int(pos.max()) + 1
    need = -(-(np.array(start) + lens) // size)
    P = int(need.sum()) + 5
    pt = np.full((4, int(need.max())), -1, np.int32)
    pt[np.arange(pt.shape[1])[None] < need[:, None]] = rng.permutation(P)[:need.sum()]
    shape = (P, size, Hkv, D) if order == "tokens" else (P, Hkv, size, D)
    kv, vv = (x if order == "tokens" else x.transpose(1, 2)
              for x in (randn(s, dtype, *shape) for s in (1, 2)))
    k0, v0 = kv.clone(), vv.clone()
    qkv = randn(3, dtype, T, Hq + 2 * Hkv, D)
    table = torch.from_numpy(tq.tq_rope_table(n_pos, rot, 1e4)).cuda()
    Q = tq.tq_rope_append(qkv, table, i32(pos), i32(pt), kv, vv, interleaved=interleaved,
                          seqs=i32(seq))
    assert Q.dtype == DT[dtype] and Q.shape == (T, Hq, D)
    # a sample against fp64, and all of it against the bits of tq_rope
    at = np.unique(np.concatenate([rng.integers(0, T, 60), ends - 1, ends, [0, T - 1]]))
    on = torch.as_tensor(at).cuda()
    freq = rope_frequencies_ref(rot, 1e4)
    check_rope(Q[on], qkv[on][:, :Hq], i32(pos[at]), freq, dtype, interleaved, False)
    turned = tq.tq_rope(qkv[:, :Hq + Hkv], table, i32(pos), interleaved=interleaved)
    assert torch.equal(Q, turned[:, :Hq])
    page, slot = (torch.as_tensor(x).cuda().long() for x in (pt[seq, pos // size], pos % size))
    assert torch.equal(kv[page, slot], turned[:, Hq:])
    assert torch.equal(vv[page, slot], qkv[:, Hq + Hkv:])
    # every other slot is as it was
    k0[page, slot], v0[page, slot] = kv[page, slot], vv[page, slot]
    assert torch.equal(kv, k0) and torch.equal(vv, v0)
