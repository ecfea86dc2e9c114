"""Further GPU parity tests of tq_paged_attention; helpers, oracle and the
derivation of the bounds as in test_decode_gpu.py."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

from test_decode_gpu import check_attention, f64, paged, run_attention  # noqa: E402


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


def exact_rows(dtype, tokens, seed=0):
    """64 sequences of `tokens` slots with a page each, one head of 8 numbers: q is
    (y, 0, ..), y in dtype, all keys 0 but the last one, -(1, 0, ..): scores 0 and -y."""
    rng = np.random.default_rng(seed)
    B, t = 64, {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    size = -(-tokens // 16) * 16
    y = torch.from_numpy(rng.uniform(0.1, 3.0, B)).to(t)
    q = torch.zeros(B, 1, 8, dtype=t)
    q[:, 0, 0] = y
    k, v = torch.zeros(B, size, 1, 8, dtype=t), torch.zeros(B, size, 1, 8, dtype=t)
    k[:, tokens - 1, 0, 0] = -1
    pt = torch.arange(B, dtype=torch.int32)[:, None]
    lens = torch.full((B,), tokens, dtype=torch.int32)
    return y.double().numpy(), q, k, v, pt, lens


def truncated(x, bits):
    """x > 0 cut to so many significant bits."""
    e = np.frexp(x)[1] - bits
    return np.ldexp(np.floor(np.ldexp(x, -e)), e)


@pytest.mark.parametrize("dtype,bits,weight_bits", [("f16", 11, 22), ("bf16", 8, 16)])
def test_attention_weights_are_rounded_to_nearest(dtype, bits, weight_bits):
    """A weight w = e^-y of two 16-bit numbers is off by 2^-weight_bits of itself at
    most.  Two tokens of weight 1 carry the two leading pieces of w, cut, with the
    opposite sign, so that what is left is of the size of the error.  Besides: the
    score's product and scaling (2^-24 y each) and the fp32 exponential and sums, at
    most (3 + 16) 2^-23 of sum w |v| as in test_decode_gpu.py."""
    y, q, k, v, pt, lens = exact_rows(dtype, 3)
    w = np.exp(-y)
    first = truncated(w, bits)
    second = truncated(w - first, bits)
    at = torch.tensor([5])
    for t, x in enumerate((-first, -second, np.ones_like(w))):
        v[:, t, 0, at] = torch.from_numpy(256 * x)[:, None].to(v.dtype)
        assert np.array_equal(v[:, t, 0, 5].double().numpy(), 256 * x)  # exact in the type
    out = tq.tq_paged_attention(*(x.cuda() for x in (q, k, v, pt, lens)), scale=1.0)
    got = out[:, 0, 5].double().cpu().numpy()
    total = 2 + w
    want = 256 * (w - first - second) / total
    before = 256 / total * w * (2.0 ** -weight_bits + 2 * 2.0 ** -24 * y) \
        + 256 * 2 * w / total * (3 + 16) * 2.0 ** -23
    ulp = np.ldexp(1.0, np.frexp(np.abs(want) + before)[1] - 1 - bits)
    err = np.abs(got - want)
    assert np.all(err <= before + np.maximum(ulp, 2.0 ** -25)), float((err / before).max())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,size,n", [(64, 16, 1000), (128, 24, 300), (256, 32, 1500)])
def test_attention_many_tokens_without_weight(dtype, D, size, n):
    """One token of a small value has all the weight; the others, of weight e^-400 (0
    in fp32) and large values of one sign, leave no trace, however many they are."""
    q, k, v, pt, lens = paged(D, dtype, [n, 1, 40], 3, 1, D, size)
    q[:] = 1
    used = ~torch.isnan(k)
    k[used], v[used] = -400 / D, 6e4  # the key is exact in both types
    assert float(k[used][0]) == -400 / D
    first = pt[:, 0].long()
    k[first, 0], v[first, 0] = 0, 1e-3
    run_attention(q, k, v, pt, lens, dtype, scale=1.0)


def test_attention_infinite_values_of_small_weights():
    """An infinite value stays infinite down to weights of 2^-38 (fp16) or 2^-126
    (bf16) of the largest, also where nothing remains of the weight for its second number."""
    for dtype, exps in (("f16", (0, 1, 12, 24, 37, 38)), ("bf16", (0, 1, 24, 37, 100, 125))):
        for e in exps:
            q, k, v, pt, lens = paged(e, dtype, [20], 1, 1, 64, 16, poison=False)
            q.zero_(), k.zero_()
            q[..., 0], k[pt[0, 0].long(), 3, 0, 0] = 1, -e
            v[pt[0, 0].long(), 3, 0, 7] = float("inf")
            out = tq.tq_paged_attention(q, k, v, pt, lens, scale=float(np.log(2.0)))[0, 0]
            assert out[7] == float("inf"), (dtype, e)
            assert torch.isfinite(out[torch.arange(64) != 7]).all()


def test_single_slot_pages_in_a_turned_cache():
    """Pages of one token in a cache made as [1][pages][heads][D]: the stride between the
    slots of a page is that of the whole cache, and is never taken."""
    P, Hkv, D = 70000, 2, 128
    q, k, v, pt, lens = paged(1, "f16", [50, 7, 0], 4, Hkv, D, 1, poison=False)
    n = k.shape[0]
    big = [torch.zeros(1, P, Hkv, D, dtype=torch.float16, device="cuda") for _ in range(2)]
    for b, x in zip(big, (k, v)):
        b[0, :n] = x[:, 0]
    kt, vt = (b.transpose(0, 1) for b in big)
    assert kt.stride(1) == P * Hkv * D > 1 << 24
    want = tq.tq_paged_attention(q, k, v, pt, lens)
    assert torch.equal(tq.tq_paged_attention(q, kt, vt, pt, lens), want)
    table = torch.from_numpy(tq.tq_rope_table(64, D)).cuda()
    qkv = torch.randn(3, 4 + 2 * Hkv, D, device="cuda").half()
    pos = torch.tensor([3, 6, 0], dtype=torch.int32, device="cuda")
    assert torch.equal(tq.tq_rope_append(qkv, table, pos, pt, kt, vt),
                       tq.tq_rope_append(qkv, table, pos, pt, k, v))
    assert torch.equal(kt[:n], k) and torch.equal(vt[:n], v)


def check_on_gpu(q, k, v, pt, lens, dtype):
    """Every row and head against fp64 on the GPU (products of matrix and vector), for
    caches over which the oracle's loops would take minutes."""
    size, Hkv, D = k.shape[1:]
    G = q.shape[1] // Hkv
    out, lse = tq.tq_paged_attention(q, k, v, pt, lens, return_lse=True)
    for b, n in enumerate(lens.tolist()):
        if n == 0:
            assert torch.all(out[b] == 0) and torch.all(lse[b] == -float("inf"))
            continue
        ids = pt[b, :-(-n // size)].long()
        for h in range(Hkv):
            kk, vv = (x[ids, :, h].flatten(0, 1)[:n].double() for x in (k, v))
            vt = vv.t().contiguous()
            for g in range(G):
                qh = q[b, h * G + g].double()
                s = kk @ qh / D ** 0.5
                w = torch.softmax(s, 0)
                ref = (f64(vt @ w)[None, None], f64(torch.logsumexp(s, 0))[None, None],
                       np.array([[float((kk.abs() @ qh.abs()).max()) / D ** 0.5]]),
                       f64(vt.abs() @ w)[None, None])
                at = slice(h * G + g, h * G + g + 1)
                check_attention(out[b:b + 1, at], lse[b:b + 1, at], ref, dtype, D, n)
    again = tq.tq_paged_attention(q, k, v, pt, lens)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype,D,size,shift", [
    ("f16", 128, 16, 0), ("bf16", 128, 64, 0),  # whole lines: half of the waves work
    ("f16", 128, 16, 8),                        # lines shared between heads
    ("f16", 120, 16, 0), ("bf16", 104, 32, 0), ("f16", 128, 24, 0), ("f16", 256, 16, 0)])
def test_attention_many_tiles_a_wave(dtype, D, size, shift):
    """More than 12 tiles for every wave of the GPU, in rows that begin and end anywhere."""
    q, k, v, pt, lens = paged(21, dtype, [60001, 0, 41000, 3, 33, 7000], 8, 8, D, size,
                              poison=False)
    if shift:
        k, v = (torch.cat([torch.zeros(shift, dtype=x.dtype, device="cuda"), x.flatten()])
                [shift:].view(x.shape) for x in (k, v))
        assert k.data_ptr() % 128 == 2 * shift
    check_on_gpu(q, k, v, pt, lens, dtype)
