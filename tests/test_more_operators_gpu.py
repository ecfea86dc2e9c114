"""The cases of perf/more_operators.py in their two forms: what the library's calls return is
what the plain form returns, by name, shape, type and value, on the first pass and on a
second one of the same state."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
pytest.importorskip("bit_mixed_precision_amd.binding")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEADS = dict(Hq=8, Hkv=2, D=64, page=16)
CASES = [
    dict(op="mask", B=3, T=37, deep=2),
    dict(op="tree", dtype="f16", B=3, T=5, lo=1, hi=300, ragged=True, deep=2, empty=1, window=0, **HEADS),
    dict(op="tree", dtype="bf16", B=2, T=40, lo=90, hi=700, ragged=False, deep=0, empty=0, window=77, **HEADS),
    dict(op="weights", dtype="f16", B=3, T=5, lo=1, hi=300, ragged=True, deep=2, empty=1, window=0, decay=1.0, **HEADS),
    dict(op="weights", dtype="bf16", B=2, T=1, lo=90, hi=700, ragged=False, deep=1, empty=0, window=0, decay=0.97,
         **HEADS),
    dict(op="select", B=4, H=3, lo=5, hi=900, budget=64, recent=8, sinks=4),
    dict(op="select", B=2, H=1, lo=3, hi=20, budget=40, recent=0, sinks=0),
    dict(op="keep", kind="path", dtype="f16", B=4, T=9, lo=10, hi=200, budget=0, groups=1, planes=4, shared=1, Hkv=2,
         D=64, page=16),
    dict(op="keep", kind="evict", dtype="bf16", B=4, T=0, lo=60, hi=200, budget=50, groups=2, planes=4, shared=1,
         Hkv=2, D=64, page=16),
]


def _cases():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _bound(name, c, state, want):
    """How far two computed outputs may be apart.  With dq, dk the largest norms of a query and a
    key, a score's magnitude is at most scale dq dk, and fp32 sums of D products in any order are
    off by (D + 4) 2^-24 of it, on either side."""
    q, k = state["q"].float(), state["k"].float()
    size = float(q.norm(dim=-1).max() * k.norm(dim=-1).max()) * c["D"] ** -0.5
    ds = 2 * (c["D"] + 4) * 2.0 ** -24 * size
    tokens = c["hi"] + c["T"]
    if name == "lse":  # log of a sum of that many terms, and the number itself rounded a few times
        return ds + (tokens + 16) * 2.0 ** -23 + 2.0 ** -20 * want.abs()
    if name == "scores":  # lse is given: each weight by its score, sums of rows, what was there before
        rows = c["T"] * c["Hq"] // c["Hkv"]
        return (ds + 2.0 ** -21 * (size + 50) + (rows + 16) * 2.0 ** -23) * want.abs() + 2.0 ** -23
    # a weight in 16 bits (half a step), the output's rounding on either side
    half = torch.finfo(want.dtype).eps / 2
    return (2 * ds + 3 * half + (tokens + 16) * 2.0 ** -23) * state["v"].float().abs().max()


@pytest.mark.parametrize("i", range(len(CASES)))
def test_both_forms_return_the_same(i):
    m, c = _cases(), CASES[i]
    results = []
    for own in (False, True):
        state = m.prepare(c, 11)
        m.own = own
        results.append([{n: x.clone() for n, x in m.run(state).items()} for _ in range(2)])
    for plain, library in zip(*results):
        assert list(plain) == list(library)
        for name, want in plain.items():
            got = library[name]
            assert got.shape == want.shape and got.dtype == want.dtype, name
            if not want.is_floating_point() or c["op"] in ("select", "keep"):
                assert torch.equal(got, want), name
                continue
            fin = torch.isfinite(want)
            assert torch.equal(got[~fin], want[~fin]), name
            err = (got - want).float().abs()[fin]
            bound = _bound(name, c, state, want.float() if name != "out" else want)
            bound = bound.expand(want.shape)[fin]
            assert torch.all(err <= bound), (name, float((err / bound).max()))
