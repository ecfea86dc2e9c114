"""The example that decodes with drafted trees, end to end: paths, appending at slots,
attention, the accepted path, and the cache kept short."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
pytest.importorskip("bit_mixed_precision_amd.binding")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("decode_drafts",
                                                  os.path.join(ROOT, "examples", "decode_drafts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("requests,prompt,steps", [(2, 21, 40), (1, 1, 30), (2, 40, 5)])
def test_drafted_decoding(requests, prompt, steps):
    ex = _example()
    out = ex.main(["--requests", str(requests), "--prompt", str(prompt), "--steps", str(steps), "--check"])
    # as in test_decode_example_gpu.py
    assert out["error"] <= 2.0 ** -6 * out["scale"]
    cache = out["cache"]
    assert int(cache.refused) == 0
    # every token but the newest is cached, in pages of the row's own
    assert cache.lens.tolist() == cache.at.tolist() == [len(h) - 1 for h in out["history"]]
    for row, n in zip(cache.pages.tolist(), cache.lens.tolist()):
        held = -(-n // ex.PAGE)
        assert min(row[:held]) >= 0 and set(row[held:]) <= {-1}
    assert all(steps <= len(h) - len(p) <= steps + ex.BRANCH for h, p in zip(out["history"], out["prompts"]))


@pytest.mark.parametrize("budget", [16, 33])
def test_drafted_decoding_with_a_short_cache(budget):
    ex = _example()
    out = ex.main(["--prompt", "30", "--steps", "40", "--budget", str(budget)])
    cache = out["cache"]
    assert int(cache.refused) == 0 and cache.lens.tolist() == [budget] * 2
    assert cache.at.tolist() == [len(h) - 1 for h in out["history"]]
    s = cache.scores[..., :budget]
    assert torch.isfinite(out["logits"]).all() and torch.isfinite(s).all() and (s >= 0).all()
    # a budget that nothing exceeds changes nothing
    whole = ex.decode(ex.Model(0), out["prompts"], 20)
    again = ex.decode(ex.Model(0), out["prompts"], 20, budget=200)
    assert whole["history"] == again["history"] and torch.equal(whole["logits"], again["logits"])
