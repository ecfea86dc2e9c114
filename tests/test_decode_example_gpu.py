"""The beam-decoding example end to end: products, rotary positions, paged cache,
attention, fork, grow and compact together, against fp64 without a cache."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
pytest.importorskip("bit_mixed_precision_amd.binding")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("decode_beams",
                                                  os.path.join(ROOT, "examples", "decode_beams.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("requests,beams,prompt,steps", [(2, 4, 21, 24), (1, 1, 1, 3), (5, 3, 16, 17),
                                                         (1, 16, 40, 9)])
def test_beam_decoding(requests, beams, prompt, steps):
    out = _example().main(["--requests", str(requests), "--beams", str(beams), "--prompt",
                           str(prompt), "--steps", str(steps), "--check"])
    # activations are rounded to fp16 some ten times on the way (2^-11 each) and the
    # residual stream doubles what a layer adds: 2^-6 of the largest logit is ample
    # for rounding and far below any wrong token, position, page or weight
    assert out["error"] <= 2.0 ** -6 * out["scale"]
    assert int(out["refused"]) == 0
    rows = requests * beams
    assert out["lens"].tolist() == [prompt + steps] * rows
    held = -(-(prompt + steps) // 16)
    pages = out["pages"][:, :held]
    assert int(out["used"]) == len(torch.unique(pages)) <= rows * held
    assert int(pages.max()) == int(out["used"]) - 1 and int(pages.min()) == 0
