"""The JSON line of bench.py's default run: every key of the contract, and short enough
to be read back from the end of a log."""

import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
bench = pytest.importorskip("bench")

KERNEL = "tq1_tab_tiled_kernel<4, 2, 1, 4, false>"


def call(fmt, M, N, K, **more):
    return dict(fmt=fmt, M=M, N=N, K=K, kernel=KERNEL, us=123.456, TBps=1.234, TFLOPps=1234.56,
                bound="mfma", hbm_frac=0.1234, mfma_frac=0.1234, roof_frac=0.1234,
                of_read_ceiling=0.123, **more)


def full():
    """A line with every table as long as the default run makes it."""
    calls = [call(f, M, N, K) for f, M, N, K in bench.workload_calls()]
    small = [(n, N, K) for n, K, N in bench.SMALL_LAYER]
    totals = {f"layer_3b_m1_{f}_total": dict(us=123.456, TBps=1.234, hbm_frac=0.1234)
              for f in ("tq2", "tq1")}
    return {
        "metric": "m" * 80, "value": 0.1234, "unit": "u" * 60, "n_gpus": 1, "steps": 20,
        "warmup": 5, "ms_per_step": 1.2345, "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "f16", "data": "synthetic", "config": {"workload": "w" * 240},
        "roofline": {"kernel": KERNEL, "note": "r" * 220},
        "context": {"read_ceiling": [dict(N=28672, K=8192, bytes=60628992, us=10.509, TBps=5.769,
                                          hbm_frac=0.7211)] * 2,
                    "fp16_matmul": [dict(M=c["M"], N=c["N"], K=c["K"], us=112.156, TFLOPps=536.12,
                                         tq2_us=67.874, tq2_speedup=1.65)
                                    for c in calls if c["fmt"] == "tq2"]},
        "other_configs": {"gemv_1024": [call(f, 1, 1024, 1024, linear="w") for f in ("tq2", "tq1")],
                          "layer_3b_m1": [call(f, 1, N, K, linear=n) for n, N, K in small
                                          for f in ("tq2", "tq1")], **totals},
        "tq1_vs_tq2_same_weights": [
            dict(p=p, M=M, N=N, K=K, tq1=call("tq1", M, N, K), tq2=call("tq2", M, N, K),
                 tq1_over_tq2_time=1.369)
            for K, N in bench.SHAPES for p in bench.TQ1_PS for M in bench.TQ1_MS],
        "cpu_baseline": {"sample": "c" * 480}, "calls": calls}


def test_the_line_is_short_and_complete():
    out = full()
    before = json.dumps(out)
    line = bench.line_of(out)
    assert len(before) > 20000 and len(line) < 8000 and "\n" not in line
    assert json.dumps(out) == before  # what goes to a file stays whole
    got = json.loads(line)
    assert list(got) == list(out)
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "config",
              "higher_is_better", "scaling", "vs_baseline", "dtype", "data", "roofline",
              "cpu_baseline"):
        assert got[k] == out[k]
    assert len(got["calls"]) == len(out["calls"])
    assert all(r["us"] == 123.456 and r["roof_frac"] == 0.1234 for r in got["calls"])
    name, K, N = bench.SMALL_LAYER[0]
    assert got["other_configs"]["layer_3b_m1"][0] == dict(linear=name, N=N, K=K, tq2_us=123.456,
                                                          tq1_us=123.456)
    assert got["tq1_vs_tq2_same_weights"][0]["tq1_us"] == 123.456


def test_a_run_without_the_other_tables():
    out = {k: v for k, v in full().items()
           if k not in ("context", "other_configs", "tq1_vs_tq2_same_weights", "cpu_baseline")}
    assert list(json.loads(bench.line_of(out))) == list(out)
