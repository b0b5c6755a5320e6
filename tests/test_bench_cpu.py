"""Host-side checks of bench.py (CPU only): the reference arm's JSON line
(it times the oracle, so it runs without a GPU) and the rule that a
recorded DRAM traffic figure is reported only for the sources it was
captured on."""
import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402


def test_reference_arm_prints_the_contract_line():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--impl", "reference", "--steps", "2",
                          "--warmup", "3", "--quiet"], capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert out.returncode == 0, out.stderr[-2000:]
    lines = [l for l in out.stdout.splitlines() if l.strip()]
    assert len(lines) == 1
    d = json.loads(lines[0])
    assert d["impl"] == "reference" and d["metric"] == bench.METRIC and d["unit"] == "tokens/s"
    assert d["steps"] == 2 and d["warmup"] == 3 and d["higher_is_better"] is True and d["value"] > 0
    assert d["cpu_baseline"]["kind"] == "oracle" and d["cpu_baseline"]["value"] == d["value"]
    assert d["cpu_baseline"]["cores"] >= 1 and d["cpu_baseline"]["sample"]
    assert d["e2e"] == {"value": d["value"], "unit": d["unit"], "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0}
    assert d["config"]["workload"] == bench.WORKLOAD


def test_traffic_only_for_the_captured_sources(monkeypatch):
    sha = bench.sources_sha("decode")
    monkeypatch.setitem(bench.TRAFFIC, "probe_key", {"bytes": 1000, "alg": 800, "sha": sha, "how": "test"})
    b, note = bench.traffic_of("probe_key", "decode", 1600)
    assert b == 2000 and "scaled" in note  # the recorded ratio times the leg's algorithmic bytes
    b, _ = bench.traffic_of("probe_key", "decode")
    assert b == 1000
    monkeypatch.setitem(bench.TRAFFIC, "probe_key", {"bytes": 1000, "alg": 800, "sha": "0" * 16, "how": "test"})
    b, note = bench.traffic_of("probe_key", "decode", 1600)
    assert b is None and note.startswith("stale")
    b, note = bench.traffic_of("no_such_key", "decode", 1600)
    assert b is None and "not captured" in note


def test_throughput_and_peaks():
    assert bench.job_throughput(100, 4, 10.0) == 100 * 4 / 0.010
    peak, kind = bench.hbm_peak()
    assert peak > 1000 and kind in ("measured", "fallback")
    alu, akind = bench.alu_peak()
    assert abs(alu - 148 * 128 * 1965e6 / 1e12) < 1.0 and akind.startswith("derived")


def test_result_line_stays_short_with_every_leg():
    """The line carries the contract's keys unchanged and each leg's figures in under 3600 characters; the legs' records
    go to stderr whole."""
    leg = {"metric": bench.METRIC, "value": 45577.18839066676, "unit": "tokens/s", "n_gpus": 1, "steps": 20, "warmup": 5,
           "ms_per_step": 0.021940800000000003, "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
           "dtype": bench.DTYPE_W4, "data": "synthetic", "config": {"workload": "w" * 500},
           "roofline": {"bound": "hbm", "frac": 0.17330865452654687, "how": "r" * 400},
           "e2e": {"value": 13165697019.755371, "unit": "tokens/s", "h2d_bytes_per_step": 134217728, "d2h_bytes_per_step": 33},
           "gpu_launches": 20, "clocks": {"sm_mhz": 1965.0, "sm_max_mhz": 1965.0, "reasons": [], "samples": 3},
           "cpu_baseline": {"value": 2.35, "unit": "tokens/s", "cores": 16, "kind": "oracle", "sample": "s" * 250}}
    names = [f"decode_stream_T{i}" for i in range(12)]
    out = {**leg, "legs": {n: dict(leg) for n in names}, "gpu_launches_all_legs": 260}
    line, records = bench.result_lines(out)
    assert len(line) < 3600 and "\n" not in line
    d = json.loads(line)
    for k in leg:
        assert d[k] == leg[k], k
    assert list(d["legs"]) == names and d["gpu_launches_all_legs"] == 260
    assert d["legs"][names[0]] == {"value": 45577.0, "unit": "tokens/s", "e2e": 13166000000.0, "frac": 0.17331}
    assert [json.loads(r.split(": ", 1)[1]) for r in records] == [leg] * 12
    assert bench.result_lines(leg) == (json.dumps(leg), [])
