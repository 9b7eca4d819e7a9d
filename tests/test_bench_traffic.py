"""A stored DRAM-traffic figure is reported only for the sources it was taken on: the GEMM's kernel and the host
code that chooses its tiles, splits and launches."""
import json
import os
import shutil

import bench


def test_a_change_of_the_kernel_or_of_its_plans_makes_the_figure_stale(tmp_path, monkeypatch):
    sources = []
    for path in bench.gemm_sources():
        sources.append(str(tmp_path / os.path.basename(path)))
        shutil.copy(path, sources[-1])
    names = {os.path.basename(p) for p in sources}
    assert "gemm_tc.cu" in names  # gemm_tc_plan, the two-launch rule
    assert "gemm_tc.cuh" in names
    (tmp_path / "profiles").mkdir()
    (tmp_path / "profiles" / "traffic.json").write_text(json.dumps({
        "decode_bgmv": {"dram_bytes_per_launch": 5.0, "kernel_sha256_16": bench.source_hash(sources)}}))
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.traffic_from_profile(sources, "decode_bgmv") == 5.0
    for path in sources:
        with open(path) as f:
            text = f.read()
        with open(path, "w") as f:
            f.write(text + "\n")
        assert bench.traffic_from_profile(sources, "decode_bgmv") is None, path
        with open(path, "w") as f:
            f.write(text)
    assert bench.traffic_from_profile(sources, "decode_bgmv") == 5.0


def test_the_bench_goes_by_these_sources():
    for path in bench.gemm_sources():
        assert os.path.exists(path)
    with open(bench.__file__) as f:
        text = f.read()
    assert text.count("kernel_src = gemm_sources()") == 2
