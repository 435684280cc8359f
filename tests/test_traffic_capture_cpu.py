"""The DRAM figures that bench.py reports belong to the sources they were captured on."""
import json
import os

import bench

PATH = os.path.join(bench.ROOT, "profiles", "traffic.json")


def test_the_file_names_one_set_of_sources():
    with open(PATH) as f:
        d = json.load(f)
    assert set(d) == {"source_hash", "commands", "note", "kernels"}
    assert len(d["source_hash"]) == 16


def test_figures_of_other_sources_are_not_reported(monkeypatch):
    with open(PATH) as f:
        d = json.load(f)
    monkeypatch.setattr(bench, "source_hash", lambda: d["source_hash"])
    assert all(bench.ncu_traffic(k) == v["dram_bytes_per_launch"] for k, v in d["kernels"].items())
    monkeypatch.setattr(bench, "source_hash", lambda: "0" * 16)
    assert all(bench.ncu_traffic(k) is None for k in d["kernels"])
