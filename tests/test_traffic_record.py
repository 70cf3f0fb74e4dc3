"""The recorded DRAM traffic that the bench reports: the figures are the kept capture's, and the
hash that they are keyed to covers the sources of the workload's own kernels alone."""

import csv
import json
import os
import re

import pytest

import bench

PROFILES = os.path.join(bench.ROOT, "profiles")
CSRC = os.path.join(bench.ROOT, "speculative_decoding_verification_05_gb300", "csrc")
RECORD = json.load(open(os.path.join(PROFILES, "traffic.json")))


@pytest.mark.parametrize("workload", RECORD)
def test_figures_are_the_captures(workload):
    with open(os.path.join(PROFILES, "traffic_capture.csv")) as f:
        rows = [r for r in csv.DictReader(f) if r["workload"] == workload]
    e = RECORD[workload]
    moved = sum(int(r["dram_bytes_read"]) + int(r["dram_bytes_written"]) for r in rows)
    assert e["bytes_per_launch"] * int(rows[0]["steps"]) == moved * e["stacked"]
    assert e["ratio_to_algorithmic"] == round(moved / int(rows[0]["algorithmic_bytes_of_the_call"]), 4)
    assert e["kernel"].split(" + ") == [r["kernel"] for r in rows]


@pytest.mark.parametrize("workload", RECORD)
def test_sources_hold_the_kernels(workload):
    e = RECORD[workload]
    files = bench.kernel_sources(workload)
    assert e["sources"] == files
    text = "".join(open(os.path.join(CSRC, f)).read() for f in files)
    for k in e["kernel"].split(" + "):
        assert re.search(r"\b" + k.split("<")[0] + r"\(const __grid_constant__", text), k


def test_other_sources_leave_the_hash(tmp_path, monkeypatch):
    """A change of another kernel's file does not touch a workload's hash; one of its own, or of a
    header that it includes, does, and the figure is then no longer reported."""
    pkg = tmp_path / "speculative_decoding_verification_05_gb300" / "csrc"
    pkg.mkdir(parents=True)
    for f in os.listdir(CSRC):
        (pkg / f).write_bytes(open(os.path.join(CSRC, f), "rb").read())
    (tmp_path / "profiles").mkdir()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    for w in RECORD:
        record = {w: {**RECORD[w], "sources_sha16": bench.kernel_sources_sha(w)}}
        (tmp_path / "profiles" / "traffic.json").write_text(json.dumps(record))
        assert bench.recorded_traffic(w, RECORD[w]["stacked"]) == RECORD[w]["bytes_per_launch"]
        assert bench.recorded_traffic(w, RECORD[w]["stacked"] + 1) is None
        for f in ("evict.cu", "weigh.cuh", "attention_tc.cu"):
            (pkg / f).write_bytes((pkg / f).read_bytes() + b"\n")
        assert bench.recorded_traffic(w, RECORD[w]["stacked"]) is not None
        for f in bench.kernel_sources(w):
            was = (pkg / f).read_bytes()
            (pkg / f).write_bytes(was + b"\n")
            assert bench.recorded_traffic(w, RECORD[w]["stacked"]) is None, f
            (pkg / f).write_bytes(was)
