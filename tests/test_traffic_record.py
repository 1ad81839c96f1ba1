"""The committed record of the bf16 kernel's DRAM traffic belongs to the sources in the tree (no GPU)."""
import json
import os
import re

import bench
from speculative_decode_mla_gb300 import _build


def included(name, seen):
    """The file and what it includes from this tree, by file name."""
    path = next(p for p in (os.path.join(_build.CSRC, name), os.path.join(_build.INCLUDE, name)) if os.path.exists(p))
    seen.add(name)
    with open(path) as f:
        for n in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
            if n not in seen:
                included(n, seen)
    return seen


def test_the_record_is_keyed_by_what_the_kernel_is_built_from():
    assert set(bench.TC_SOURCES) == included("verify_tc.cu", set())


def test_the_record_is_current():
    with open(os.path.join(_build.ROOT, "profiles", "traffic.json")) as f:
        d = json.load(f)
    assert d["fingerprint"] == _build.source_fingerprint(bench.TC_SOURCES)
    assert bench.traffic_record(d["fingerprint"]) == d["dram_bytes_per_launch"] == d["dram_bytes_read"] + d["dram_bytes_write"]


def test_a_key_changes_with_a_source_and_not_with_other_headers(tmp_path, monkeypatch):
    key = _build.source_fingerprint(bench.TC_SOURCES)
    for d in ("CSRC", "INCLUDE"):
        for n in os.listdir(getattr(_build, d)):
            with open(os.path.join(getattr(_build, d), n), "rb") as f:
                (tmp_path / d).mkdir(exist_ok=True)
                (tmp_path / d / n).write_bytes(f.read())
        monkeypatch.setattr(_build, d, str(tmp_path / d))
    assert _build.source_fingerprint(bench.TC_SOURCES) == key
    (tmp_path / "INCLUDE" / "mla_kv4.h").write_text("// other\n")
    assert _build.source_fingerprint(bench.TC_SOURCES) == key
    for n in bench.TC_SOURCES:
        at = tmp_path / ("INCLUDE" if (tmp_path / "INCLUDE" / n).exists() else "CSRC") / n
        text = at.read_text()
        at.write_text(text + "\n")
        assert _build.source_fingerprint(bench.TC_SOURCES) != key, n
        at.write_text(text)
