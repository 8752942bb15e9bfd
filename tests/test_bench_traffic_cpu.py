"""The guard of the committed HBM counters: bench.py reports them for the sources that they were measured on."""
import json
import os
import re
import shutil

import pytest

import bench


def changed(tmp_path, name):
    """The hash with one more line in this source of a copy, and without."""
    csrc = tmp_path / "csrc"
    if not csrc.exists():
        shutil.copytree(bench.CSRC, csrc)
    before = bench.src_hash(str(csrc))
    with open(csrc / name, "a") as fh:
        fh.write("// one more line\n")
    return before, bench.src_hash(str(csrc))


def test_hash_covers_the_units_of_the_counted_launches_and_their_headers():
    """Every local header that a listed file includes is listed too."""
    listed = set(bench.GEMM_SRCS)
    for name in listed:
        with open(os.path.join(bench.CSRC, name)) as fh:
            for inc in re.findall(r'#include "([^"]+)"', fh.read()):
                assert inc in listed or not os.path.exists(os.path.join(bench.CSRC, inc)), (name, inc)


@pytest.mark.parametrize("name", ["mx.hpp", "moe_common.hpp", "gemm_kernel.hpp", "gemm_rows.hip", "gemm_wgrad.hip"])
def test_hash_changes_with_what_the_counted_launches_are_compiled_from(tmp_path, name):
    before, after = changed(tmp_path, name)
    assert before == bench.src_hash() and after != before


@pytest.mark.parametrize("name", ["gemm4.hip", "mx.hip", "gemm_swiglu8.hip", "gemm_dgrad8.hip", "route.hip"])
def test_hash_stays_with_other_sources(tmp_path, name):
    before, after = changed(tmp_path, name)
    assert after == before


def test_counters_of_other_sources_are_refused(tmp_path, monkeypatch):
    rec = {"gemm_src_sha": bench.src_hash(), "traffic_bytes_per_launch": 123}
    path = tmp_path / "traffic.json"
    path.write_text(json.dumps({"expert_up@tiny": rec, "expert_down@tiny": dict(rec, gemm_src_sha="0" * 16)}))
    monkeypatch.setattr(bench, "TRAFFIC_FILE", str(path))
    assert bench.measured_traffic("expert_up", "tiny") == 123
    assert bench.measured_traffic("expert_down", "tiny") is None and bench.measured_traffic("other", "tiny") is None
