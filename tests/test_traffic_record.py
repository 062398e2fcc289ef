"""The benchmark's record of measured memory traffic belongs to the sources that the
scoring kernels are compiled from (CPU only)."""

import json
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402


def test_the_record_is_of_todays_sources():
    """After a change to one of them it has to be taken again (its commands stand in it)."""
    record = json.load(open(bench.TRAFFIC_FILE))
    assert record["score_sources_sha256"] == bench.score_source_hash()
    assert bench.measured_traffic() == record["bytes_per_launch"] == \
        record["fetch_bytes_per_launch"] + record["write_bytes_per_launch"] > 0


def test_the_sources_are_all_there_are():
    """score.hip and every header of this directory that it reaches."""
    names, todo = set(), ["score.hip"]
    here = os.path.dirname(bench.SCORE_SOURCES[0])
    while todo:
        name = todo.pop()
        if name in names or not os.path.exists(os.path.join(here, name)):
            continue
        names.add(name)
        todo += re.findall(r'#include "(\w+\.h)"', open(os.path.join(here, name)).read())
    assert names == {os.path.basename(p) for p in bench.SCORE_SOURCES}


def test_a_change_is_seen(tmp_path, monkeypatch):
    for i in range(len(bench.SCORE_SOURCES)):
        other = tmp_path / "source"
        other.write_text(open(bench.SCORE_SOURCES[i]).read() + "\n")
        paths = list(bench.SCORE_SOURCES)
        paths[i] = str(other)
        with monkeypatch.context() as m:
            m.setattr(bench, "SCORE_SOURCES", paths)
            assert bench.measured_traffic() is None
    assert bench.measured_traffic() is not None
