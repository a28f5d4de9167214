"""The committed counter records name the sources they were taken from by a hash, and
the bench leaves out a record whose sources have changed since.  So a change to one of
these files, a comment or a declaration too, ends either with the counters taken again
or, where the kernel's instructions are shown to be the same, with its new hash."""
import importlib.util
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bench():
    spec = importlib.util.spec_from_file_location("bench_records", os.path.join(ROOT, "bench.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def records():
    return json.load(open(os.path.join(ROOT, "profiles", "traffic.json")))


@pytest.mark.parametrize("kernel", sorted(records()))
def test_record_is_of_the_current_sources(bench, kernel):
    rec = records()[kernel]
    assert bench.traffic_for(kernel, rec["workload"]) == rec["bytes_per_launch"] > 0
    assert bench.traffic_for(kernel, "another workload") is None
