"""The record of DRAM bytes per launch names the sources it was taken on: every
device header that the decode kernels include has to be among them."""
import json
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "paged_kv_cache_150_gb300", "csrc")


def included(names):
    seen, todo = set(), list(names)
    while todo:
        f = todo.pop()
        if f in seen or not os.path.exists(os.path.join(CSRC, f)):
            continue
        seen.add(f)
        todo += re.findall(r'#include "([^"]+)"', open(os.path.join(CSRC, f)).read())
    return seen


def test_the_record_covers_every_device_source_of_decode():
    units = [f for f in bench.KERNEL_SOURCES if f.endswith(".cu")]
    assert {f for f in included(units) if f.endswith(".cuh")} <= set(bench.KERNEL_SOURCES)


def test_every_recorded_workload_was_taken_on_the_same_sources():
    record = json.load(open(os.path.join(bench.ROOT, "profiles", "decode_traffic.json")))
    assert len({e["source_sha"] for e in record.values()}) == 1
    for e in record.values():
        assert e["dram_bytes_per_launch"] > 0 and os.path.exists(os.path.join(bench.ROOT, e["report"]))


def test_the_record_was_taken_on_the_present_sources():
    """The benchmark reports no DRAM traffic from a record of other sources."""
    record = json.load(open(os.path.join(bench.ROOT, "profiles", "decode_traffic.json")))
    assert {e["source_sha"] for e in record.values()} == {bench.source_sha()}
