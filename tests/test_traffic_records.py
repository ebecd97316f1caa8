"""The DRAM bytes that bench.py reports come from committed counters, which count only while the code that
they were taken of is unchanged: a change of the shared headers makes them void without a word."""

import glob
import json
import os

import pytest

import bench

RECORDS = sorted(glob.glob(os.path.join(os.path.dirname(bench.__file__), "profiles", "traffic_*.json")))


@pytest.mark.parametrize("path", RECORDS, ids=[os.path.basename(p)[8:-5] for p in RECORDS])
def test_the_records_are_of_the_kernels_as_they_are(path):
    with open(path) as f:
        records = {k: r for k, r in json.load(f).items() if not k.startswith("_")}
    assert records
    for kernel, rec in records.items():
        fn = rec.get("kernel_fn", bench.KERNEL_OF[kernel])
        assert bench.kernel_source_digest(rec["source"], fn) == rec["kernel_sha256"], kernel
