"""The tracked counters of the prefill kernels belong to the sources as they
are: the bench line leaves out those that do not."""

import json
import os

import pytest

import bench

with open(os.path.join(bench.ROOT, "profiles", "prefill_gemm_counters.json")) as f:
    KERNELS = json.load(f)["kernels"]


@pytest.mark.parametrize("key", bench.PREFILL_SOURCES)
def test_prefill_counters_are_of_these_sources(key):
    assert KERNELS[key]["source_hash"] == bench.source_hash(bench.PREFILL_SOURCES[key])
