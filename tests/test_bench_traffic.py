"""The committed DRAM traffic of a kernel counts as long as the sources that it was taken on: all of them."""
import json
import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "vision_language_model_b200", "csrc")


def _reached(name, seen):
    """name and the headers beside it that it includes, and theirs."""
    if name in seen or not os.path.exists(os.path.join(CSRC, name)):
        return seen
    seen.add(name)
    with open(os.path.join(CSRC, name)) as fh:
        for inc in re.findall(r'^#include "([^"/]+)"', fh.read(), re.M):
            _reached(inc, seen)
    return seen


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_every_source_of_a_kernel_voids_its_traffic(kernel):
    sources = bench.KERNEL_SOURCES[kernel]
    assert set(sources) == _reached(sources[0], set())
    with open(os.path.join(bench.ROOT, "profiles", "traffic_per_launch.json")) as fh:
        entry = json.load(fh)[kernel]
    assert sorted(entry["sources"]) == sorted(sources)
