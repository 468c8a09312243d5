"""bench.py gives a kernel's recorded DRAM traffic only while its sources are those of the capture: they have to be
all of them (no GPU needed)."""

import os
import re

import pytest

import bench


@pytest.mark.parametrize("sources", [bench.PREFILL_SOURCES, bench.DECODE_SOURCES])
def test_a_kernels_sources_are_all_that_it_includes(sources):
    csrc = os.path.join(bench.ROOT, "paged_kv_cache_317_gb300", "csrc")
    seen, left = set(), [os.path.basename(sources[0])]
    while left:
        name = left.pop()
        if name in seen or not os.path.exists(os.path.join(csrc, name)):   # (the public header declares the calls)
            continue
        seen.add(name)
        with open(os.path.join(csrc, name)) as f:
            left += re.findall(r'#include "([^"]+)"', f.read())
    assert seen == {os.path.basename(s) for s in sources}
