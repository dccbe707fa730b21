"""bench.py reports a kernel's captured DRAM traffic only while the sources it was captured on are unchanged:
the files that it hashes have to be the kernel's own, with everything of the library that they include."""

import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "paged_kv_attention_slot_gb300", "csrc")


@pytest.mark.parametrize("sources, kernel", [(bench.DECODE_SOURCES, "decode_kernel"), (bench.PREFILL_SOURCES, "prefill_kernel")])
def test_hashed_sources_hold_the_kernel_and_its_includes(sources, kernel):
    text = {n: open(os.path.join(CSRC, n), encoding="utf-8").read() for n in sources}
    assert any(re.search(r"__global__[^;{]*\b" + kernel + r"\(", t) for t in text.values())
    for name, t in text.items():
        for inc in re.findall(r'#include "([^"]+)"', t):
            if os.path.exists(os.path.join(CSRC, inc)):  # (the public header is not under csrc)
                assert inc in sources, (name, inc)
