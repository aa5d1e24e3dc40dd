"""Every kernel is launched so that it may start while the kernel before it still runs, and what that one
writes (lengths, positions, uniforms, page tables, rows) must not change while a kernel holds it on the
read-only path: no kernel source reads global memory that way."""
import os
import re

import pytest

import block_masked_window_b200 as bmw

CSRC = os.path.join(os.path.dirname(bmw.library_path()), "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


@pytest.mark.parametrize("name", SOURCES)
def test_no_read_only_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert re.findall(r"__ldg\w*\(|ld\.global(?:\.\w+)*\.nc\b", code) == []


def test_sources_are_found():
    assert {"attn_tc.cu", "rope.cu", "kv_evict.cu", "verify.cu", "pbd_common.cuh"} <= set(SOURCES)
