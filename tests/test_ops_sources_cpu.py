"""Rules of the sources that no run can show to be broken reliably."""
import os

import pytest

import token_level_early_gb300 as rv

CSRC = os.path.join(os.path.dirname(os.path.abspath(rv.__file__)), "csrc")


@pytest.mark.parametrize("name", ["ops.cuh", "rope.cu", "kv8.cu", "kv8_attention.cuh", "kv8_attention.cu", "kv8_attention_e4m3.cu", "rows_mma.cu"])
def test_no_read_only_loads_in_chained_kernels(name):
    """These kernels are launched before their predecessor in the stream has
    ended: the read-only path is for memory that no one writes while a kernel
    lives.  A load hoisted above the wait, or served from a line of before,
    would give old positions or old codes."""
    with open(os.path.join(CSRC, name)) as f:
        code = [line.split("//")[0] for line in f]
    text = "".join(code)
    assert "pdl" in text or name.endswith("e4m3.cu") or name == "ops.cuh"
    for word in ("__ldg(", "ld.global.nc", "ld.const", "__restrict__"):
        assert word not in text, word
