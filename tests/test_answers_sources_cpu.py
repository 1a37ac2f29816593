"""What the sources of the operators for several answers to one prompt have to
hold to, and no run can show to be broken reliably."""
import os
import re

import pytest

import token_level_early_gb300 as rv

HERE = os.path.dirname(os.path.abspath(rv.__file__))


def source(name):
    with open(os.path.join(HERE, "csrc", name)) as f:
        return f.read()


def code(name):
    return "\n".join(line.split("//")[0] for line in source(name).split("\n"))


@pytest.mark.parametrize("entry,name", [("rv_kv8_copy", "kv8_copy.cu"), ("rv_kv8_attention_shared", "kv8_shared.cuh")])
def test_status_bits_are_documented(entry, name):
    """A kernel that reports a wait that ran out does so in a bit that its entry's comment gives."""
    assert "kErrWait" in code(name) and "kErrWait = 16" in code("async.cuh")
    with open(os.path.join(os.path.dirname(HERE), "include", "rv.h")) as f:
        text = f.read()
    comment = text[:text.index("int %s(" % entry)]
    comment = " ".join(re.sub(r"\n \* ?", " ", comment[comment.rindex("/*"):]).split())
    assert "bit 4 (16)" in comment
