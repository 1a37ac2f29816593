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


def body(text, name):
    """A function's text between its outermost braces."""
    at = text.index("{", text.index(name + "("))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(name)


@pytest.mark.parametrize("kernel", ["k_attn8", "k_attn8_join"])
def test_the_kernel_before_the_prefix_waits_first(kernel):
    """k_prefix begins without a wait: every block of the kernel before it has to have waited
    before it lets a successor start, and before it may leave."""
    text = body(code("kv8_attention.cuh"), " " + kernel)
    wait = text.index("pdl_wait()")
    assert "pdl_trigger()" in text[wait:]
    for word in ("pdl_trigger", "return", "if ("):
        assert word not in text[:wait], word


def test_nothing_is_launched_between():
    text = body(code("kv8_shared.cu"), "int rv_kv8_attention_shared")
    first, second = text.index("launch_kv8_attention("), text.index("launch_prefix_")
    assert first < second and "launch" not in text[first + len("launch_kv8_attention("):second].replace("launched", "")


def test_kernels_that_do_not_wait_first_are_named():
    """The rule for all kernels names the one that it does not hold for, and that one waits at its end."""
    text = body(code("kv8_shared.cuh"), " k_prefix")
    assert "pdl_wait()" in text[-40:]
    assert "k_prefix" in source("ops.cuh")[:source("ops.cuh").index("op_fail")]


@pytest.mark.parametrize("entry,name", [("rv_kv8_copy", "kv8_copy.cu"), ("rv_kv8_attention_shared", "kv8_shared.cuh")])
def test_status_bits_are_documented(entry, name):
    """A kernel that reports a wait that ran out does so in a bit that its entry's comment gives."""
    assert "kErrWait" in code(name) and "kErrWait = 16" in code("async.cuh")
    with open(os.path.join(os.path.dirname(HERE), "include", "rv.h")) as f:
        text = f.read()
    comment = text[:text.index("int %s(" % entry)]
    comment = " ".join(re.sub(r"\n \* ?", " ", comment[comment.rindex("/*"):]).split())
    assert "bit 4 (16)" in comment
