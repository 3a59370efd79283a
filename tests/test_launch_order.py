"""Launches that overlap: what a kernel does before it waits for the launch before it.

With programmatic launches a kernel may start while the one before it runs.  A kernel that lets its own
successor start before it has waited itself passes this on: the successor may then run beside a launch
two places before it.  So the kernels of the 4-bit weights and the block norms wait first, and let their
successors start afterwards.  Read from the sources: a race cannot be shown by running it.
"""
import os
import re

import pytest

from int8_mixed_precision_absmax_b200 import build as B

FILES = ["int4.cu", "int4_stream.cu", "int4_tile.cu", "norm.cu"]
WAIT, LET_START = "grid_dependency_wait();", "grid_launch_dependents();"


def source(name):
    text = open(os.path.join(B.CSRC, name), encoding="utf-8").read()
    return re.sub(r"//[^\n]*", "", text)


def kernels(name):
    """{name: body} of the __global__ functions of a source file."""
    text = source(name)
    found = {}
    for m in re.finditer(r"__global__", text):
        start = text.index("{", m.end())
        # the body opens behind the parameter list
        while True:
            head = text[m.end():start]
            if head.count("(") == head.count(")") and re.search(r"\w+_kernel\s*\(", head):
                break
            start = text.index("{", start + 1)
        depth, end = 0, start
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        found[re.search(r"(\w+_kernel)\s*\(", text[m.end():start]).group(1)] = text[start:end]
    return found


def test_the_kernels_are_found():
    assert [len(kernels(f)) for f in FILES] == [3, 1, 1, 2]


@pytest.mark.parametrize("name", FILES)
def test_a_kernel_waits_before_its_successor_may_start(name):
    for kernel, body in kernels(name).items():
        if LET_START in body:
            assert body.count(WAIT) == 1, kernel
            assert body.index(WAIT) < body.index(LET_START), kernel


def test_the_streaming_product_reads_nothing_before_the_wait():
    """Its weights may be what the launch before writes: before the wait they are only brought to L2."""
    body = kernels("int4_stream.cu")["int4_stream_kernel"]
    # what runs there: lambdas are defined, not called
    early = body[:body.index(WAIT)]
    lambdas = re.compile(r"auto \w+ = \[&\]\([^)]*\) \{.*?\n  \};", re.S)
    assert len(lambdas.findall(early)) == 2
    early = lambdas.sub("", early)
    early = "".join(line for line in early.splitlines(True) if "prefetch_l2(" not in line)
    for read in ("request(", "load_groups", "tma_load", "bulk_load", "load_x", "p.X", "p.bias",
                 "p.scales", "p.zeros"):
        assert read not in early, read
    late = body[body.index(WAIT):]
    assert "request();" in late and "load_groups<SUB, ZP>(nxt" in late
