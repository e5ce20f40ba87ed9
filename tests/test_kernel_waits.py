"""Programmatic dependent launch: what an earlier kernel has written is promised to a kernel that has waited for it.  So every
kernel of the operators for several continuations waits, on all paths, before it reads through a pointer of its arguments."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_speculative_decoding_03_gb300", "csrc", "serving")


def read(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


POINTERS = set(re.findall(r"^\s+(?:const )?\w+(?: \w+)?\* (\w+);", read("continue_args.cuh"), re.M))


def kernels(text):
    """(name, body) of each __global__ function."""
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\(", text):
        start = text.index("{", text.index(")", m.end()))
        depth = 0
        for i in range(start, len(text)):
            depth += (text[i] == "{") - (text[i] == "}")
            if depth == 0:
                yield m.group(1), text[start + 1: i]
                break


@pytest.mark.parametrize("name", ["pages.cu", "prefix_attn.cu", "prefix_tc.cu", "logprobs.cu"])
def test_every_kernel_waits_before_it_reads(name):
    found = list(kernels(read(name)))
    assert {"seq_err", "block_table", "start", "tc_begin", "used", "logits"} <= POINTERS
    assert len(found) >= {"pages.cu": 10, "prefix_attn.cu": 3, "prefix_tc.cu": 1, "logprobs.cu": 2}[name]
    for kernel, body in found:
        before, wait, _ = body.partition("pdl_wait();")
        assert wait, kernel
        assert before.count("{") == before.count("}") and re.search(r"(^|[;{}])\s*$", before), f"{kernel}: the wait is conditional"
        used = set(re.findall(r"\ba\.(\w+)", before)) & POINTERS
        assert not used, f"{kernel} reads {used} before it waits"
        assert body.count("pdl_wait();") == 1, kernel
