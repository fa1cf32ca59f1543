"""Kernels that start while the kernel before them still runs: what that kernel
writes must not reach them through a pointer that promises read-only data."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "prompt_compression_b200", "csrc")

# Read-only for the whole call: written before the first kernel of the call starts.
READ_ONLY = {"idx", "dst"}


def _kernels(text):
    """(name, parameters, body) of each __global__ function."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\(([^{]*)\)\s*\{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(1), m.group(2), text[m.end():at]


def _overlapping():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu"):
            for kernel, params, body in _kernels(open(os.path.join(CSRC, name)).read()):
                if "wait_for_previous()" in body or "griddepcontrol.wait" in body:
                    yield kernel, params, body


def test_the_overlapping_kernels_are_found():
    assert {k for k, _, _ in _overlapping()} >= {"copy_tail_kernel", "compact_rows_kernel", "tree_join_kernel"}


@pytest.mark.parametrize("kernel,params,body", [pytest.param(*k, id=k[0]) for k in _overlapping()])
def test_what_the_kernel_before_writes_is_not_promised_to_be_read_only(kernel, params, body):
    promised = {m.group(1) for m in re.finditer(r"const\s+\w+\s*\*\s*__restrict__\s+(\w+)", params)}
    assert promised <= READ_ONLY, f"{kernel}: {promised - READ_ONLY}"
    loaded = {m.group(1) for m in re.finditer(r"__ldg\(\s*&?(\w+)", body)}
    assert loaded <= READ_ONLY, f"{kernel}: non-coherent loads of {loaded - READ_ONLY}"
