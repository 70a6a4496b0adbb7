"""Kernels that may start while an earlier kernel still writes (they wait with griddepcontrol.wait) read by plain loads.
The read-only path is specified for data that does not change while the kernel runs, and a compiler may move such a load
above the wait: this is a property of the sources, so they are what is looked at."""
import os
import re

import pytest

import flow_matching_action_denoise_gb300 as fmad

CSRC = os.path.join(fmad.PKG, "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels(text):
    """(name, parameters, body) of every __global__ function."""
    for m in re.finditer(r"__global__", text):
        head = re.compile(r"(\w+)\(([^()]*(?:\([^()]*\)[^()]*)*)\)\s*\{").search(text, m.end())
        at, depth = head.end(), 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield head.group(1), head.group(2), text[head.end():at]


def test_the_sources_are_understood():
    found = {n: b for f in SOURCES for n, _, b in kernels(code(f))}
    for name in ("combine_kernel", "paged_attn_kernel", "decode_kernel", "append_kernel", "share_kernel", "qkv_finalize_kernel"):
        assert "pdl_wait" in found[name]
    assert "pdl_wait" not in found["pack_fp8_kernel"]


@pytest.mark.parametrize("name", SOURCES)
def test_no_read_only_loads_behind_a_wait(name):
    text = code(name)
    waits = [(n, p, b) for n, p, b in kernels(text) if "pdl_wait" in b]
    if waits or name.endswith(".cuh"):
        assert "__ldg" not in text and "ld.global.nc" not in text
    for kernel, params, body in waits:
        # a __restrict__ parameter may be read before the wait only: constants
        for param in re.findall(r"__restrict__\s+(\w+)", params):
            assert not re.search(rf"\b{param}\b", body[body.index("pdl_wait"):]), (kernel, param)
