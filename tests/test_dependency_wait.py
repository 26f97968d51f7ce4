"""Kernels that may be scheduled beside their predecessor read with ordinary
loads what that one may have written.

A read-only load (__ldg, or one that nvcc makes of an ordinary load through a
`const T *__restrict__` kernel parameter) is for data that nothing writes while
the kernel lives: it need not stay behind griddepcontrol.wait.  Checked on the
source, because the fault itself shows only by timing.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_weight_mat_gb300", "csrc")
# Weights declared static (pq_set_weight_prefetch), which this kernel reads before its wait.
STATIC = {"gemv_q8_0_short": ["w"]}


def code(path):
    """The source without comments and strings' contents apart from the wait's."""
    with open(path) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def waiting_files():
    return sorted(p for p in glob.glob(os.path.join(CSRC, "*.cu*")) if "griddepcontrol.wait" in code(p))


def kernels(text):
    """(name, parameter list, body) of every __global__ function."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\((?:[^()]|\([^()]*\))*\))*\)\s*)?(\w+)\s*\(", text):
        at, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        params, begin = text[m.end():at - 1], text.index("{", at)
        end, depth = begin + 1, 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        yield m.group(1), params, text[begin:end]


def test_the_files_are_found():
    names = [os.path.basename(p) for p in waiting_files()]
    assert {"gemv_generic.cu", "gemv_stream.cu", "gemv_tc.cu", "kv_cache.cu", "attn_mma.cu", "attn_tc.cu"} <= set(names)
    found = [k for p in waiting_files() for k, _, _ in kernels(code(p))]
    assert {"gemv_generic_q4_k", "gemv_q8_0_short", "gemv_rows", "prep_x_tc", "tc_finish", "kv_append", "attn_join"} <= set(found)


@pytest.mark.parametrize("path", waiting_files(), ids=os.path.basename)
def test_no_kernel_parameter_is_declared_read_only(path):
    bad = []
    for name, params, _ in kernels(code(path)):
        for p in params.split(","):
            if re.search(r"\bconst\b[^*]*\*\s*__restrict__", p) and p.split()[-1].lstrip("*") not in STATIC.get(name, []):
                bad.append((name, " ".join(p.split())))
    assert not bad


@pytest.mark.parametrize("path", waiting_files() + [os.path.join(CSRC, f) for f in ("pq_device.cuh", "pq_kfamily.cuh", "kv_device.cuh")],
                         ids=os.path.basename)
def test_no_read_only_load_behind_the_wait(path):
    text = code(path)
    for name, _, body in kernels(text):
        if name in STATIC:      # up to the wait
            text = text.replace(body, body[body.index("griddepcontrol.wait"):])
    assert "__ldg(" not in text and "ld.global.nc" not in text
