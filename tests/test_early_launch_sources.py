"""Kernels that are launched before the kernel ahead has ended: what that kernel may write is not read as constant.

A load through __ldg promises memory that does not change while the grid lives, and may be moved above the wait for the
kernel ahead.  Only the rotation table, written when the handle is made, is such memory.  No run shows the fault for sure, so the
sources are looked through."""
import os
import re

import pytest

OPS = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "auto_regressive_decode_b200", "csrc_ops")
CONSTANT = {"mk_append.cu": ["r4 + i"]}      # float4s of the rotation table


def code(name):
    with open(os.path.join(OPS, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


EARLY = sorted(f for f in os.listdir(OPS) if f.endswith(".h") or f.endswith(".cu") and "grid_wait()" in code(f))


def test_the_kernels_launched_early_are_among_them():
    assert {"mk_append.cu", "mk_attend.cu", "mk_attend_tc.cu", "mk_cache.h"} <= set(EARLY)


@pytest.mark.parametrize("name", EARLY)
def test_constant_loads(name):
    text = code(name)
    assert re.findall(r"__ldg\(([^()]*)\)", text) == CONSTANT.get(name, [])
    assert text.count("__ldg(") == len(CONSTANT.get(name, []))
    assert "ld.global.nc" not in text
