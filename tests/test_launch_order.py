"""Kernels that let the next kernel's blocks start early, checked in the source.

A block allocates tensor memory with one warp and waits there until the SM has the
columns.  Blocks of the next kernel may only be let in once that is done: one that took
the columns first would hold them until the grid in front has ended, whose block on the
same SM would still be waiting for them.  No GPU run can show that order reliably, so the
source is read: between an allocation and the trigger there is a barrier of the block.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_deltanet_linear_chunked_b200", "csrc")
STEPS = re.compile(r"\b(tmem_alloc\(&|pdl_trigger\(\)|__syncthreads\(\)|block_sync_async\(\);)")


def steps(path):
    text = re.sub(r"//[^\n]*", "", open(path, encoding="utf-8").read())
    return [m.group(1) for m in STEPS.finditer(text)]


def kernels_with_both():
    return [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu")))
            if {"tmem_alloc(&", "pdl_trigger()"} <= set(steps(p))]


def test_there_are_such_kernels():
    assert len(kernels_with_both()) >= 2


@pytest.mark.parametrize("path", kernels_with_both(), ids=os.path.basename)
def test_tensor_memory_comes_before_the_trigger(path):
    waiting = False  # allocated by one warp, the others not yet past a barrier
    for s in steps(path):
        if s == "tmem_alloc(&":
            waiting = True
        elif s in ("__syncthreads()", "block_sync_async();"):  # the second holds the first
            waiting = False
        elif s == "pdl_trigger()":
            assert not waiting, os.path.basename(path)
