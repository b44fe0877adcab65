"""Reads the CUDA sources: every bounded wait's outcome is looked at, and every read of the tensor cores'
accumulators waits for the values it names.

A wait on the device gives up after a time limit.  The only report that a user gets of it is the error
word that the caller of the wait sets, so a call whose result is dropped would let a kernel store what
it never waited for and still be reported as a success.  Such a wait cannot be made to run out from
outside without hanging a GPU's pipeline, so the sources are read instead.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_expert_ffn_router_b200", "csrc")
WAITS = ("mbar_wait_bounded", "wait_or_abort", "rt_wait", "grid_wait", "grid_sync", "few_barrier")


def _code(path):
    src = open(path).read()
    src = re.sub(r"/\*.*?\*/", lambda m: "\n" * m.group().count("\n"), src, flags=re.S)
    return re.sub(r"//[^\n]*", "", src)


def dropped(src):
    """Lines of `src` with a wait as a whole statement.  A result that is not needed because an error has
    been raised already is dropped by a cast to void."""
    names = "|".join(WAITS)
    lines = []
    for m in re.finditer(rf"(?:^|[;{{}})]|\belse\b)\s*({names})\s*(?:<[^<>;]*>)?\s*\(", src):
        if not src[: m.start(1)].rstrip().endswith("(void)"):
            lines.append(src.count("\n", 0, m.start(1)) + 1)
    return lines


def test_the_reading_finds_dropped_results():
    assert dropped("a();\n  mbar_wait_bounded(&b, 0);\n") == [2]
    assert dropped("if (x) wait_or_abort<true>(&b, 0, f);") == [1]
    assert dropped("for (;;) mbar_wait_bounded(&b, 0);") == [1]
    assert dropped("else grid_sync<0>(c, G, f);") == [1]
    assert dropped("if (!mbar_wait_bounded(&b, 0)) f(); const bool g = a && grid_wait(c, 0, G, f);") == []
    assert dropped("return grid_wait<k>(c, 0, G, f); (void)mbar_wait_bounded(&b, 0);") == []
    assert dropped("__device__ __forceinline__ bool mbar_wait_bounded(uint64_t* bar, uint32_t parity) {") == []


@pytest.mark.parametrize("name", sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu*"))))
def test_no_wait_result_is_dropped(name):
    assert dropped(_code(os.path.join(CSRC, name))) == []


@pytest.mark.parametrize("name", sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu*"))))
def test_loads_from_tensor_memory_pass_through_their_wait(name):
    # tcgen05.ld delivers its registers later; arithmetic on them is held behind the wait only if the wait
    # has them as operands (a clobber of memory does not order arithmetic)
    src = _code(os.path.join(CSRC, name))
    assert not re.search(r"tmem_ld_wait\w*\(\s*\)\s*;", src)
    assert src.count("tcgen05.wait::ld") == (1 if name == "common.cuh" else 0)
