"""The rules by which a sequence attention call chooses how it runs (csrc/sequence_rules.h),
compiled for the host."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "memory_bound_row_softmax_gb300", "csrc")
WRAPPER = """
#include "sequence_rules.h"
using namespace mbrs::seq;
extern "C" int plan_cuts_c(uint64_t blocks, uint64_t tiles, uint32_t most, uint32_t least, uint32_t kv_heads, uint32_t sms,
                           uint32_t capacity, uint32_t cut_cost) {
    return plan_cuts(PlanCounts{blocks, tiles, most, least}, kv_heads, sms, capacity, cut_cost);
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    src, so = d / "rules.cpp", d / "rules.so"
    src.write_text(WRAPPER)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(so), str(src)], check=True)
    lib = ctypes.CDLL(str(so))
    u32, u64 = ctypes.c_uint32, ctypes.c_uint64
    lib.plan_cuts_c.argtypes = [u64, u64] + [u32] * 6
    return lib


def test_more_row_blocks_than_the_plan_has_room_for_are_cut(rules):
    """Overlapping sequences can name 2^32 row blocks and more: 2^32 + 5 of them are not 5."""
    for blocks in (101, 2**31, 2**32, 2**32 + 5, 2**33 + 100, 2**62):
        assert rules.plan_cuts_c(blocks, blocks, 1, 1, 8, 152, 100, 14)
    assert not rules.plan_cuts_c(95, 95 * 20, 20, 20, 8, 152, 100, 14)


def test_cutting(rules):
    # 8 whole waves of equal items; one item too many of 20 tiles, idle for longer than 14; of 5, not
    assert not rules.plan_cuts_c(152, 152 * 20, 20, 20, 8, 152, 1000, 14)
    assert rules.plan_cuts_c(153, 153 * 20, 20, 20, 8, 152, 1000, 14)
    assert not rules.plan_cuts_c(153, 153 * 5, 5, 5, 8, 152, 1000, 14)
    # one item longer than an SM's share of all
    assert rules.plan_cuts_c(100, 100 + 200, 200, 1, 8, 152, 1000, 14)
    # nothing to do
    assert not rules.plan_cuts_c(0, 0, 0, 2**31 - 1, 8, 152, 1000, 14)
