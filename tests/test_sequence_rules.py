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
extern "C" int few_rows_c(int64_t tokens, int64_t batch, int64_t group) { return few_rows(tokens, batch, group); }
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    src, so = d / "rules.cpp", d / "rules.so"
    src.write_text(WRAPPER)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(so), str(src)], check=True)
    lib = ctypes.CDLL(str(so))
    u32, u64 = ctypes.c_uint32, ctypes.c_uint64
    lib.few_rows_c.argtypes = [ctypes.c_int64] * 3
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


def test_which_kernel(rules):
    few = rules.few_rows_c
    # single tokens and drafts, whatever their number
    for batch in (1, 64, 5000):
        for group in (1, 4, 8, 16):
            assert few(batch, batch, group)
    assert few(128 * 4, 128, 4) and few(32 * 4, 32, 8) and few(48 * 6, 48, 4) and few(5, 1, 5)
    # many rows a sequence
    assert not few(300, 1, 1) and not few(16 * 5, 16, 8) and not few(512, 1, 4)
    # a low average of a few long sequences and many of one token, or of none
    assert not few(448 + 64, 65, 4) and not few(900 + 128, 129, 4) and not few(97 + 190, 191, 16)
    assert not few(2000, 256, 4) and not few(16000, 2000, 4)
    # padding rows count like tokens of no sequence
    assert few(64 + 13, 64, 8)
    # sizes at the index range
    assert few(2**31 - 1025, 2**31 - 1025, 16) and not few(2**31 - 1025, 1, 128)
