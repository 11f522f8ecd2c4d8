"""Infinite and NaN values in every variant of the attention kernels: they reach the rows
that keep their keys, in their own column, and change no bit of anything else.

A value stands in one column of one key, so the same call with a zero in its place must
give the same bits everywhere but in that column of the rows that keep the key: both calls
round the same sums in the same order, and a kept value of zero adds nothing.  In that
column the result is the value itself: its weight is positive (scores deviate by 2, and
no weight above 2^-32 of a row's largest is rounded to zero, 22 in scores)."""
import math

import pytest
import torch

from memory_bound_row_softmax_gb300 import binding as B
from memory_bound_row_softmax_gb300 import build as build_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    yield
    assert B.check_device_error() == B.OK


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# new tokens and keys of a sequence, sequences, query heads, kv heads
VARIANTS = {
    "one row group, whole": (3, 60, 1, 4, 1), "one row group, cut": (3, 5000, 1, 4, 1),
    "two row groups, whole": (5, 60, 1, 5, 1), "two row groups, cut": (5, 5000, 1, 5, 1),
    "two row groups, many sequences": (5, 200, 90, 10, 2),
    "one tile, whole": (40, 100, 1, 4, 1), "one tile, cut": (40, 5000, 1, 2, 1),
    "two tiles, whole": (100, 100, 1, 2, 1), "two tiles, cut": (300, 2000, 1, 2, 1),
    "planned": (300, 700, 40, 8, 8),
}


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("causal", [True, False])
def test_values_that_are_not_finite(dtype, d, variant, bad, causal):
    n, c, batch, heads, kv_heads = VARIANTS[variant]
    page = 16
    per = -(-c // page)
    g = torch.Generator(device="cuda").manual_seed(n + c)
    k, v = (torch.randn(batch * per, page, kv_heads, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    k[per - 1::per, (c - 1) % page + 1:], v[per - 1::per, (c - 1) % page + 1:] = math.nan, math.inf  # past the last key
    q = (2 * torch.randn(batch * n, heads, d, generator=g, device="cuda")).to(dtype)
    table = torch.arange(batch * per, dtype=torch.int32, device="cuda").view(batch, per)
    klen, starts = ints(*[c] * batch), torch.arange(batch + 1, dtype=torch.int32, device="cuda") * n
    # the last key, one in the middle of the new ones, the first new one, one that all rows keep
    # (the first of the cache; without older keys, the first token's own)
    keys = {c - 1: 5, c - n // 2 - 1: d - 3, c - n: 8, 0: 33}
    hit = sorted({0, batch // 2, batch - 1})

    def call():
        return B.attention_paged_fwd(q, k, v, table, klen, starts, causal=causal).view(batch, n, heads, d)

    def put(value):
        for b in hit:
            for j, column in keys.items():
                v[table[b, j // page].item(), j % page, kv_heads - 1, column] = value

    put(0.0)
    zero = call()
    assert zero.isfinite().all()
    put(bad)
    got = call()
    touched = torch.zeros(batch, n, heads, d, dtype=torch.bool, device="cuda")
    rows = torch.arange(n, device="cuda")
    for b in hit:
        for j, column in keys.items():
            keep = rows + c - n >= j if causal else rows >= 0
            touched[b, keep, heads - heads // kv_heads:, column] = True
    assert torch.equal(got[~touched], zero[~touched])
    assert got[touched].isnan().all() if math.isnan(bad) else (got[touched] == bad).all()
