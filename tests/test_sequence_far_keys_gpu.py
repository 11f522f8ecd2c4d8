"""Keys whose weight is too small for 32 bits beside a row's largest: their values are
multiplied by zero, so finite ones add nothing and infinite or NaN ones make the element
infinite or NaN -- whichever warp, part or product holds the key."""
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


# rows of one sequence and its keys: a single token in one block and cut into parts, two
# groups of rows likewise, and the tiles of many rows, whole and cut.
SHAPES = [(1, 4, 64), (1, 4, 9000), (5, 5, 64), (5, 5, 9000), (200, 2, 256), (200, 2, 9000)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,heads,keys", SHAPES)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_value_far_below_the_rows_max(dtype, d, n, heads, keys, bad):
    """Scores: -300 for the first keys (exp underflows in 32 bits), 0 for the others.  Of
    many keys, the first 128: a part of a cut item with no others."""
    page, at, column, low = 16, 3, 9, 128 if keys > 256 else 16
    pages = -(-keys // page)
    k, v = (torch.zeros(pages, page, 1, d, dtype=dtype, device="cuda") for _ in range(2))
    v += 1.0
    k[:low // page, :, 0, 0] = -18.75
    q = torch.zeros(n, heads, d, dtype=dtype, device="cuda")
    q[:, :, 0] = 16.0
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lse = torch.empty(n, heads, device="cuda")

    def call():
        return B.attention_paged_fwd(q, k, v, table, ints(keys), ints(0, n), causal=False, sm_scale=1.0, lse=lse)

    one = call()
    # 1 divided by its own sum of ones: exact weights, so within a rounding of the type
    assert (one.double() - 1).abs().max() <= torch.finfo(dtype).eps / 2
    v[0, at, 0, column] = bad
    out = call()
    assert not out[..., column].isfinite().any()
    out[..., column] = one[..., column]
    assert torch.equal(out, one)
    # log of keys - low: the tests' bound of a log-sum-exp, n 2^-24 + 2^-19 and its own rounding
    want = math.log(keys - low)
    assert (lse.double() - want).abs().max() <= keys * 2.0 ** -24 + 2.0 ** -19 + 3 * 2.0 ** -24 * want
