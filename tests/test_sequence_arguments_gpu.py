"""Arguments of the sequence calls at the edge of what they take."""
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


@pytest.mark.parametrize("scale", [1e39, -1e39, 1e300, math.nan, math.inf])
def test_scales_that_32_bits_cannot_hold(scale):
    """Refused by the library's own status, as the dense call does."""
    x = torch.zeros(4, 1, 64, dtype=torch.float16, device="cuda")
    cache, table = torch.zeros(2, 8, 1, 64, dtype=torch.float16, device="cuda"), ints(0, 1)[None]
    dense = torch.zeros(1, 1, 4, 128, dtype=torch.float16, device="cuda")
    for call in (lambda: B.attention_fwd(dense, dense, dense, sm_scale=scale),
                 lambda: B.attention_varlen_fwd(x, x, x, ints(0, 4), sm_scale=scale),
                 lambda: B.attention_paged_fwd(x, cache, cache, table, ints(4), ints(0, 4), sm_scale=scale)):
        with pytest.raises(B.SoftmaxError) as e:
            call()
        assert e.value.status == B.ERR_ARG
