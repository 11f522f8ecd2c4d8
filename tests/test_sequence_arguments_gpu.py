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


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_takes_positions_from_lengths_as_they_are(interleaved):
    """Lengths past the table and below zero: tokens with a place are written there, the
    others' keys and values nowhere, and every query turns by its own position."""
    page, pages, d, n = 8, 5, 64, 6
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v, q = (torch.randn(2 * n, 1, d, generator=g, device="cuda").half() for _ in range(3))
    kc, vc = (torch.zeros(pages, page, 1, d, dtype=torch.float16, device="cuda") for _ in range(2))
    table, freq = ints(3, 1, 2, 0).view(2, 2), torch.linspace(1.0, 0.01, d // 2, device="cuda")
    # positions 14 .. 19 of 16 slots, and -8 .. -3
    out = B.kv_cache_append(k, v, kc, vc, table, ints(20, -2), ints(0, n, 2 * n), inv_freq=freq, interleaved=interleaved, q=q)
    assert torch.equal(vc[1, 6:], v[:2]) and not vc[[0, 2, 3, 4]].any() and not vc[1, :6].any()
    assert kc[1, 6:].any() and not kc[[0, 2, 3, 4]].any() and not kc[1, :6].any()
    pos = torch.cat([torch.arange(14, 20), torch.arange(-8, -2)]).cuda().double()
    turn = torch.polar(torch.ones(2 * n, d // 2, dtype=torch.float64, device="cuda"), pos[:, None] * freq.double())[:, None]
    first = torch.arange(d // 2, device="cuda") * (2 if interleaved else 1)
    second = first + (1 if interleaved else d // 2)
    for got, x, rows in ((out, q, slice(0, 2 * n)), (kc[1, 6:], k, slice(0, 2))):
        x = x[rows].double()
        z = torch.complex(x[..., first], x[..., second]) * turn[rows]
        want = torch.empty_like(x)
        want[..., first], want[..., second] = z.real, z.imag
        # half a step of fp16, and 2^-20 of the pair for the fp32 rotation and its sines
        size = torch.empty_like(x)
        size[..., first] = size[..., second] = x[..., first].abs() + x[..., second].abs()
        assert ((got.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -19 * size + 2.0 ** -25).all()


def test_two_tokens_on_one_slot():
    """Two sequences that share their last page: each 16 bytes of a slot both write are
    those of one of the two tokens, and nothing else is touched."""
    page, d, kv = 8, 128, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(2, kv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    for _ in range(20):
        kc, vc = (torch.zeros(3, page, kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        B.kv_cache_append(k, v, kc, vc, ints(2, 2).view(2, 1), ints(4, 4), ints(0, 1, 2))
        for cache, x in ((kc, k), (vc, v)):
            got, both = cache[2, 3].view(kv, d // 8, 8), x.view(2, kv, d // 8, 8)
            assert ((got == both[0]).all(-1) | (got == both[1]).all(-1)).all()
            cache[2, 3] = 0
            assert not cache.any()
