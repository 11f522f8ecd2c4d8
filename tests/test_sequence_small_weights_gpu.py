"""Many keys of small weight beside a few of large weight: what they add up to is kept.

Of c keys, `tops` score x1 = q.k and the others 0, so a row's output is
o = (c - tops) w / (tops + (c - tops) w), w = 2^(-x1 log2 e), times the others' value 1
(the tops' is 0).  At c = 131000, tops = 1 and w = 2^-25.4 that is 0.003: six half steps of
fp16 at 1, made of weights below fp16's least positive number, 2^-24.

Tolerance, u the type's half step:
  * P is rounded once: u of o, and in fp16, where P is 2^7 times the weight of a row's
    shift, an absolute 2^-25 / 2^7 = 2^-32 a key: c 2^-32 / tops;
  * a score is off by at most d 2^-24 x1, which moves weights by twice that: of o;
  * sums over c keys: c 2^-24 of o, and of the normaliser;
  * ex2, the join and the final division: 2^-19 of o; o rounded once: u of o.
"""
import math

import pytest
import torch

from memory_bound_row_softmax_gb300 import binding as B
from memory_bound_row_softmax_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

KEYS, PAGE = 131000, 64


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    yield
    assert B.check_device_error() == B.OK


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["single tokens", "five tokens of five heads", "one long sequence"])
def test_small_weights_add_up(dtype, d, kind):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    pages = -(-KEYS // PAGE)
    k, v = (torch.zeros(pages, PAGE, 1, d, dtype=dtype, device="cuda") for _ in range(2))
    v += 1.0
    # work in equal items, as many as blocks, so that none is cut: a row's weights meet in
    # one state, or in the four of the warps that share a tile, with a top key in each
    if kind == "one long sequence":
        tops, lens, heads = [0], [256 * 2 * sms], 1
    else:
        tops = [0, 16, 32, 48]
        lens, heads = ([1] * 2 * sms, 1) if kind == "single tokens" else ([5] * sms, 5)
    for t in tops:
        k[0, t, 0, 0] = 4.4
        v[0, t] = 0.0
    q = torch.zeros(sum(lens), heads, d, dtype=dtype, device="cuda")
    q[..., 0] = 4.0
    starts = torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda")
    starts[1:] = torch.tensor(lens, device="cuda").cumsum(0)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].repeat(len(lens), 1)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = B.attention_paged_fwd(q, k, v, table, ints([KEYS] * len(lens)), starts, causal=False, sm_scale=1.0, lse=lse)
    x1 = 4.0 * float(k[0, 0, 0, 0])
    w, n = math.exp(-x1), len(tops)
    rest = (KEYS - n) * w
    want = rest / (n + rest)
    u = torch.finfo(dtype).eps / 2
    relative = 2 * u + 2 * d * 2.0 ** -24 * x1 + 2 * KEYS * 2.0 ** -24 + 2.0 ** -19
    absolute = KEYS * 2.0 ** -32 / n if dtype == torch.float16 else 0.0
    assert (out.double() - want).abs().max().item() <= relative * want + absolute
    want = x1 + math.log(n + rest)
    assert (lse.double() - want).abs().max().item() <= d * 2.0 ** -24 * x1 + KEYS * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** -22 * want
