"""How the sequence calls are launched: the process-wide launch-overlap switch holds for
them too, and waits that run out end a call of every kernel and variant."""
import ctypes
import math

import pytest
import torch

from memory_bound_row_softmax_gb300 import binding as B
from memory_bound_row_softmax_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

SENTINEL = 7.0
PROGRAMMATIC = 1  # CU_GRAPH_DEPENDENCY_TYPE_PROGRAMMATIC


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    yield
    assert B.check_device_error() == B.OK


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def normal(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


class EdgeData(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte),
                ("reserved", ctypes.c_ubyte * 5)]


def captured_edges(calls):
    """The dependency types between the launches of `calls`, captured on a stream and not run."""
    cuda = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph, n = ctypes.c_void_p(), ctypes.c_size_t(0)
    with torch.cuda.stream(stream):
        assert cuda.cuStreamBeginCapture_v2(ctypes.c_void_p(stream.cuda_stream), 2) == 0  # relaxed
        try:
            for call in calls:
                call()
        finally:
            assert cuda.cuStreamEndCapture(ctypes.c_void_p(stream.cuda_stream), ctypes.byref(graph)) == 0
    try:
        assert cuda.cuGraphGetEdges_v2(graph, None, None, None, ctypes.byref(n)) == 0
        ends, data = [(ctypes.c_void_p * n.value)() for _ in range(2)], (EdgeData * n.value)()
        assert cuda.cuGraphGetEdges_v2(graph, *ends, data, ctypes.byref(n)) == 0
        return [e.type for e in data[:n.value]]
    finally:
        cuda.cuGraphDestroy(graph)


@pytest.mark.parametrize("overlap", [True, False])
def test_launch_overlap_switch(overlap):
    """Two appends, single tokens (two launches), a short chunk (two) and many prompts
    (three), one after the other: eight edges, all programmatic or none."""
    pages, page, kv, d = 64, 16, 8, 64
    kc, vc = (torch.zeros(pages, page, kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, lens = torch.arange(pages, dtype=torch.int32, device="cuda")[None], ints(900)
    k = normal(1, 20000, kv, d)
    space = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    out, one, chunk = torch.empty_like(k), ints(0, 1), ints(0, 300)
    many = torch.arange(0, 20001, 2000, dtype=torch.int32, device="cuda")
    calls = [lambda: B.kv_cache_append(k[:300], k[:300], kc, vc, table, lens, chunk)] * 2 + [
        lambda: B.attention_paged_fwd(k[:1], kc, vc, table, lens, one, out=out[:1], workspace=space),
        lambda: B.attention_paged_fwd(k[:300], kc, vc, table, lens, chunk, out=out[:300], workspace=space),
        lambda: B.attention_varlen_fwd(k, k, k, many, out=out, workspace=space)]
    try:
        B.set_launch_overlap(overlap)
        types = captured_edges(calls)
    finally:
        B.set_launch_overlap(True)
    assert len(types) == 8 and all((t == PROGRAMMATIC) == overlap for t in types), types


def test_results_with_and_without_overlap():
    pages, page, kv, d, n = 64, 16, 2, 128, 260
    k, v, q = normal(1, n, kv, d), normal(2, n, kv, d), normal(3, n, 8, d)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    results = []
    try:
        for overlap in (True, False):
            B.set_launch_overlap(overlap)
            kc, vc = (torch.zeros(pages, page, kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            got = []
            for lo, hi in ((0, 200), (200, 259), (259, 260)):
                starts, lens = ints(0, hi - lo), ints(hi)
                B.kv_cache_append(k[lo:hi], v[lo:hi], kc, vc, table, lens, starts)
                got.append(B.attention_paged_fwd(q[lo:hi], kc, vc, table, lens, starts))
            got.append(B.attention_varlen_fwd(q, k, v, ints(0, n)))
            results.append([*got, kc, vc])
    finally:
        B.set_launch_overlap(True)
    assert all(torch.equal(a, b) for a, b in zip(*results))


# rows of a sequence, keys and head dim: one group of 16 rows and two, each in whole items
# and cut ones; tiles of head dim 64 (three S buffers) and 128, whole and cut
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,heads,keys", [([1] * 3, 4, 40), ([1], 4, 5000), ([5] * 3, 5, 40), ([5], 5, 5000),
                                             ([200, 90], 2, 300), ([300], 2, 9000)], ids=str)
def test_waits_that_run_out(lens, heads, keys, d):
    """A tile that never lands: the waits give up and report it, the rows are left as they
    were (nothing is merged from a workspace that nobody wrote), and the next call is right."""
    page = 8
    pages = -(-keys // page)
    kc, vc = normal(1, pages, page, 1, d), normal(2, pages, page, 1, d)
    q = normal(3, sum(lens), heads, d)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].repeat(len(lens), 1)
    klen = ints(*[keys] * len(lens))
    starts = torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda")
    starts[1:] = ints(*lens).cumsum(0)
    space = torch.full((B.sequence_workspace_bytes(q.shape[0], len(lens), heads, 1, d, "bf16", page_size=page, pages=pages,
                                                   max_pages=pages),), 255, dtype=torch.uint8, device="cuda")

    def call(out, lse):
        B.attention_paged_fwd(q, kc, vc, table, klen, starts, out=out, lse=lse, workspace=space)
        torch.cuda.synchronize()
        return out, lse

    def outputs():
        return torch.full_like(q, SENTINEL), torch.full(q.shape[:2], SENTINEL, device="cuda")

    out, lse = outputs()
    B.set_wait_test(20_000_000)
    B.set_attention_wait_test(True)
    try:
        call(out, lse)
        assert B.check_device_error() == B.ERR_TIMEOUT
    finally:
        B.set_attention_wait_test(False)
        B.set_wait_test(0)
    assert (out == SENTINEL).all() and (lse == SENTINEL).all()
    assert B.check_device_error() == B.OK
    out, lse = call(*outputs())
    assert B.check_device_error() == B.OK
    x = torch.einsum("nhd,cd->nhc", q.double(), kc.flatten(0, 1)[:keys, 0].double()) / math.sqrt(d)
    seen = torch.cat([torch.arange(keys - n, keys, device="cuda") for n in lens])
    x = torch.where(torch.arange(keys, device="cuda") <= seen[:, None, None], x, -math.inf)
    want = x.softmax(-1) @ vc.flatten(0, 1)[:keys, 0].double()
    # P and o each rounded to bf16 (2^-8 of max|v| and of |o|), and 2^-12 for what is in fp32
    tol = 2.0 ** -8 * (vc.double().abs().max() + want.abs()) + 2.0 ** -12
    assert ((out.double() - want).abs() <= tol).all()
    assert ((lse.double() - torch.logsumexp(x, -1)).abs() <= 2.0 ** -12).all()
