"""A model of what the two softmax groups of the tile kernel (k_seq_tiles.cu) do to a
value that is infinite or NaN in a tile they share, before their products read it.

A group's thread looks at the value with an ordinary load, sets it to zero with an
ordinary store if it is not finite, and lets its group's product read the tile.  The
product reads shared memory through the async proxy: an ordinary store is sure to be
seen there only once a thread that made it, or that has seen it, has run a proxy fence.
Every order of the two groups' steps is walked through; whether the kernel fences where a
look found nothing is read from its source.
"""
import os

import pytest

BAD, ZERO = "bad", 0
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "memory_bound_row_softmax_gb300",
                      "csrc", "k_seq_tiles.cu")


def kernel_fences_when_clean():
    """The look ends in the fence, at the function's outer level, and nothing returns before it."""
    with open(SOURCE) as f:
        body = f.read().split("void zero_bad_values(", 1)[1].split("\n}\n", 1)[0]
    return body.endswith("\n    mbrs::fence_proxy_async_smem();") and "return" not in body


def steps(fence_when_clean):
    """A group's steps: look, store if the look found a bad value, fence, product.
    fence_when_clean: the fence is run where nothing bad was found too."""
    return ("look", "store", "fence" if fence_when_clean else "fence if bad", "product")


def orders(a, b):
    """All interleavings of the steps of groups 0 and 1."""
    if not a or not b:
        yield tuple((0, s) for s in a) + tuple((1, s) for s in b)
        return
    for rest in orders(a[1:], b):
        yield ((0, a[0]),) + rest
    for rest in orders(a, b[1:]):
        yield ((1, b[0]),) + rest


def run(order):
    """What each group's product may read at worst."""
    value, sure_in_async, seen, read = BAD, False, [None, None], [None, None]
    for group, step in order:
        if step == "look":
            seen[group] = value
        elif step == "store" and seen[group] == BAD:
            value = ZERO
        elif step == "fence" or (step == "fence if bad" and seen[group] == BAD):
            sure_in_async |= value == ZERO  # the thread has made the store or seen its zero
        elif step == "product":
            read[group] = ZERO if sure_in_async else BAD
    return read


def test_every_product_reads_the_zero():
    kernel = steps(kernel_fences_when_clean())
    every = list(orders(kernel, kernel))
    assert len(every) == 70
    assert all(run(o) == [ZERO, ZERO] for o in every)


def test_a_look_that_finds_the_zero_and_does_not_fence_is_caught():
    with pytest.raises(AssertionError):
        assert all(run(o) == [ZERO, ZERO] for o in orders(steps(False), steps(False)))
