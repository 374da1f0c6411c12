"""The rows of a plan that hold every routing: no row fewer, none more."""
import numpy as np
import pytest

import moe_ragged_contraction_gb300 as mx


def padded(counts, align):
    return sum(-(-c // align) * align for c in counts)


def most_rows(pairs, local, align):
    """Over all ways to spread the pairs, by dynamic programming: the rows that n pairs of so many experts can need."""
    best = [0] * (pairs + 1)  # (any number of pairs may be absent)
    for _ in range(local):
        best = [max(best[n - c] + -(-c // align) * align for c in range(n + 1)) for n in range(pairs + 1)]
    return best[pairs]


@pytest.mark.parametrize("align", [1, 2, 3, 7, 32])
@pytest.mark.parametrize("local", [1, 2, 3, 5, 40])
@pytest.mark.parametrize("T,k", [(0, 1), (1, 1), (1, 2), (3, 3), (5, 7), (11, 3), (40, 1), (16, 4)])
def test_over_every_routing(T, k, local, align):
    mx.build()
    assert mx.token_plan_rows(T, k, local, align) == most_rows(T * k, local, align)


@pytest.mark.parametrize("T,k,local,align", [(1, 1, 1, 32), (100, 4, 9, 1), (3, 2, 100, 128), (16384, 6, 64, 32), (32768, 8, 32, 128), (1 << 20, 8, 2048, 1024), (777, 33, 1597, 256)])
def test_a_routing_that_needs_them_all(T, k, local, align):
    """One pair each for as many experts as there are, and of the others as many whole groups as there are to one of them."""
    mx.build()
    pairs, used = T * k, min(local, T * k)
    counts = np.ones(used, np.int64)
    counts[0] += (pairs - used) // align * align
    assert counts.sum() <= pairs
    assert mx.token_plan_rows(T, k, local, align) == padded(counts.tolist(), align)
