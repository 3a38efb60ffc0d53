"""The order of distinct picks among many experts, against numpy's stable sort."""
import numpy as np
import pytest
import torch

from test_token_order import dispatch, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k", [(5000, 1024, 8), (70001, 1024, 2), (3001, 512, 32)])
def test_distinct_picks_of_many_experts(T, E, k):
    """A token's picks differ: an odd stride from a random first one."""
    rng = np.random.default_rng(T)
    first, stride = rng.integers(0, E, (T, 1)), 2 * rng.integers(0, E // 2, (T, 1)) + 1
    ids = ((first + stride * np.arange(k)) % E).astype(np.int32)
    assert all(len(set(r)) == k for r in ids[:50])
    say(f"[order] distinct T={T} E={E} k={k}")
    start, rows, pos, _ = dispatch(ids, E)
    want = np.argsort(ids.reshape(-1), kind="stable").astype(np.int32)
    assert np.array_equal(rows.cpu().numpy(), want)
    assert np.array_equal(start.cpu().numpy(), np.searchsorted(ids.reshape(-1)[want], np.arange(E + 1)))
    back = np.empty_like(want)
    back[want] = np.arange(T * k)
    assert np.array_equal(pos.cpu().numpy().reshape(-1), back)
