"""The workspace query of gradient clipping on sizes that the calls reject.  Nothing here
touches a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def query():
    from activation_sparse_feed_gate_amd import tw

    return lambda *n: tw._lib.tw_grad_norm_workspace_bytes(len(n), (ctypes.c_int64 * len(n))(*n))


@pytest.mark.parametrize("n", [2 ** 63 - 1, 2 ** 63 - 8192, 2 ** 62, 1 << 35, (1 << 34) + 1])
def test_no_bytes_for_sizes_that_the_calls_reject(query, n):
    assert query(n) == 0 and query(5, n) == 0 and query(n, 5) == 0 and query(*[7] * 200, n) == 0


def test_bytes_for_sizes_that_they_take(query):
    # a part of 4 bytes for each of up to 2048 workgroups a table of 96 buffers, and one
    assert query() == 4 and query(0) == 4 and query(1) == 8 and query(8193, 0, 8192) == 16
    assert query(1 << 34) == query(1 << 34, 1 << 34) == 4 * 2049
    assert query(*[1 << 34] * 97) == 4 * (2048 + 2048 + 1)
