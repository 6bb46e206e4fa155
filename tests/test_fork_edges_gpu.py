"""Forks at the edge: rows whose length is any value below 1, and parents whose
last entry lies outside the pool."""
import numpy as np
import pytest
import torch

from tests.helpers import to_dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


def fork(ops, tables, ctx, refs, parents, children):
    """(err, src, dst, forked, tables, ctx, refs) after the call."""
    t, c, r = to_dev_i32(tables), to_dev_i32(ctx), to_dev_i32(refs)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ops.fork_pages(t, c, to_dev_i32(parents), to_dev_i32(children), r, error_flags=err)
    return (int(err.item()), *(x.cpu().numpy() for x in (*out, t, c, r)))


@pytest.mark.parametrize("n", [3, 1100])
def test_empty_rows_of_any_negative_length(ops, n):
    """Every length below 1 is an empty row, the least integers among them (the
    plan marks claimed rows with those), as a child and as a parent."""
    rows, NB = 2 * n + 2, 2 * n + 4
    tables = np.full((rows, 2), -1, np.int32)
    tables[0] = [0, 1]
    refs = np.zeros(NB, np.int32)
    refs[:2] = 1
    ctx = np.zeros(rows, np.int32)
    ctx[0] = 20
    ctx[1:n + 1] = -2 ** 31 + np.arange(n)[::-1]  # child i holds another fork's mark
    ctx[n + 1] = -2 ** 31
    parents, children = [0] * n, list(range(1, n + 1))
    err, src, dst, forked, t, c, r = fork(ops, tables, ctx, refs, parents, children)
    assert err == 0
    assert list(forked) == [20] * n and list(src) == [1] * n
    assert list(dst) == list(range(2, n + 2))
    assert list(c[:n + 1]) == [20] * (n + 1) and r[0] == n + 1 and list(r[1:n + 2]) == [1] * (n + 1)
    assert np.array_equal(t[1:n + 1], [[0, d] for d in dst])
    # a parent of such a length gives an empty child; a child named twice is refused
    err, src, dst, forked, t, c, r = fork(ops, tables, ctx, refs, [n + 1, 0, 0], [2, 3, 3])
    assert err == ops.DEVERR_SHAPE
    assert list(forked) == [0, 20, -1] and list(dst) == [-1, 2, -1]
    assert c[2] == 0 and c[3] == 20


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 12, 2 ** 31 - 1])
def test_last_entry_outside_the_pool(ops, bad):
    """Copied and reported like any other: no page is taken in its place and
    no pair names it."""
    tables = np.array([[0, bad], [1, 2], [-1, -1], [-1, -1]], np.int32)
    refs = np.zeros(12, np.int32)
    refs[:3] = 1
    err, src, dst, forked, t, c, r = fork(ops, tables, [20, 20, 0, 0], refs, [0, 1], [2, 3])
    assert err == ops.DEVERR_BLOCK_INDEX
    assert list(forked) == [20, 20] and list(c) == [20] * 4
    assert (src[0], dst[0]) == (-1, -1) and list(t[2]) == [0, bad]
    assert src[1] == 2 and dst[1] >= 3 and list(t[3]) == [1, dst[1]]
    want = np.zeros(12, np.int32)
    want[[0, 1, 2, dst[1]]] = [2, 2, 1, 1]
    assert np.array_equal(r, want)
