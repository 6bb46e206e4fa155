"""Lengths up to the largest int32: a row longer than its table is reported by
every page operator and by the append and the prefill of the block-scaled cache."""
import numpy as np
import pytest
import torch

from tests.helpers import to_dev_i32

pytestmark = pytest.mark.gpu
LENGTHS = [65, 2 ** 31 - 16, 2 ** 31 - 15, 2 ** 31 - 1]  # rows of four pages below


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


def state(length):
    tables = to_dev_i32([[5, 1, 6, 3], [0, 2, -1, -1], [-1] * 4])
    refs = np.zeros(8, np.int32)
    refs[[5, 1, 6, 3, 0, 2]] = 1
    return tables, to_dev_i32([length, 20, 0]), to_dev_i32(refs), to_dev_i32([0])


@pytest.mark.parametrize("length", LENGTHS)
def test_free(ops, length):
    t, c, r, err = state(length)
    ops.free_pages(t, c, to_dev_i32([0]), r, error_flags=err)
    assert err.tolist() == [ops.DEVERR_SHAPE]
    assert c.tolist() == [0, 20, 0] and r.tolist() == [1, 0, 1, 0, 0, 0, 0, 0]


@pytest.mark.parametrize("length", LENGTHS)
def test_compact(ops, length):
    t, c, r, err = state(length)
    _, _, counts, remap = ops.compact_pages(t, c, r, error_flags=err)
    assert err.tolist() == [ops.DEVERR_SHAPE]
    assert counts.tolist() == [1, 6] and remap.tolist() == [0, 1, 2, 3, 4, 5, 4, 7]
    assert t.tolist() == [[5, 1, 4, 3], [0, 2, -1, -1], [-1] * 4]
    assert r.tolist() == [1] * 6 + [0, 0] and c.tolist() == [length, 20, 0]


@pytest.mark.parametrize("length", LENGTHS)
def test_fork(ops, length):
    t, c, r, err = state(length)
    src, dst, forked = ops.fork_pages(t, c, to_dev_i32([0]), to_dev_i32([2]), r, error_flags=err)
    assert err.tolist() == [ops.DEVERR_SHAPE] and forked.tolist() == [-1]
    assert src.tolist() == dst.tolist() == [-1] and c.tolist() == [length, 20, 0]


@pytest.mark.parametrize("length", LENGTHS)
def test_append_and_prefill(ops, length):
    t, c, _, err = state(length)
    pools = [p.zero_() for p in ops.fp8_block_pools(8, 2, device="cuda")]
    rows = torch.ones((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    cu = to_dev_i32([0, 1, 2, 2])
    ops.store_kv_fp8_block(rows, rows, *pools, cu, t, c, error_flags=err)
    assert err.tolist() == [ops.DEVERR_SHAPE]
    touched = [i for i in range(8) if pools[0][i].any()]
    assert touched == [2]  # position 19 of the second row
    err.zero_()
    q = torch.ones((2, 4, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.full((2, 4, 128), 7.0, device="cuda")
    ops.prefill_varlen_fp8_block(q, cu, *pools, t, c, 0.1, 1, out=out, error_flags=err)
    assert err.item() & ops.DEVERR_SHAPE
    assert torch.all(out[0] == 7.0) and not torch.any(out[1] == 7.0)
