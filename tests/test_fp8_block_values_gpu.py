"""Values at the edge of the block-scaled FP8 cache's attention: codes and
query rows that are NaN, infinite, huge or tiny, and where their effect ends."""
import numpy as np
import pytest
import torch

from tests import fp8_block_reference as ref
from tests.helpers import normal_bits, random_tables, to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu
SCALE = 1 / np.sqrt(128)


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def decode(ops, q, cache, tables, ctx, scale=SCALE, num_splits=0):
    ws = ops.decode_workspace(q.shape[1], cache[0].shape[2], num_splits, 128, "cuda")
    out = ops.decode_fp8_block(to_dev_bf16(q), *[dev(a) for a in cache], to_dev_i32(tables),
                               to_dev_i32(ctx), scale, out_dtype=torch.float32,
                               num_splits=num_splits, workspace=ws)
    assert ops.read_error_word(ws) == 0
    return out.double().cpu().numpy()


def check(got, want, mag, tiny, score=64.0, room=0.0):
    """NaN where the definition has NaN, within the bound elsewhere."""
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    err, bound = np.abs(got - want), ref.tolerance(want, mag, tiny, score=score) + room
    assert np.all(err[fine] <= bound[fine]), np.max(err[fine] / bound[fine])


@pytest.mark.parametrize("Hkv", [1, 2, 4, 8])
@pytest.mark.parametrize("lens", [[128], [60], [3000], [70, 500, 1]])
@pytest.mark.parametrize("num_splits", [0, 7])
def test_decode_nan_codes(ops, Hkv, lens, num_splits):
    """A NaN code of K makes every dim of its head's group NaN, one of V that
    dim, whichever piece holds it."""
    rng = np.random.default_rng(Hkv + len(lens))
    ctx = np.array(lens, np.int32)
    NB = int(((ctx + 15) // 16).sum()) + 2
    tables = random_tables(rng, ctx, NB)
    q = normal_bits(rng, (len(lens), 2 * Hkv, 128))
    kc, vc, ks, vs = ref.random_cache(rng, NB, Hkv)
    n = lens[0]
    for at in sorted({0, 17 % n, n // 2, n - 1}):
        page, row = tables[0, at // 16], at % 16
        for which in (0, 1):
            k2, v2 = kc.copy(), vc.copy()
            if which == 0:
                k2[page, row, Hkv - 1, 77] = 0x7F
            else:
                v2[page, 0, 33, row] = 0xFF
            cache = (k2, v2, ks, vs)
            with np.errstate(invalid="ignore"):
                want = ref.attention(q, *cache, tables, ctx, SCALE)
            assert np.isnan(want[0]).any()
            check(decode(ops, q, cache, tables, ctx, num_splits=num_splits), *want)

