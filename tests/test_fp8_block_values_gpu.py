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



def prefill(ops, q, cu, cache, tables, ctx, scale=SCALE):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ops.prefill_varlen_fp8_block(
        to_dev_bf16(q), to_dev_i32(cu), *[dev(a) for a in cache], to_dev_i32(tables),
        to_dev_i32(ctx), scale, int(np.diff(cu).max()), out_dtype=torch.float32, error_flags=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out.double().cpu().numpy()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (8, 1), (12, 2), (16, 8)])
def test_prefill_nan_codes_reach_the_rows_that_see_them(ops, Hq, Hkv):
    """A NaN code makes NaN of the rows at or after its position alone: of K
    every dim of its head's group, of V that dim.  In the prefix, at the start,
    inside and at the end of a chunk, several in one tile."""
    rng = np.random.default_rng(Hq)
    spec = [(150, 70), (40, 0), (1, 30)]
    ql = np.array([a for a, _ in spec])
    ctx = np.array([a + b for a, b in spec], np.int32)
    cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    NB = int(((ctx + 15) // 16).sum()) + 2
    tables = random_tables(rng, ctx, NB)
    q = normal_bits(rng, (int(cu[-1]), Hq, 128))
    kc, vc, ks, vs = ref.random_cache(rng, NB, Hkv)
    good = prefill(ops, q, cu, (kc, vc, ks, vs), tables, ctx)
    for spots in ([(0, 3)], [(0, 70)], [(0, 100), (0, 101), (0, 130)], [(0, 219)], [(0, 160)],
                  [(1, 0)], [(1, 39), (1, 16)], [(2, 30)], [(2, 5), (0, 127), (0, 128)]):
        k2, v2 = kc.copy(), vc.copy()
        k3, v3 = kc.copy(), vc.copy()
        for i, (s, at) in enumerate(spots):
            page, row = tables[s, at // 16], at % 16
            k2[page, row, 0, 77] = 0xFF
            v3[page, Hkv - 1, (33 + 40 * i) % 128, row] = 0x7F + 128 * (i & 1)
            v3[page, 0, 127, row] = 0x7F
        for cache in ((k2, v2, ks, vs), (k3, v3, ks, vs)):
            with np.errstate(invalid="ignore"):
                want, mag, tiny = ref.attention(q, *cache, tables, ctx, SCALE, cu)
            got = prefill(ops, q, cu, cache, tables, ctx)
            check(got, want, mag, tiny)
            assert np.array_equal(got[~np.isnan(got)], good[~np.isnan(got)])
