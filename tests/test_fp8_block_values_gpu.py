"""Values at the edge of the block-scaled FP8 cache's attention: codes and
query rows that are NaN, infinite, huge or tiny, and where their effect ends."""
import numpy as np
import pytest
import torch

from paged_kv_continuous_gb300.synth import bf16_bits, bf16_to_f64
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


def test_decode_query_rows_of_any_size(ops):
    """Rows whose magnitudes lie far apart and far from 1 (each takes its own
    power of two), elements of one row far apart.  An element of less than
    2^-31 of its row's largest may be off by 2^-39 of that, which moves a score
    by at most that times the sum of the key's magnitudes."""
    rng = np.random.default_rng(10)
    B, Hq, Hkv = 20, 8, 2
    ctx = rng.integers(1, 90, B).astype(np.int32)
    NB = int(((ctx + 15) // 16).sum()) + 2
    tables = random_tables(rng, ctx, NB)
    cache = ref.random_cache(rng, NB, Hkv)
    kk = np.abs(ref.widen(*cache)[0]).sum(-1).max()
    f = bf16_to_f64(normal_bits(rng, (B, Hq, 128)))
    rows = 2.0 ** rng.integers(-60, 60, (B, Hq, 1))
    for spread in (0, 40):
        x = f * 2.0 ** rng.integers(-spread, 1, f.shape)
        for scale, y in ((SCALE, x), (SCALE * 2.0 ** -60, x * 2.0 ** 60),
                         (SCALE * 2.0 ** 60, x * 2.0 ** -60), (SCALE * 2.0 ** -17, x * 2.0 ** 17),
                         (SCALE * 2.0 ** 26, x * 2.0 ** -26), (2.0 ** -40, x * rows)):
            bits = bf16_bits(y.astype(np.float32))
            want, mag, tiny = ref.attention(bits, *cache, tables, ctx, scale)
            top = np.abs(bf16_to_f64(bits)).max(-1, keepdims=True)
            # only rows whose scores stay where a rounding of fp32 is small
            fine = (scale * top * kk < 2000).squeeze(-1)
            move = scale * top * 2.0 ** -39 * kk
            got = decode(ops, bits, cache, tables, ctx, scale)
            bound = ref.tolerance(want, mag, tiny, score=3000.0) + \
                2 * np.expm1(np.minimum(move, 1.0)) * mag
            assert fine.any() and np.all(np.abs(got - want)[fine] <= bound[fine]), scale


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (12, 2), (32, 8)])
def test_decode_query_rows_at_the_ends_of_bf16(ops, Hq, Hkv):
    """The largest and the smallest (subnormal) magnitudes, and rows of zeros."""
    rng = np.random.default_rng(Hq)
    ctx = np.array([40, 200, 17], np.int32)
    tables = random_tables(rng, ctx, 30)
    cache = ref.random_cache(rng, 30, Hkv)
    f = bf16_to_f64(normal_bits(rng, (3, Hq, 128)))
    q = bf16_bits((f * 2.0 ** 120).astype(np.float32))
    q[:, 3, 5] = 0xFF7F  # the largest finite one, negative
    q[:, 1] = bf16_bits((f[:, 1] * 2.0 ** -130).astype(np.float32))
    q[:, 2] = 0
    scale = SCALE * 2.0 ** -120
    want = ref.attention(q, *cache, tables, ctx, scale)
    check(decode(ops, q, cache, tables, ctx, scale), *want, score=512.0)


@pytest.mark.parametrize("Hkv", [1, 2, 4, 8])
@pytest.mark.parametrize("lens", [[1, 40], [128], [3000, 5]])
def test_decode_query_rows_that_are_not_finite(ops, Hkv, lens):
    """A NaN or an infinity in a query row makes that row NaN and no other,
    as in the prefill."""
    rng = np.random.default_rng(11)
    ctx = np.array(lens, np.int32)
    NB = int(((ctx + 15) // 16).sum()) + 2
    tables = random_tables(rng, ctx, NB)
    cache = ref.random_cache(rng, NB, Hkv)
    Hq = 4 * Hkv
    q = normal_bits(rng, (len(lens), Hq, 128))
    good = decode(ops, q, cache, tables, ctx)
    bad = np.zeros((len(lens), Hq), bool)
    for h, d, x in ((0, 7, 0x7FC0), (2, 0, 0x7F80), (Hq - 1, 127, 0xFF80)):
        q[0, h, d] = x
        bad[0, h] = True
    got = decode(ops, q, cache, tables, ctx)
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], good[~bad])
    out = ops.prefill_varlen_fp8_block(
        to_dev_bf16(q), to_dev_i32(np.arange(len(lens) + 1)), *[dev(a) for a in cache],
        to_dev_i32(tables), to_dev_i32(ctx), SCALE, 1, out_dtype=torch.float32)
    assert np.array_equal(np.isnan(out.cpu().numpy()), np.isnan(got))


@pytest.mark.parametrize("Hkv", [1, 2, 4, 8])
def test_scale_arrays_of_layers_in_one_tensor(ops, Hkv):
    """Layers as views of [layers, num_blocks, Hkv] scale tensors with an odd
    number of pages: stored, decoded and prefilled like arrays of their own."""
    rng = np.random.default_rng(Hkv)
    layers, NB, Hq = 5, 13, 2 * Hkv
    ctx = np.array([40, 100], np.int32)
    tables = random_tables(rng, ctx, NB)
    q = normal_bits(rng, (2, Hq, 128))
    k, v = (to_dev_bf16(normal_bits(rng, (2, Hkv, 128))) for _ in range(2))
    td, cd, one = to_dev_i32(tables), to_dev_i32(ctx), to_dev_i32([0, 1, 2])
    ks, vs = (torch.zeros((layers, NB, Hkv), dtype=torch.uint8, device="cuda") for _ in range(2))
    for i in range(layers):
        cache = [dev(a) for a in ref.random_cache(rng, NB, Hkv)]
        ks[i], vs[i] = cache[2], cache[3]
        views = [cache[0].clone(), cache[1].clone(), ks[i], vs[i]]
        outs = []
        for c in (cache, views):
            ops.store_kv_fp8_block(k, v, *c, one, td, cd)
            outs.append(ops.decode_fp8_block(to_dev_bf16(q), *c, td, cd, SCALE))
            outs.append(ops.prefill_varlen_fp8_block(to_dev_bf16(q), one, *c, td, cd, SCALE, 1))
        assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3]), i
        assert all(torch.equal(a, b) for a, b in zip(cache, views))


@pytest.mark.parametrize("seqs", [3, 300])
def test_prefill_context_past_its_table_row(ops, seqs):
    """A context that needs more entries than its table row has, one below its
    chunk and a chunk that ends before it starts: reported, skipped (their rows
    stay as they were), the other sequences attended."""
    rng = np.random.default_rng(seqs)
    cu = np.arange(seqs + 1, dtype=np.int32) * 2
    ctx = rng.integers(2, 33, seqs).astype(np.int32)
    NB = int(((ctx + 15) // 16).sum()) + 2
    tables = random_tables(rng, ctx, NB)
    assert tables.shape[1] == 2
    cache = ref.random_cache(rng, NB, 2)
    q = normal_bits(rng, (2 * seqs, 12, 128))
    args = [to_dev_bf16(q), to_dev_i32(cu), *[dev(a) for a in cache], to_dev_i32(tables)]
    good = ops.prefill_varlen_fp8_block(*args, to_dev_i32(ctx), SCALE, 2,
                                        out_dtype=torch.float32)
    for wrong in (33, 4000, 2 ** 20, 1, -2 ** 31, -2 ** 31 + 1):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        bad = ctx.copy()
        bad[1] = wrong
        out = torch.full((2 * seqs, 12, 128), 7.0, device="cuda")
        ops.prefill_varlen_fp8_block(*args, to_dev_i32(bad), SCALE, 2, out=out, error_flags=err)
        assert int(err.item()) & ops.DEVERR_SHAPE, wrong
        assert torch.all(out[2:4] == 7.0)
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:])
    # cu_seqlens that fall, at the last sequence
    err.zero_()
    fall = cu.copy()
    fall[-1] = fall[-2] - 1
    args[1] = to_dev_i32(fall)
    out.fill_(7.0)
    ops.prefill_varlen_fp8_block(*args, to_dev_i32(ctx), SCALE, 2, out=out, error_flags=err)
    assert int(err.item()) & ops.DEVERR_SHAPE
    assert torch.equal(out[:-2], good[:-2]) and torch.all(out[-2:] == 7.0)
