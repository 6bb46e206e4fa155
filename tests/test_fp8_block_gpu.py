"""GPU parity of the block-scaled FP8 cache.

pa_store_kv_fp8_block must leave the reference's bytes and scales in the whole
pool; pa_decode_fp8_block is held to an elementwise bound that follows from
the rounding of its weights (fp8_block_reference.tolerance)."""
import numpy as np
import pytest
import torch

from paged_kv_continuous_gb300.synth import BF16_NAN, bf16_bits
from tests import fp8_block_reference as ref
from tests.helpers import normal_bits, random_tables, to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_cache(c):
    return [dev(a) for a in c]


def same_bytes(got, want, what=""):
    torch.cuda.synchronize()
    for name, g, w in zip(("k codes", "v codes", "k scales", "v scales"), got, want):
        g = g.cpu().numpy()
        bad = np.argwhere(g != w)
        assert not len(bad), f"{what} {name}: {len(bad)} differ, first at {bad[0]}: " \
                             f"{g[tuple(bad[0])]:#x} for {w[tuple(bad[0])]:#x}"


def chunks(rng, spec, NB, hkv, extra_rows=0):
    """cu, ctx, tables and rows of the (q_len, prefix) pairs of ``spec``."""
    ql = np.array([q for q, _ in spec])
    ctx = np.array([q + p for q, p in spec], np.int32)
    cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    tables = random_tables(rng, np.maximum(ctx, 1), NB)
    T = int(cu[-1]) + extra_rows
    amp = 2.0 ** rng.integers(-6, 7, (T, 1, 1))
    k, v = (bf16_bits((rng.standard_normal((T, hkv, 128)) * amp).astype(np.float32))
            for _ in range(2))
    return cu, ctx, tables, k, v


def run_store(ops, k, v, cache, cu, tables, ctx, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = dev_cache(cache)
    ops.store_kv_fp8_block(to_dev_bf16(k), to_dev_bf16(v), *d, to_dev_i32(cu), to_dev_i32(tables),
                           to_dev_i32(ctx), error_flags=err, **kw)
    torch.cuda.synchronize()
    return d, int(err.item())


SPECS = {
    "one token": [(1, 0)],
    "decode step": [(1, p) for p in (0, 1, 14, 15, 16, 17, 31, 32, 100, 271)],
    "chunks": [(16, 0), (15, 1), (17, 15), (100, 7), (33, 16), (0, 5), (0, 0), (64, 0)],
    "ragged": [(2, 15), (18, 14), (31, 31), (1, 63), (0, 16), (5, 3)],
}


@pytest.mark.parametrize("hkv", [1, 2, 3, 8])
@pytest.mark.parametrize("name", list(SPECS))
def test_store_bytes(ops, name, hkv):
    rng = np.random.default_rng(10 * hkv + len(name))
    cu, ctx, tables, k, v = chunks(rng, SPECS[name], 80, hkv)
    cache = ref.random_cache(rng, 80, hkv)
    got, err = run_store(ops, k, v, cache, cu, tables, ctx)
    want = [a.copy() for a in cache]
    ref.store(k, v, *want, cu, tables, ctx)
    assert err == 0
    same_bytes(got, want, name)


def test_store_special_values(ops):
    """Zero rows, infinities, NaN, the largest and the smallest bf16 values,
    in first and in later rows of a block."""
    rng = np.random.default_rng(3)
    spec = [(16, 0), (16, 0), (16, 0), (8, 8), (8, 8), (8, 8), (20, 0), (1, 0)]
    cu, ctx, tables, k, v = chunks(rng, spec, 40, 2)
    special = bf16_bits(np.array([np.inf, -np.inf, 3.3e38, -3.3e38, 1e-38, -1e-40, 0.0, 448.0,
                                  449.0, 2.0 ** 40 * 448, 2.0 ** -41], np.float32))
    for x in (k, v):
        x[0:16] = 0
        x[16:32, 0] = special[0]
        x[33, 1, ::7] = BF16_NAN
        x[50, :, 5] = special[1]
        for i, s in enumerate(special):
            x[70 + i % 12, i % 2, 11 * i % 128] = s
        x[int(cu[-2]), 0, :len(special)] = special
    cache = ref.random_cache(rng, 40, 2, e_lo=-40, e_hi=40)
    got, err = run_store(ops, k, v, cache, cu, tables, ctx)
    want = [a.copy() for a in cache]
    ref.store(k, v, *want, cu, tables, ctx)
    assert err == 0
    # a NaN keeps a NaN code; its sign is not part of the definition
    got = [g.cpu().numpy() for g in got]
    for i in (0, 1):
        for a in (got[i], want[i]):
            a[(a & 127) == 127] = 127
    same_bytes([torch.from_numpy(g) for g in got], want)


def test_store_appends_token_by_token(ops):
    """Sixty tokens of growing and shrinking size, one call each, in place."""
    rng = np.random.default_rng(4)
    n, hkv = 60, 2
    cu, ctx, tables, k, v = chunks(rng, [(n, 0), (n, 9)], 16, hkv)
    cache = ref.random_cache(rng, 16, hkv)
    d, want = dev_cache(cache), [a.copy() for a in cache]
    kd, vd = to_dev_bf16(k), to_dev_bf16(v)
    td, cu1 = to_dev_i32(tables), np.array([0, 1, 2], np.int32)
    for t in range(n):
        rows = [t, n + t]
        now = np.array([t + 1, 9 + t + 1], np.int32)
        ops.store_kv_fp8_block(kd[rows], vd[rows], *d, to_dev_i32(cu1), td, to_dev_i32(now))
        ref.store(k[rows], v[rows], *want, cu1, tables, now)
    same_bytes(d, want)


@pytest.mark.parametrize("shift", [0, 1, 2])
def test_store_strides(ops, shift):
    """Views of a fused QKV row (token stride past the heads), an odd base
    (scalar loads) and heads in another order of memory."""
    rng = np.random.default_rng(5)
    cu, ctx, tables, k, v = chunks(rng, SPECS["ragged"], 40, 2)
    T = k.shape[0]
    if shift < 2:
        buf = torch.zeros(T * 777 + 8, dtype=torch.bfloat16, device="cuda")
        kd = buf.as_strided((T, 2, 128), (777 - shift, 129 if shift else 128, 1), shift)
        vd = buf.as_strided((T, 2, 128), (777 - shift, 129 if shift else 128, 1), 300 + shift)
    else:
        kd, vd = (torch.empty(2, T, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
                  for _ in range(2))
    kd.copy_(to_dev_bf16(k))
    vd.copy_(to_dev_bf16(v))
    cache = ref.random_cache(rng, 40, 2)
    d, want = dev_cache(cache), [a.copy() for a in cache]
    ops.store_kv_fp8_block(kd, vd, *d, to_dev_i32(cu), to_dev_i32(tables), to_dev_i32(ctx))
    ref.store(k, v, *want, cu, tables, ctx)
    same_bytes(d, want)


def test_store_many_sequences_and_rows_behind(ops):
    """1500 sequences of 0 to 3 tokens, and rows behind the last sequence
    that must not be read into the pool."""
    rng = np.random.default_rng(6)
    spec = [(int(rng.integers(0, 4)), int(rng.integers(0, 20))) for _ in range(1500)]
    cu, ctx, tables, k, v = chunks(rng, spec, 4000, 1, extra_rows=40)
    cache = ref.random_cache(rng, 4000, 1)
    got, err = run_store(ops, k, v, cache, cu, tables, ctx)
    want = [a.copy() for a in cache]
    ref.store(k, v, *want, cu, tables, ctx)
    assert err == 0
    same_bytes(got, want)


def test_store_reports_and_skips(ops):
    """A table entry outside the pool, a context shorter than its chunk, a
    chunk past the table row and one past the rows: reported, skipped, and
    the others stored."""
    rng = np.random.default_rng(7)
    spec = [(20, 0), (20, 0), (20, 0), (20, 0), (20, 20)]
    cu, ctx, tables, k, v = chunks(rng, spec, 30, 2)
    cache = ref.random_cache(rng, 30, 2)
    good = [a.copy() for a in cache]
    for s in (0, 4):
        ref.store(k[cu[s]:cu[s + 1]], v[cu[s]:cu[s + 1]], *good, [0, 20], tables[s:s + 1],
                  ctx[s:s + 1])
    bad_tables, bad_ctx = tables.copy(), ctx.copy()
    bad_tables[1, :2] = (-1, 30)
    bad_ctx[2] = 19
    bad_ctx[3] = 16 * tables.shape[1] + 20  # first page past the row
    got, err = run_store(ops, k, v, cache, cu, bad_tables, bad_ctx)
    assert err == ops.DEVERR_BLOCK_INDEX | ops.DEVERR_SHAPE
    same_bytes(got, good)
    # rows past k / v
    bad_cu = cu.copy()
    bad_cu[5] = 300
    got, err = run_store(ops, k, v, cache, bad_cu, tables, ctx)
    assert err == ops.DEVERR_SHAPE
    want = [a.copy() for a in cache]
    ref.store(k[:80], v[:80], *want, cu[:5], tables[:4], ctx[:4])
    same_bytes(got, want)


# ---- decode -----------------------------------------------------------------

def check_decode(ops, q, cache, tables, ctx, scale, num_splits=0, out_dtype=torch.float32,
                 score=64.0):
    ws = ops.decode_workspace(q.shape[1], cache[0].shape[2], num_splits, 128, "cuda")
    out = ops.decode_fp8_block(to_dev_bf16(q), *dev_cache(cache), to_dev_i32(tables),
                               to_dev_i32(ctx), scale, out_dtype=out_dtype,
                               num_splits=num_splits, workspace=ws)
    torch.cuda.synchronize()
    assert ops.read_error_word(ws) == 0
    want, mag, tiny = ref.attention(q, *cache, tables, ctx, scale)
    got = out.double().cpu().numpy()
    bound = ref.tolerance(want, mag, tiny, out_dtype == torch.bfloat16, score)
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    assert np.all(err <= bound), f"largest error over bound {np.max(err / bound):.3g} " \
                                 f"({np.max(err):.3g})"
    return out


SCALE = 1 / np.sqrt(128)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (12, 2), (2, 2), (14, 2), (20, 4), (32, 8),
                                    (64, 8)])
@pytest.mark.parametrize("num_splits", [0, 5])
def test_decode_shapes(ops, Hq, Hkv, num_splits):
    rng = np.random.default_rng(100 + Hq + Hkv + num_splits)
    ctx = np.array([1, 0, 16, 17, 700, 33, 255, 1, 0, 90], np.int32)
    tables = random_tables(rng, ctx, 120)
    check_decode(ops, normal_bits(rng, (10, Hq, 128)), ref.random_cache(rng, 120, Hkv), tables,
                 ctx, SCALE, num_splits)


@pytest.mark.parametrize("Hq,Hkv", [(12, 2), (32, 8)])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.0])
def test_decode_scales_and_bf16(ops, Hq, Hkv, scale):
    """Softmax scales of either sign and zero; bf16 output."""
    rng = np.random.default_rng(200 + Hq)
    ctx = np.array([300, 5, 64], np.int32)
    tables = random_tables(rng, ctx, 40)
    cache = ref.random_cache(rng, 40, Hkv)
    q = normal_bits(rng, (3, Hq, 128))
    check_decode(ops, q, cache, tables, ctx, scale, score=512.0)
    check_decode(ops, q, cache, tables, ctx, scale, out_dtype=torch.bfloat16, score=512.0)


def test_decode_single_long_sequence(ops):
    """One long context over every split (in-kernel merge and merge kernel)."""
    rng = np.random.default_rng(300)
    for Hq, Hkv in ((6, 1), (8, 4)):
        ctx = np.array([20011], np.int32)
        tables = random_tables(rng, ctx, 1300)
        check_decode(ops, normal_bits(rng, (1, Hq, 128)), ref.random_cache(rng, 1300, Hkv),
                     tables, ctx, SCALE)


@pytest.mark.parametrize("spread", [10, 40])
def test_decode_scales_far_apart(ops, spread):
    """V scales of a sequence's blocks far apart: blocks of large values whose
    keys score low beside blocks of small values that hold the weight.  K
    scales follow, so that the scores stay moderate."""
    rng = np.random.default_rng(400 + spread)
    n = 200
    ctx = np.array([n], np.int32)
    tables = random_tables(rng, ctx, 20)
    kc, vc, ks, vs = ref.random_cache(rng, 20, 1)
    vs[:] = rng.integers(-spread, spread + 1, vs.shape) + ref.BIAS
    q = normal_bits(rng, (1, 4, 128))
    check_decode(ops, q, (kc, vc, ks, vs), tables, ctx, SCALE)
    # the weight on a block of the smallest V scale, the rest with large ones:
    # its own relative error has to stay an f16 rounding.  Keys of block 0
    # point along q, the others against it.
    q[:] = bf16_bits(np.ones(128, np.float32))
    kc[:] = 0x80 | 0x38  # -1
    kc[tables[0, 0]] = 0x38
    ks[:] = ref.BIAS
    vs[:] = ref.BIAS + spread // 2
    vs[tables[0, 0]] = ref.BIAS - spread // 2
    out = ops.decode_fp8_block(to_dev_bf16(q), *dev_cache((kc, vc, ks, vs)), to_dev_i32(tables),
                               to_dev_i32(ctx), 1.0, out_dtype=torch.float32)
    torch.cuda.synchronize()
    want, mag, _ = ref.attention(q, kc, vc, ks, vs, tables, ctx, 1.0)
    # scores +-185 (base 2): the other keys weigh 2^-369 2^spread, nothing
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= mag * (2.0 ** -11 + 8 * 185 * 2.0 ** -24 + 2.0 ** -16))


def test_decode_ignores_what_no_key_holds(ops):
    """Stale NaN codes past the last key, blocks no table names and scale
    bytes of any value there; table entries past the context."""
    rng = np.random.default_rng(500)
    ctx = np.array([1, 17, 100], np.int32)
    tables = random_tables(rng, ctx, 30)
    kc, vc, ks, vs = ref.random_cache(rng, 30, 2)
    live = np.zeros((30, 16), bool)
    for s, n in enumerate(ctx):
        for j in range(n):
            live[tables[s, j // 16], j % 16] = True
    kc[~live] = 0x7F
    vc.transpose(0, 3, 1, 2)[~live] = 0xFF
    dead = ~live.any(1)
    ks[dead], vs[dead] = 255, 0
    tables[tables == -1] = 2 ** 30
    check_decode(ops, normal_bits(rng, (3, 12, 128)), (kc, vc, ks, vs), tables, ctx, SCALE)


def test_decode_clamps_scale_bytes(ops):
    """Scale bytes outside the span read as its ends."""
    rng = np.random.default_rng(501)
    ctx = np.array([40], np.int32)
    tables = random_tables(rng, ctx, 4)
    kc, vc, ks, vs = ref.random_cache(rng, 4, 1)
    ks[:] = 3
    vs[tables[0, :2], 0] = (0, 255)
    check_decode(ops, normal_bits(rng, (1, 2, 128)), (kc, vc, ks, vs), tables, ctx, SCALE)


def test_decode_bad_table_entry_is_reported(ops):
    rng = np.random.default_rng(502)
    ctx = np.array([40, 20], np.int32)
    tables = random_tables(rng, ctx, 8)
    tables[0, 1] = 8
    cache = ref.random_cache(rng, 8, 2)
    q = normal_bits(rng, (2, 12, 128))
    ws = ops.decode_workspace(12, 2, 0, 128, "cuda")
    out = ops.decode_fp8_block(to_dev_bf16(q), *dev_cache(cache), to_dev_i32(tables),
                               to_dev_i32(ctx), SCALE, out_dtype=torch.float32, workspace=ws)
    assert ops.read_error_word(ws) == ops.DEVERR_BLOCK_INDEX
    want, mag, tiny = ref.attention(q[1:], *cache, tables[1:], ctx[1:], SCALE)
    err = np.abs(out[1:].double().cpu().numpy() - want)
    assert np.all(err <= ref.tolerance(want, mag, tiny))


def test_decode_many_sequences(ops):
    """More sequences than a CTA has threads, one to three blocks each."""
    rng = np.random.default_rng(503)
    ctx = rng.integers(0, 41, 400).astype(np.int32)
    tables = random_tables(rng, np.maximum(ctx, 1), 1300)
    for Hq, Hkv in ((2, 1), (8, 4)):
        check_decode(ops, normal_bits(rng, (400, Hq, 128)), ref.random_cache(rng, 1300, Hkv),
                     tables, ctx, SCALE)


@pytest.mark.parametrize("Hkv", [1, 2, 4, 8])
@pytest.mark.parametrize("order", ["short first", "long first", "mixed", "none between"])
def test_decode_short_sequences_beside_long(ops, order, Hkv):
    """Runs of short sequences beside long ones, whose piece ends weigh in the
    division of the work: bounds that fall between, at the start and at the end
    of sequences, empty sequences among them."""
    rng = np.random.default_rng(900 + Hkv)
    short, long = rng.integers(1, 40, 70), rng.integers(900, 2500, 5)
    ctx = {"short first": np.concatenate([short, long]),
           "long first": np.concatenate([long, short]),
           "mixed": rng.permutation(np.concatenate([short, long])),
           "none between": np.concatenate([[0, 0], short * (rng.random(70) < 0.6), long, [0],
                                           short[:9], [0]])}[order].astype(np.int32)
    tables = random_tables(rng, np.maximum(ctx, 1), 1200)
    Hq = 3 * Hkv
    check_decode(ops, normal_bits(rng, (len(ctx), Hq, 128)), ref.random_cache(rng, 1200, Hkv),
                 tables, ctx, SCALE)


@pytest.mark.parametrize("batch", [151, 152, 153, 160, 352, 353, 700])
def test_decode_one_block_sequences(ops, batch):
    """As many sequences as splits and a few more, and as many as a block has
    threads and one more; one or two blocks each."""
    rng = np.random.default_rng(950 + batch)
    ctx = rng.integers(1, 18, batch).astype(np.int32)
    tables = random_tables(rng, ctx, 1500)
    check_decode(ops, normal_bits(rng, (batch, 4, 128)), ref.random_cache(rng, 1500, 2), tables,
                 ctx, SCALE)


@pytest.mark.parametrize("Hkv", [1, 2, 4, 8])
def test_decode_default_splits_over_batches(ops, Hkv):
    """The splits in use with the default count, from one block to thousands,
    alone and beside others."""
    rng = np.random.default_rng(504 + Hkv)
    for lens in ([1], [20], [300], [5000], [17, 16, 4], [900] * 5, [60, 2000, 1, 0, 0, 33] * 4,
                 [16] * 21):
        ctx = np.array(lens, np.int32)
        NB = int(((ctx + 15) // 16).sum()) + 2
        tables = random_tables(rng, np.maximum(ctx, 1), NB + len(lens))
        check_decode(ops, normal_bits(rng, (len(lens), 4 * Hkv, 128)),
                     ref.random_cache(rng, NB + len(lens), Hkv), tables, ctx, SCALE)


def test_pools_past_four_gigabytes(ops):
    """Pages at the far end of pools of 5 GB each: offsets need 64 bits in the
    store, the decode and the prefill."""
    rng = np.random.default_rng(505)
    NB, Hkv, Hq = 1_250_000, 2, 12
    spec = [(40, 0), (17, 30)]
    cu, ctx, tables, k, v = chunks(rng, spec, 10, Hkv)
    cache = ref.random_cache(rng, 10, Hkv)
    pools = ops.fp8_block_pools(NB, Hkv, device="cuda")
    far = NB - 10
    for pool, small in zip(pools, dev_cache(cache)):
        pool[far:] = small
    td = to_dev_i32(np.where(tables >= 0, tables + far, tables))
    args = [to_dev_i32(cu), td, to_dev_i32(ctx)]
    ops.store_kv_fp8_block(to_dev_bf16(k), to_dev_bf16(v), *pools, *args)
    want = [a.copy() for a in cache]
    ref.store(k, v, *want, cu, tables, ctx)
    same_bytes([p[far:] for p in pools], want)
    q = normal_bits(rng, (2, Hq, 128))
    out = ops.decode_fp8_block(to_dev_bf16(q), *pools, td, args[2], SCALE,
                               out_dtype=torch.float32)
    w, mag, tiny = ref.attention(q, *want, tables, ctx, SCALE)
    assert np.all(np.abs(out.double().cpu().numpy() - w) <= ref.tolerance(w, mag, tiny))
    q = normal_bits(rng, (int(cu[-1]), Hq, 128))
    out = ops.prefill_varlen_fp8_block(to_dev_bf16(q), args[0], *pools, td, args[2], SCALE, 40,
                                       out_dtype=torch.float32)
    w, mag, tiny = ref.attention(q, *want, tables, ctx, SCALE, cu)
    assert np.all(np.abs(out.double().cpu().numpy() - w) <= ref.tolerance(w, mag, tiny))


def test_store_many_heads(ops):
    rng = np.random.default_rng(506)
    cu, ctx, tables, k, v = chunks(rng, SPECS["ragged"], 30, 64)
    cache = ref.random_cache(rng, 30, 64)
    got, err = run_store(ops, k, v, cache, cu, tables, ctx)
    want = [a.copy() for a in cache]
    ref.store(k, v, *want, cu, tables, ctx)
    assert err == 0
    same_bytes(got, want)


def test_strided_tables(ops):
    """Tables as columns of a wider buffer; a view whose last row has no room
    for its stride is refused."""
    rng = np.random.default_rng(507)
    ctx = np.array([40, 17], np.int32)
    tables = random_tables(rng, ctx, 12)
    cache = ref.random_cache(rng, 12, 2)
    q = normal_bits(rng, (2, 12, 128))
    wide = torch.full((2, 9), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[:, :3] = to_dev_i32(tables)
    out = ops.decode_fp8_block(to_dev_bf16(q), *dev_cache(cache), wide[:, :3], to_dev_i32(ctx),
                               SCALE, out_dtype=torch.float32)
    w, mag, tiny = ref.attention(q, *cache, tables, ctx, SCALE)
    assert np.all(np.abs(out.double().cpu().numpy() - w) <= ref.tolerance(w, mag, tiny))
    with pytest.raises(ops.PagedAttentionError, match="whole stride"):
        ops.decode_fp8_block(to_dev_bf16(q), *dev_cache(cache), wide[:, 6:], to_dev_i32(ctx),
                             SCALE)


# ---- together ---------------------------------------------------------------

def test_steps_of_store_and_decode(ops):
    """A prompt chunk and twenty decode steps, store and decode chained with
    programmatic launches, eager and as one replayed graph: the pool's bytes
    and the outputs against the reference, and both runs the same bits."""
    rng = np.random.default_rng(600)
    B, Hq, Hkv, NB, steps = 5, 12, 2, 40, 20
    pre = np.array([3, 16, 31, 64, 100])
    cu, ctx, tables, k, v = chunks(rng, [(p, 0) for p in pre], NB, Hkv)
    tables = random_tables(rng, pre + steps, NB)
    cache = ref.random_cache(rng, NB, Hkv)
    d, want = dev_cache(cache), [a.copy() for a in cache]
    td = to_dev_i32(tables)
    ops.store_kv_fp8_block(to_dev_bf16(k), to_dev_bf16(v), *d, to_dev_i32(cu), td,
                           to_dev_i32(pre))
    ref.store(k, v, *want, cu, tables, pre)
    same_bytes(d, want, "prompt")
    start = [a.clone() for a in d]
    nk, nv = (bf16_bits(rng.standard_normal((steps, B, Hkv, 128)).astype(np.float32))
              for _ in range(2))
    q = normal_bits(rng, (steps, B, Hq, 128))
    kd, vd, qd = to_dev_bf16(nk[0]), to_dev_bf16(nv[0]), to_dev_bf16(q[0])
    ctx_d, one = to_dev_i32(pre), to_dev_i32(np.arange(B + 1))
    out = torch.empty((B, Hq, 128), dtype=torch.float32, device="cuda")
    rows = [to_dev_bf16(a) for a in (nk, nv, q)]
    store = ops.StoreKvFp8BlockCall(kd, vd, *d, one, td, ctx_d, pdl=True)
    decode = ops.DecodeFp8BlockCall(qd, *d, td, ctx_d, SCALE, out, pdl=True)

    def load(t):
        for to, x in zip((kd, vd, qd), rows):
            to.copy_(x[t])
        ctx_d.copy_(to_dev_i32(pre + t + 1))

    eager = []
    for t in range(steps):
        load(t)
        store()
        decode()
        eager.append(out.clone())
        now = (pre + t + 1).astype(np.int32)
        ref.store(nk[t], nv[t], *want, np.arange(B + 1), tables, now)
        w, mag, tiny = ref.attention(q[t], *want, tables, now, SCALE)
        err = np.abs(eager[-1].double().cpu().numpy() - w)
        assert np.all(err <= ref.tolerance(w, mag, tiny)), t
    same_bytes(d, want, "steps")
    assert ops.read_error_word(decode.workspace) == 0
    for a, b in zip(d, start):
        a.copy_(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            store()
            decode()
    torch.cuda.current_stream().wait_stream(side)
    for t in range(steps):
        load(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[t]), t
    same_bytes(d, want, "replayed")


def test_calls_on_another_stream(ops):
    """Both calls on a side stream, with work before them that they must
    wait for."""
    rng = np.random.default_rng(601)
    cu, ctx, tables, k, v = chunks(rng, [(50, 0), (7, 30)], 12, 2)
    cache = ref.random_cache(rng, 12, 2)
    q = normal_bits(rng, (2, 12, 128))
    d, want = dev_cache(cache), [a.copy() for a in cache]
    args = [to_dev_i32(cu), to_dev_i32(tables), to_dev_i32(ctx)]
    kd, vd, qd = to_dev_bf16(k), to_dev_bf16(v), to_dev_bf16(q)
    late = torch.zeros_like(kd)
    ws = ops.decode_workspace(12, 2, 0, 128, "cuda")
    out = torch.empty((2, 12, 128), dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        late.copy_(kd)
        ops.store_kv_fp8_block(late, vd, *d, *args)
        ops.decode_fp8_block(qd, *d, args[1], args[2], SCALE, out=out, workspace=ws)
    side.synchronize()
    ref.store(k, v, *want, cu, tables, ctx)
    same_bytes(d, want)
    w, mag, tiny = ref.attention(q, *want, tables, ctx, SCALE)
    assert np.all(np.abs(out.double().cpu().numpy() - w) <= ref.tolerance(w, mag, tiny))


def test_two_calls_at_once(ops):
    """Two decode calls in flight on two streams, each with its own workspace
    and output, give what each gives alone."""
    rng = np.random.default_rng(602)
    sets = []
    for n in (9000, 5):
        ctx = rng.integers(1, n, 6).astype(np.int32)
        tables = random_tables(rng, ctx, 3500)
        cache = dev_cache(ref.random_cache(rng, 3500, 2))
        out = torch.empty((6, 12, 128), dtype=torch.float32, device="cuda")
        call = ops.DecodeFp8BlockCall(to_dev_bf16(normal_bits(rng, (6, 12, 128))), *cache,
                                      to_dev_i32(tables), to_dev_i32(ctx), SCALE, out)
        alone = call().clone()
        sets.append((call, alone))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for (call, _), s in zip(sets, streams):
            call(s)
    torch.cuda.synchronize()
    for call, alone in sets:
        assert torch.equal(call.out, alone)
        assert ops.read_error_word(call.workspace) == 0
