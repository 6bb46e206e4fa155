"""GPU parity of pa_prefill_fp8_block against the float64 reference, held to
the bound that follows from the rounding of its weights
(fp8_block_reference.tolerance)."""
import numpy as np
import pytest
import torch

from paged_kv_continuous_gb300.synth import bf16_bits
from tests import fp8_block_reference as ref
from tests.helpers import normal_bits, random_tables, to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu
SCALE = 1 / np.sqrt(128)


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


def case(rng, spec, Hq, Hkv, extra_blocks=3, **kw):
    ql = np.array([q for q, _ in spec])
    ctx = np.array([q + p for q, p in spec], np.int32)
    cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    NB = int(((ctx + 15) // 16).sum()) + extra_blocks
    return normal_bits(rng, (int(cu[-1]), Hq, 128)), cu, ref.random_cache(rng, NB, Hkv, **kw), \
        random_tables(rng, np.maximum(ctx, 1), NB), ctx


def run(ops, q, cu, cache, tables, ctx, scale=SCALE, dtype=torch.float32, max_q=None):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ops.prefill_varlen_fp8_block(
        to_dev_bf16(q), to_dev_i32(cu), *[torch.from_numpy(a).cuda() for a in cache],
        to_dev_i32(tables), to_dev_i32(ctx), scale,
        int(np.diff(cu).max()) if max_q is None else max_q, out_dtype=dtype, error_flags=err)
    torch.cuda.synchronize()
    return out, int(err.item())


def check(ops, q, cu, cache, tables, ctx, scale=SCALE, dtype=torch.float32, score=64.0, **kw):
    out, err = run(ops, q, cu, cache, tables, ctx, scale, dtype, **kw)
    assert err == 0
    want, mag, tiny = ref.attention(q, *cache, tables, ctx, scale, cu)
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    e = np.abs(got - want)
    bound = ref.tolerance(want, mag, tiny, dtype == torch.bfloat16, score)
    assert np.all(e <= bound), f"over the bound: {np.max(e / bound):.3g} ({np.max(e):.3g})"
    return out


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (6, 2), (4, 1), (5, 1), (12, 2), (7, 1),
                                    (64, 8), (8, 4)])
def test_shapes(ops, Hq, Hkv):
    """Group sizes 1 to 8; chunks that start and end inside pages and tiles,
    single tokens, empty chunks, prefixes of zero to several tiles."""
    rng = np.random.default_rng(Hq * 10 + Hkv)
    spec = [(1, 0), (17, 0), (0, 5), (64, 64), (33, 31), (1, 200), (70, 129), (0, 0)]
    check(ops, *case(rng, spec, Hq, Hkv))


def test_long_prefix_and_chunk(ops):
    rng = np.random.default_rng(1)
    check(ops, *case(rng, [(40, 3000), (130, 1111), (1, 2047)], 12, 2))


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.0, 1e-38])
def test_scales(ops, scale):
    rng = np.random.default_rng(2)
    c = case(rng, [(50, 30), (3, 100)], 12, 2)
    check(ops, *c, scale=scale, score=512.0)
    check(ops, *c, scale=scale, dtype=torch.bfloat16, score=512.0)


@pytest.mark.parametrize("spread", [10, 40])
def test_scales_far_apart(ops, spread):
    """V scales of a sequence's blocks far apart; and all weight on a block of
    the smallest V scale beside blocks of large ones."""
    rng = np.random.default_rng(3 + spread)
    q, cu, (kc, vc, ks, vs), tables, ctx = case(rng, [(30, 170)], 4, 1)
    vs[:] = rng.integers(-spread, spread + 1, vs.shape) + ref.BIAS
    check(ops, q, cu, (kc, vc, ks, vs), tables, ctx)
    q[:] = bf16_bits(np.ones(128, np.float32))
    kc[:] = 0x80 | 0x38  # -1
    kc[tables[0, 0]] = 0x38
    ks[:] = ref.BIAS
    vs[:] = ref.BIAS + spread // 2
    vs[tables[0, 0]] = ref.BIAS - spread // 2
    out, err = run(ops, q, cu, (kc, vc, ks, vs), tables, ctx, 1.0)
    want, mag, _ = ref.attention(q, kc, vc, ks, vs, tables, ctx, 1.0, cu)
    e = np.abs(out.double().cpu().numpy() - want)
    assert err == 0
    assert np.all(e <= mag * (2.0 ** -11 + 8 * 185 * 2.0 ** -24 + 2.0 ** -16))


def test_query_rows_of_any_size(ops):
    """Rows whose magnitudes lie far apart and far from 1 (each takes its own
    scale), elements of one row far apart: an element below 2^-11 of the row's
    largest may be off by 2^-10 where the largest is 224 or more, so by at most
    2^-17 of it, which moves a score by at most that times the sum of the key's
    magnitudes, and a weight by that in base e."""
    rng = np.random.default_rng(10)
    q, cu, cache, tables, ctx = case(rng, [(40, 60)], 4, 1)
    kk = np.abs(ref.widen(*cache)[0]).sum(-1).max()
    f = ref.bf16_to_f64(q)
    rows = 2.0 ** rng.integers(-60, 60, (40, 4, 1))
    for spread in (0, 16):
        x = f * 2.0 ** rng.integers(-spread, 1, f.shape)
        for scale, y in ((SCALE, x), (SCALE * 2.0 ** -60, x * 2.0 ** 60), (2.0 ** -40, x * rows)):
            bits = bf16_bits(y.astype(np.float32))
            out, err = run(ops, bits, cu, cache, tables, ctx, scale)
            assert err == 0
            want, mag, tiny = ref.attention(bits, *cache, tables, ctx, scale, cu)
            top = np.abs(ref.bf16_to_f64(bits)).max(-1, keepdims=True)
            move = scale * top * 2.0 ** -17 * kk
            # only rows whose scores stay where a rounding of fp32 is small
            fine = (scale * top * kk < 2000).squeeze(-1)
            bound = ref.tolerance(want, mag, tiny, score=3000.0) + 2 * np.expm1(np.minimum(move, 1.0)) * mag
            e = np.abs(out.double().cpu().numpy() - want)
            assert fine.any() and np.all(e[fine] <= bound[fine])


def test_query_rows_that_are_not_finite(ops):
    """A NaN or an infinity in a query row makes that row NaN and no other."""
    rng = np.random.default_rng(11)
    q, cu, cache, tables, ctx = case(rng, [(30, 40)], 4, 1)
    good, _ = run(ops, q, cu, cache, tables, ctx)
    q[3, 1, 7] = 0x7FC0
    q[9, 0, 0] = 0x7F80
    q[20, 3, 127] = 0xFF80
    out, err = run(ops, q, cu, cache, tables, ctx)
    bad = torch.zeros(30, 4, dtype=torch.bool, device="cuda")
    for i, h in ((3, 1), (9, 0), (20, 3)):
        bad[i, h] = True
    assert err == 0
    assert torch.all(torch.isnan(out[bad])) and torch.equal(out[~bad], good[~bad])


def test_ignores_what_no_key_holds(ops):
    """Stale NaN codes past the last key, unused blocks and table entries."""
    rng = np.random.default_rng(4)
    q, cu, (kc, vc, ks, vs), tables, ctx = case(rng, [(5, 0), (20, 13), (1, 99)], 12, 2)
    live = np.zeros(kc.shape[:2], bool)
    for s, n in enumerate(ctx):
        for j in range(n):
            live[tables[s, j // 16], j % 16] = True
    kc[~live] = 0x7F
    vc.transpose(0, 3, 1, 2)[~live] = 0xFF
    dead = ~live.any(1)
    ks[dead], vs[dead] = 255, 0
    tables[tables == -1] = 2 ** 30
    check(ops, q, cu, (kc, vc, ks, vs), tables, ctx)


def test_rows_behind_the_last_sequence_stay(ops):
    rng = np.random.default_rng(5)
    q, cu, cache, tables, ctx = case(rng, [(9, 20), (30, 0)], 12, 2)
    pad = np.concatenate([q, normal_bits(rng, (13, 12, 128))])
    out = torch.full(pad.shape, 7.0, device="cuda")
    ops.prefill_varlen_fp8_block(to_dev_bf16(pad), to_dev_i32(cu),
                                 *[torch.from_numpy(a).cuda() for a in cache], to_dev_i32(tables),
                                 to_dev_i32(ctx), SCALE, 64, out=out)
    torch.cuda.synchronize()
    assert torch.all(out[39:] == 7.0)
    want = check(ops, q, cu, cache, tables, ctx)
    assert torch.equal(out[:39], want)


def test_many_sequences(ops):
    """More sequences than a CTA has threads (grid order)."""
    rng = np.random.default_rng(6)
    spec = [(int(rng.integers(0, 4)), int(rng.integers(0, 40))) for _ in range(300)]
    check(ops, *case(rng, spec, 6, 1, extra_blocks=320))


@pytest.mark.parametrize("seqs", [31, 32, 33, 65, 255, 256, 257])
def test_work_order_at_any_count(ops, seqs):
    """Every row once, whatever the number of sequences a lane holds: ragged
    chunks of up to four tiles, empty ones and single rows among them."""
    rng = np.random.default_rng(600 + seqs)
    spec = [(int(rng.choice([0, 1, 1, rng.integers(2, 70)])), int(rng.integers(0, 90)))
            for _ in range(seqs)]
    check(ops, *case(rng, spec, 7, 1, extra_blocks=seqs + 40))


def test_decode_is_a_chunk_of_one(ops):
    """Single-token chunks against pa_decode_fp8_block, both within the bound
    of the same reference."""
    rng = np.random.default_rng(7)
    q, cu, cache, tables, ctx = case(rng, [(1, n - 1) for n in (1, 16, 17, 500)], 32, 8)
    check(ops, q, cu, cache, tables, ctx)
    out = ops.decode_fp8_block(to_dev_bf16(q), *[torch.from_numpy(a).cuda() for a in cache],
                               to_dev_i32(tables), to_dev_i32(ctx), SCALE,
                               out_dtype=torch.float32)
    torch.cuda.synchronize()
    want, mag, tiny = ref.attention(q, *cache, tables, ctx, SCALE)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= ref.tolerance(want, mag, tiny))


def test_errors_are_reported(ops):
    rng = np.random.default_rng(8)
    q, cu, cache, tables, ctx = case(rng, [(20, 30), (20, 30)], 12, 2)
    good, _ = run(ops, q, cu, cache, tables, ctx)
    bad = tables.copy()
    bad[0, 1] = cache[0].shape[0]
    out, err = run(ops, q, cu, cache, bad, ctx)
    assert err == ops.DEVERR_BLOCK_INDEX and torch.equal(out[20:], good[20:])
    out, err = run(ops, q, cu, cache, tables, np.array([19, 50], np.int32))
    assert err == ops.DEVERR_SHAPE and torch.equal(out[20:], good[20:])
    # a chunk whose rows lie past q: skipped, the other one attended
    out, err = run(ops, q, np.array([0, 20, 99], np.int32), cache, tables,
                   np.array([50, 129], np.int32), max_q=79)
    assert err & ops.DEVERR_SHAPE and torch.equal(out[:20], good[:20])
    # rows past max_q_len that no CTA covers (a CTA takes 21 positions here)
    q, cu, cache, tables, ctx = case(rng, [(30, 0)], 12, 2)
    _, err = run(ops, q, cu, cache, tables, ctx, max_q=1)
    assert err == ops.DEVERR_SHAPE


def test_chunked_prompt_then_decode(ops):
    """A prompt stored and attended in chunks that cut blocks, then a decode
    step, captured and replayed: outputs against the reference at each chunk."""
    rng = np.random.default_rng(9)
    Hq, Hkv, NB, total = 12, 2, 20, 150
    tables = random_tables(rng, np.array([total + 1]), NB)
    kc, vc, ks, vs = ref.random_cache(rng, NB, Hkv)
    k, v = (normal_bits(rng, (total, Hkv, 128)) for _ in range(2))
    q = normal_bits(rng, (total, Hq, 128))
    d = [torch.from_numpy(a).cuda() for a in (kc, vc, ks, vs)]
    want = [kc, vc, ks, vs]
    td, at = to_dev_i32(tables), 0
    for step in (37, 1, 64, 48):
        cu, ctx = np.array([0, step], np.int32), np.array([at + step], np.int32)
        rows = slice(at, at + step)
        kd, vd, qd = to_dev_bf16(k[rows]), to_dev_bf16(v[rows]), to_dev_bf16(q[rows])
        cud, ctxd = to_dev_i32(cu), to_dev_i32(ctx)
        out = torch.empty((step, Hq, 128), dtype=torch.float32, device="cuda")
        store = ops.StoreKvFp8BlockCall(kd, vd, *d, cud, td, ctxd)
        attend = ops.PrefillFp8BlockCall(qd, cud, *d, td, ctxd, SCALE, step, out)
        store()
        attend()
        eager = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            store()  # the same rows again: the same bytes
            attend()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        ref.store(k[rows], v[rows], *want, cu, tables, ctx)
        for g, w in zip(d, want):
            assert np.array_equal(g.cpu().numpy(), w)
        w, mag, tiny = ref.attention(q[rows], *want, tables, ctx, SCALE, cu)
        assert np.all(np.abs(out.double().cpu().numpy() - w) <= ref.tolerance(w, mag, tiny))
        at += step
