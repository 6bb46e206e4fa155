"""Every chunk of the block-scaled append that is not consistent is reported,
wherever it lies in the batch."""
import numpy as np
import pytest

from tests import fp8_block_reference as ref
from tests.test_fp8_block_gpu import chunks, run_store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


@pytest.mark.parametrize("seqs", [4, 32, 33, 90])
def test_store_reports_every_inconsistent_chunk(ops, seqs):
    """cu_seqlens past the rows, below zero or falling, and a context below its
    chunk, at any place: reported.  The other chunks are stored, but where
    cu_seqlens fall (no order to find them by); no page is written that no
    table names."""
    rng = np.random.default_rng(seqs)
    spec = [(int(rng.integers(1, 40)), int(rng.integers(0, 30))) for _ in range(seqs)]
    cu, ctx, tables, k, v = chunks(rng, spec, 6 * seqs, 2)
    cache = ref.random_cache(rng, 6 * seqs, 2)
    T, mid = k.shape[0], seqs // 2

    def past(s):
        c = cu.copy()
        c[s:] = T + 1000 * (1 + np.arange(seqs + 1 - s))
        return c, ctx, range(max(s - 1, 0))

    def below(s):
        c = cu.copy()
        c[s] = -5
        return c, ctx, None

    def fall(s):
        c = cu.copy()
        c[s + 1] = max(c[s] - 48, 0)
        return c, ctx, None

    def short(s):
        n = ctx.copy()
        n[s] = spec[s][0] - 1
        return cu, n, [i for i in range(seqs) if i != s]

    def negative(s):
        n = ctx.copy()
        n[s] = -2 ** 31
        return cu, n, [i for i in range(seqs) if i != s]

    named = np.unique(tables[tables >= 0])
    other = np.setdiff1d(np.arange(6 * seqs), named)
    for make, s in ((past, 0), (past, 1), (past, seqs - 1), (past, seqs), (below, 0),
                    (below, mid), (fall, mid), (fall, seqs - 2), (short, 0), (short, seqs - 1),
                    (negative, mid)):
        c, n, stored = make(s)
        got, err = run_store(ops, k, v, cache, c, tables, n)
        assert err == ops.DEVERR_SHAPE, (make.__name__, s)
        got = [g.cpu().numpy() for g in got]
        for g, w in zip(got, cache):
            assert np.array_equal(g[other], w[other]), (make.__name__, s)
        if stored is None:
            continue
        want = [a.copy() for a in cache]
        for i in stored:
            ref.store(k[c[i]:c[i + 1]], v[c[i]:c[i + 1]], *want, [0, c[i + 1] - c[i]],
                      tables[i:i + 1], n[i:i + 1])
        for g, w in zip(got, want):
            assert np.array_equal(g, w), (make.__name__, s)
