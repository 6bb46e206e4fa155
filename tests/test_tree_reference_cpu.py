"""Pins of tests/tree_reference.py: the verification keeps the target's
distribution, closed forms of the tree's attention, and the commit's moves."""
import numpy as np
import pytest

from tests import tree_reference as ref
from tests.helpers import brute_attention, normal_bits, random_tables, scatter_pool


def test_way():
    par = np.array([-1, 0, 0, 1, 3, 2])
    assert ref.way(par, 4) == [4, 3, 1, 0] and ref.way(par, 5) == [5, 2, 0] and ref.way(par, 0) == [0]


@pytest.mark.parametrize("mode", ["without", "with", "looked up"])
def test_first_token_has_the_targets_distribution(mode):
    """Draw guesses from q, verify, and count the first new token: it is distributed as p
    whatever q is (each count within five of its standard deviations)."""
    rng = np.random.default_rng(3)
    V, n, N = 5, 4, 20000
    p = np.array([0.4, 0.3, 0.15, 0.1, 0.05], np.float32)
    q = np.array([0.1, 0.25, 0.05, 0.4, 0.2], np.float32)
    parents = np.array([-1, 0, 0, 0])
    P, Q = np.tile(p, (n, 1)), np.tile(q, (n, 1))
    hits = np.zeros(V)
    for _ in range(N):
        toks = np.zeros(n, int)
        if mode == "looked up":
            toks[1:] = [3, 0, 3]
        else:
            toks[1:] = rng.choice(V, 3, replace=mode == "with", p=q.astype(float) / q.astype(float).sum())
        _, new = ref.verify(toks, parents, P, None if mode == "looked up" else Q, rng.random(n),
                            rng.random(), again=mode == "with")
        hits[new[0]] += 1
    assert (np.abs(hits - N * p) < 5 * np.sqrt(N * p * (1 - p))).all(), hits / N


def test_one_draft_is_the_usual_rule():
    """One guess: accepted iff u < p / q, else drawn from the positive part of p - q."""
    p = np.array([[0.5, 0.25, 0.25], [0, 0, 1]], np.float32)
    q = np.array([[0.25, 0.75, 0.0], [0, 0, 0]], np.float32)
    run = lambda tok, u, last: ref.verify([0, tok], [-1, 0], p, q, [0, u], last)
    assert run(0, 0.99, 0.5) == ([0, 1], [0, 2])
    assert run(1, 0.33, 0.5) == ([0, 1], [1, 2])
    assert run(1, 0.34, 0.49) == ([0], [0])   # max(p - q, 0) = [1/4, 0, 1/4]
    assert run(1, 0.34, 0.51) == ([0], [2])


def test_last_draw_at_its_borders():
    p = np.array([[0.25, 0.0, 0.5, 0.25, 0.0]], np.float32)
    draw = lambda u: ref.verify([0], [-1], p, None, [0], u)[1]
    assert [draw(u) for u in (0.0, 0.2499, 0.25, 0.7499, 0.75, 0.9999, 1.0)] == [
        [0], [0], [2], [2], [3], [3], [3]]


def test_attention_of_a_chain_is_causal():
    rng = np.random.default_rng(5)
    ctx, cu = np.array([40, 9]), np.array([0, 6, 9])
    seqs = [[normal_bits(rng, (n, 2, 128)) for n in ctx] for _ in range(2)]
    tables = random_tables(rng, ctx, 8)
    k, v = (scatter_pool(s, tables, 8) for s in seqs)
    q = normal_bits(rng, (9, 4, 128))
    par = np.array([-1, 0, 1, 2, 3, 4, -1, 0, 1])
    out, a, big = ref.attention(q, k, v, tables, ctx, cu, par, 0.1)
    for b in range(2):
        for i in range(cu[b], cu[b + 1]):
            for h in range(4):
                n = ctx[b] - (cu[b + 1] - cu[b]) + i - cu[b] + 1
                want = brute_attention(q[i, h], seqs[0][b][:, h // 2], seqs[1][b][:, h // 2], 0.1, n)
                assert np.allclose(out[i, h], want, rtol=0, atol=1e-13)
    assert (a >= np.abs(out) - 1e-12).all() and np.isfinite(big).all()


def test_commit_moves_rows_down():
    pool = np.arange(4 * 16).reshape(4, 16, 1)
    tables, ctx = np.array([[2, 0, 3]]), np.array([36])
    want = pool.copy()
    want[0, 15], want[3, 0] = pool[3, 1], pool[3, 3]  # positions 31, 32 <- 33, 35
    refs = np.array([1, 0, 1, 1])
    ref.commit([pool], tables, ctx, [0, 6], np.array([[0, 3, 5]]), [3], refs)
    assert np.array_equal(pool, want) and ctx[0] == 33 and refs.tolist() == [1, 0, 1, 1]
    ref.commit([pool], tables, ctx, [0, 3], np.array([[0]]), [1], refs)
    assert ctx[0] == 31 and refs.tolist() == [1, 0, 1, 0]
