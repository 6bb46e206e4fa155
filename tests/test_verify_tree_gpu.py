"""pa_verify_tree against the float64 definition: everything it returns is a
whole number, so every comparison is exact."""
import numpy as np
import pytest
import torch

from tests import tree_reference as ref
from tests.helpers import to_dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


def softmax32(x):
    x = x - x.max(-1, keepdims=True)
    e = np.exp(x)
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


class Case:
    def __init__(self, seed, nodes, vocab, arity=3, again=False, drafts=True, sharp=2.0,
                 likeness=0.8):
        rng = np.random.default_rng(seed)
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        T = int(self.cu[-1])
        self.again, self.width = again, max([1, *nodes])
        z = rng.standard_normal((T, vocab))
        self.p = softmax32(sharp * z)
        q = softmax32(sharp * (likeness * z + (1 - likeness) * rng.standard_normal((T, vocab))))
        self.q = q if drafts else None
        self.parents, self.tokens = np.zeros(T, np.int32), np.zeros(T, np.int32)
        for a, e in zip(self.cu[:-1], self.cu[1:]):
            if a == e:
                continue
            par = ref.random_parents(rng, e - a, arity)
            self.parents[a:e] = par
            for j in range(e - a):
                kids = np.flatnonzero(par == j)
                if len(kids):
                    pr = q[a + j].astype(np.float64)
                    full = again or len(kids) > (pr > 0).sum()
                    self.tokens[a + kids] = rng.choice(vocab, len(kids), replace=full, p=pr / pr.sum())
        self.u = rng.random(T, np.float32)
        self.u_last = rng.random(len(nodes), np.float32)

    def want(self):
        return ref.verify_all(self.cu, self.tokens, self.parents, self.p, self.q, self.u,
                              self.u_last, self.width, self.again)

    def args(self):
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
        return (to_dev_i32(self.tokens), to_dev_i32(self.parents), to_dev_i32(self.cu),
                dev(self.p), dev(self.u), dev(self.u_last), self.width), dict(
                    draft_probs=None if self.q is None else dev(self.q),
                    with_replacement=self.again)

    def run(self, ops, flags=0, **more):
        a, kw = self.args()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = ops.verify_tree(*a, **{**kw, **more}, error_flags=err)
        torch.cuda.synchronize()
        assert int(err) == flags
        return [x.cpu().numpy() for x in got]

    def check(self, ops, flags=0, **more):
        got, want = self.run(ops, flags, **more), self.want()
        for g, w, name in zip(got, want, ("accepted", "path", "tokens")):
            assert np.array_equal(g, w), (name, np.argwhere(g != w)[:5], g[g != w][:5], w[g != w][:5])
        return want


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 127, 128, 129, 1000, 2047, 2049, 5003, 16385, 40001])
@pytest.mark.parametrize("mode", ["without", "with", "looked up"])
def test_vocabularies(ops, vocab, mode):
    c = Case(vocab, [5, 1, 9, 0, 12, 7], vocab, again=mode == "with", drafts=mode != "looked up")
    c.check(ops)


@pytest.mark.parametrize("nodes", [[1], [2], [0], [0, 0], [33], [64, 65], [256], [257], [258, 3], [600]])
@pytest.mark.parametrize("arity", [1, 3, 40])
def test_tree_sizes(ops, nodes, arity):
    c = Case(sum(nodes) + arity, nodes, 300, arity, likeness=0.97)
    c.check(ops)


@pytest.mark.parametrize("mode", ["without", "with", "looked up"])
def test_many_sequences(ops, mode):
    rng = np.random.default_rng(2)
    c = Case(4, rng.integers(0, 14, 300).tolist(), 700, 4, again=mode == "with",
             drafts=mode != "looked up")
    count, _, _ = c.check(ops)
    # walks of many lengths (guesses looked up in such rows are seldom right)
    assert len(set(count.tolist())) > (2 if mode == "looked up" else 4)


def test_long_walks_of_looked_up_guesses(ops):
    """Rows that are nearly certain: most guesses hold, and walks get long."""
    c = Case(5, [30] * 40, 50, 2, drafts=False, sharp=9.0, likeness=1.0)
    count, _, _ = c.check(ops)
    assert count.max() > 6 and len(set(count.tolist())) > 4


@pytest.mark.parametrize("vocab", [151936, 128001])
@pytest.mark.parametrize("sharp", [0.3, 3.0])
def test_large_vocabularies(ops, vocab, sharp):
    """Flat rows put many borders close together."""
    c = Case(vocab, [6, 4, 8], vocab, 2, sharp=sharp, likeness=0.7)
    c.check(ops)


@pytest.mark.parametrize("vocab", [1 << 20, (1 << 20) - 3])
@pytest.mark.parametrize("drafts", [True, False])
def test_the_largest_vocabulary(ops, vocab, drafts):
    c = Case(3, [3, 2], vocab, 2, drafts=drafts, sharp=1.0)
    c.check(ops)
    c.u[:] = np.float32(1 - 2.0 ** -24)
    c.check(ops)


@pytest.mark.parametrize("seqs", [1, 14, 30, 45, 90])
@pytest.mark.parametrize("vocab", [70000, 70001, 9000])
def test_clusters_of_every_size(ops, seqs, vocab):
    """The batch sets how many CTAs share a sequence, and the rows' length how many are worth it."""
    c = Case(seqs + vocab, [2, 3] * (seqs // 2) + [4] * (seqs % 2), vocab, 2, likeness=0.6)
    c.check(ops)


@pytest.mark.parametrize("drafts", [True, False])
def test_siblings_all_rejected(ops, drafts):
    """A star of guesses that the random numbers reject one after the other."""
    c = Case(6, [30, 30], 400, 30, drafts=drafts)
    c.parents[:] = np.tile(np.where(np.arange(30) > 0, 0, -1), 2)
    c.u[:] = np.float32(1 - 2.0 ** -24)
    count, _, _ = c.check(ops)


def test_one_token_many_times(ops):
    """Equal siblings: looked-up or drawn with replacement, the second has nothing left."""
    for drafts in (True, False):
        c = Case(7, [6], 50, 6, again=True, drafts=drafts)
        c.parents[:] = [-1, 0, 0, 0, 0, 0]
        c.tokens[:] = 3
        c.u[:] = 0.999
        c.check(ops)
        c.u[3] = 0.0
        c.check(ops)


def test_equal_rows_accept_everything(ops):
    c = Case(8, [9, 4], 200, 2)
    c.q = c.p.copy()
    count, _, _ = c.check(ops)
    c.u[:] = np.float32(1 - 2.0 ** -24)
    c.check(ops)


def test_random_numbers_at_the_ends(ops):
    for u in (0.0, 2.0 ** -24, 1 - 2.0 ** -24, 1.0):
        c = Case(9, [1, 4, 7], 1000, 3)
        c.u_last[:] = u
        c.check(ops)
        c.u[:] = u
        c.check(ops)


def test_one_hot_target(ops):
    """A target that is certain: the walk follows it, and draws it."""
    c = Case(10, [12, 5], 64, 4)
    hot = np.random.default_rng(1).integers(0, 64, c.p.shape[0])
    c.p[:] = 0
    c.p[np.arange(len(hot)), hot] = 1
    c.tokens[1::2] = hot[c.parents[1::2].clip(0)]
    for drafts in (c.q, None):
        c.q = drafts
        c.check(ops)


def test_rows_apart_and_unaligned(ops):
    c = Case(11, [8, 3], 1001, 3)
    a, kw = c.args()
    for pad in (1, 3, 7):
        p = torch.full((c.p.shape[0], 1001 + pad), float("nan"), device="cuda")
        q = torch.full((c.p.shape[0], 1001 + 2 * pad), float("nan"), device="cuda")
        p[:, :1001], q[:, :1001] = a[3], kw["draft_probs"]
        got = ops.verify_tree(*a[:3], p[:, :1001], *a[4:], draft_probs=q[:, :1001])
        for g, w in zip(got, c.want()):
            assert np.array_equal(g.cpu().numpy(), w)


def test_tokens_outside_the_vocabulary(ops):
    for bad in (-1, 90, 2**31 - 1, -2**31):
        for drafts in (True, False):
            c = Case(12, [5, 5], 90, 5, drafts=drafts)
            c.parents[:] = [-1, 0, 0, 0, 0] * 2
            c.u[:] = 0.999
            c.tokens[2] = bad
            c.p[0, c.tokens[[1, 3, 4]]] = 0
            c.check(ops, flags=64)


def test_parents_that_come_later(ops):
    c = Case(13, [6, 4], 90, 2)
    c.parents[3] = 3
    c.check(ops, flags=8)
    c.parents[3] = 2**31 - 1
    c.check(ops, flags=8)
    c.parents[3] = -2**31
    c.check(ops)


def test_sequences_that_do_not_fit(ops):
    c = Case(14, [6, 4, 5], 90, 2)
    want = c.want()
    a, kw = c.args()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = [x.cpu().numpy() for x in ops.verify_tree(*a[:6], 5, **kw, error_flags=err)]
    assert int(err) == 8
    assert got[0][0] == 0 and (got[1][0] == -1).all() and (got[2][0] == -1).all()
    for g, w in zip(got, want):
        assert np.array_equal(g[1:], w[1:, :5] if w.ndim == 2 else w[1:])
    for cu in ([0, 6, 3, 15], [-1, 6, 10, 15], [0, 6, 10, 16], [2**31 - 1, -2**31, 10, 15]):
        err.zero_()
        ops.verify_tree(*a[:2], to_dev_i32(cu), *a[3:6], 15, **kw, error_flags=err)
        assert int(err) == 8


def test_no_weight_at_all(ops):
    c = Case(15, [3], 40, 1)
    c.p[:] = 0
    for drafts in (c.q, None):
        c.q = drafts
        count, path, tokens = c.check(ops)
        assert tokens[0, count[0] - 1] == -1
    c.p[:] = np.nan
    got = c.run(ops)
    assert got[0][0] == 1 and got[2][0, 0] == -1


def test_streams_and_graphs(ops):
    c = Case(16, [8, 3, 20], 30000, 3)
    a, kw = c.args()
    call = ops.VerifyTreeCall(*a, **kw, pdl=True)
    s = torch.cuda.Stream()
    eager = [x.cpu().numpy() for x in ops.verify_tree(*a, **kw, stream=s)]
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x in (call.accepted, call.path, call.out_tokens):
        x.fill_(77)
    g.replay()
    torch.cuda.synchronize()
    for e, x, w in zip(eager, (call.accepted, call.path, call.out_tokens), c.want()):
        assert np.array_equal(e, w) and np.array_equal(x.cpu().numpy(), w)
