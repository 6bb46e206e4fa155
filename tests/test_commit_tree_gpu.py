"""pa_commit_tree against a plain model: moved rows, lengths and counts, exact."""
import numpy as np
import pytest
import torch

from tests import tree_reference as ref
from tests.helpers import random_tables, to_dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


class Case:
    """Pools of random bytes: `shapes` are the rows' trailing shape and type."""

    def __init__(self, seed, done, nodes, shapes=(((2, 128), np.uint16),) * 2, count=None, width=None):
        self.rng = rng = np.random.default_rng(seed)
        done, nodes = np.array(done), np.array(nodes)
        self.ctx = (done + nodes).astype(np.int32)
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.NB = int(((self.ctx + 15) // 16).sum()) + 3
        self.tables = random_tables(rng, self.ctx, self.NB, pad=-9)
        self.refs = np.zeros(self.NB, np.int32)
        self.refs[self.tables[self.tables >= 0]] = 1
        self.pools = [rng.integers(0, np.iinfo(t).max, (self.NB, 16, *s), endpoint=True).astype(t)
                      for s, t in shapes]
        self.width = width or max(1, int(nodes.max(initial=0)))
        self.count = np.array([rng.integers(0 if n == 0 else 1, n + 1) for n in nodes]
                              if count is None else count, np.int32)
        self.path = np.full((len(nodes), self.width), -5, np.int32)
        for b, (n, c) in enumerate(zip(nodes, self.count)):
            if c:
                self.path[b, :c] = np.sort(rng.choice(n, c, replace=False))

    def run(self, ops, refs=True, flags=0, **kw):
        dev = [torch.from_numpy(p.view(np.int16) if p.dtype == np.uint16 else p).cuda()
               for p in self.pools]
        ctx, counts = to_dev_i32(self.ctx), to_dev_i32(self.refs)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.commit_tree(ops.PagePools(dev), to_dev_i32(self.cu), to_dev_i32(self.tables), ctx,
                        to_dev_i32(self.path), to_dev_i32(self.count),
                        ref_counts=counts if refs else None, error_flags=err, **kw)
        torch.cuda.synchronize()
        assert int(err) == flags
        return ([d.cpu().numpy().view(p.dtype) for d, p in zip(dev, self.pools)],
                ctx.cpu().numpy(), counts.cpu().numpy())

    def check(self, ops, refs=True, only=None, **kw):
        pools, ctx, counts = self.run(ops, refs, **kw)
        want = [p.copy() for p in self.pools], self.ctx.copy(), self.refs.copy()
        rows = slice(None) if only is None else only
        cu = self.cu
        if only is not None:  # the others are left as they are
            lens = np.diff(self.cu)
            for b in only:
                one = want[1][b:b + 1]
                ref.commit(want[0], self.tables[b:b + 1], one, [0, lens[b]], self.path[b:b + 1],
                           self.count[b:b + 1], want[2] if refs else None)
        else:
            ref.commit(want[0], self.tables, want[1], cu, self.path, self.count,
                       want[2] if refs else None)
        assert all(np.array_equal(a, b) for a, b in zip(pools, want[0]))
        assert np.array_equal(ctx, want[1]) and np.array_equal(counts, want[2])


@pytest.mark.parametrize("done,nodes", [([0], [1]), ([5], [3]), ([0], [40]), ([15], [17]),
                                        ([16], [64]), ([100, 0, 33, 7], [8, 5, 0, 30]),
                                        ([63, 64, 65], [1, 16, 70]), ([1000], [600])])
@pytest.mark.parametrize("refs", [True, False])
def test_lengths(ops, done, nodes, refs):
    for seed in range(3):
        Case(seed, done, nodes).check(ops, refs)


@pytest.mark.parametrize("shapes", [
    (((1, 128), np.uint16),), (((8, 128), np.uint16),) * 2, (((2, 128), np.uint8),) * 3,
    (((2, 128), np.uint16), ((2, 128), np.uint8), ((3,), np.uint8), ((1,), np.uint16)),
    (((5,), np.uint8),) * 2])
def test_row_sizes(ops, shapes):
    Case(3, [30, 7], [20, 9], shapes).check(ops)


@pytest.mark.parametrize("pools", [1, 127, 128, 129, 300])
def test_many_pools(ops, pools):
    Case(4, [30, 7, 1], [20, 9, 2], (((1, 16), np.uint16),) * pools).check(ops)


def test_many_sequences(ops):
    rng = np.random.default_rng(1)
    Case(5, rng.integers(0, 90, 300), rng.integers(0, 30, 300)).check(ops)


def test_nothing_accepted(ops):
    Case(6, [30, 16, 40], [20, 16, 5], count=[0, 0, 0]).check(ops)


def test_everything_accepted(ops):
    Case(7, [30, 16, 40], [20, 16, 5], count=[20, 16, 5]).check(ops)


def test_paths_of_every_kind(ops):
    """Chains of moves in which a step's target is an earlier step's source."""
    for path in ([0, 2, 3], [1, 2, 3, 4, 5, 6, 7], [0, 8, 9, 10, 11, 12], [19], [0, 1, 2, 19],
                 list(range(1, 20)), list(range(0, 20, 2))):
        c = Case(8, [13], [20], count=[len(path)])
        c.path[0, :len(path)] = path
        c.check(ops)


def test_pages_let_go(ops):
    """Shared, free and doubled entries among the pages that are let go."""
    c = Case(9, [10, 14], [70, 50], count=[1, 1])
    page = c.tables[0, 4]
    c.refs[page] = 3
    c.check(ops)
    c.refs[page] = 0
    c.refs[c.tables[1, 3]] = 0
    pools, ctx, counts = c.run(ops, flags=32)
    assert counts[page] == 0 and counts[c.tables[1, 3]] == 0 and (counts >= 0).all()


@pytest.mark.parametrize("fault", ["count", "negative", "order", "range", "below", "width", "keys",
                                   "table"])
def test_bad_sequences_stay_as_they_were(ops, fault):
    c = Case(10, [30, 17, 5], [20, 9, 12], count=[6, 4, 5])
    if fault == "count":
        c.count[1] = 10
    elif fault == "negative":
        c.count[1] = -1
    elif fault == "order":
        c.path[1, 2] = c.path[1, 1]
    elif fault == "range":
        c.path[1, 3] = 9
    elif fault == "below":
        c.path[1, 0] = -1
    elif fault == "width":
        c.path, c.count[1] = c.path[:, :6].copy(), 7
    elif fault == "keys":
        c.ctx[1] = 8
    else:
        c.ctx[1] = 16 * c.tables.shape[1] + 1
    c.check(ops, flags=8, only=[0, 2])


@pytest.mark.parametrize("cu", [[0, 20, 10, 41], [0, 2**31 - 1, -2**31, 12]])
def test_bad_offsets(ops, cu):
    c = Case(11, [30, 17, 5], [20, 9, 12])
    keep = c.ctx.copy()
    c.cu = np.array(cu, np.int32)
    c.count[:] = 0
    _, ctx, _ = c.run(ops, refs=False, flags=8)
    assert ctx[1] == keep[1]


@pytest.mark.parametrize("bad", [-1, 10**6, 2**31 - 1, -2**31])
def test_bad_table_entry(ops, bad):
    c = Case(12, [30, 17], [40, 9], count=[3, 4])
    c.path[0, :3] = [0, 20, 36]  # positions 50 (entry 3) and 66 (entry 4)
    good = c.tables[0, 50 // 16]
    c.tables[0, 50 // 16] = bad
    pools, ctx, _ = c.run(ops, refs=False, flags=1)
    assert ctx.tolist() == [33, 21]
    t = c.tables[0]
    assert np.array_equal(pools[0][t[2], 32 % 16], c.pools[0][t[66 // 16], 66 % 16])
    assert np.array_equal(pools[0][t[31 // 16], 31 % 16], c.pools[0][t[31 // 16], 31 % 16])
    assert np.array_equal(pools[0][good], c.pools[0][good])


def test_streams_and_graphs(ops):
    c = Case(13, [100, 30], [30, 12])
    want = [p.copy() for p in c.pools], c.ctx.copy(), c.refs.copy()
    ref.commit(want[0], c.tables, want[1], c.cu, c.path, c.count, want[2])
    dev = [torch.from_numpy(p.view(np.int16)).cuda() for p in c.pools]
    first = [d.clone() for d in dev]
    ctx, refs = to_dev_i32(c.ctx), to_dev_i32(c.refs)
    call = ops.CommitTreeCall(ops.PagePools(dev), to_dev_i32(c.cu), to_dev_i32(c.tables), ctx,
                              to_dev_i32(c.path), to_dev_i32(c.count), refs, pdl=True)

    def restore():
        for d, f in zip(dev, first):
            d.copy_(f)
        ctx.copy_(to_dev_i32(c.ctx))
        refs.copy_(to_dev_i32(c.refs))

    def right():
        torch.cuda.synchronize()
        return all(np.array_equal(d.cpu().numpy().view(np.uint16), w) for d, w in zip(dev, want[0])) \
            and np.array_equal(ctx.cpu().numpy(), want[1]) \
            and np.array_equal(refs.cpu().numpy(), want[2])
    torch.cuda.synchronize()
    call(torch.cuda.Stream())
    assert right()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        restore()
        g.replay()
        assert right()
