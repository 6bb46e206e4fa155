"""Page operators against a plain Python model: copy, fork, free and compact,
alone and as a serving loop would run them.  Everything is whole numbers or
moved bytes, so every comparison is exact."""
import numpy as np
import pytest
import torch

from tests import fp8_block_reference as ref
from tests.helpers import normal_bits, to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


class Model:
    """Tables, lengths and counts, changed one operation at a time."""

    def __init__(self, rng, lens, rows, stride, num_blocks):
        self.tables = rng.integers(-5, num_blocks, (rows, stride)).astype(np.int32)
        self.ctx = np.zeros(rows, np.int32)
        self.refs = np.zeros(num_blocks, np.int32)
        perm, at = rng.permutation(num_blocks), 0
        for r, n in enumerate(lens):
            k = (n + 15) // 16
            self.tables[r, :k] = perm[at:at + k]
            self.refs[perm[at:at + k]] += 1
            self.ctx[r] = n
            at += k

    def fork(self, parents, children):
        start, R, stride = self.ctx.copy(), len(self.ctx), self.tables.shape[1]
        free = [int(p) for p in np.flatnonzero(self.refs <= 0)]
        named, made, pairs, forked = set(), [], [], []
        for p, c in zip(parents, children):
            s = d = f = -1
            ok = 0 <= p < R and 0 <= c < R and p != c and start[c] <= 0 and c not in named
            n = max(int(start[p]), 0) if ok else 0
            if ok and (n + 15) // 16 <= stride:
                named.add(c)
                row = self.tables[p, :(n + 15) // 16].copy()
                if n % 16 == 0 or free:
                    f = n
                    if n % 16:
                        s, d = int(row[-1]), free.pop(0)
                        row[-1] = d
                    made.append((c, row, n))
            pairs.append((s, d))
            forked.append(f)
        for c, row, n in made:
            self.tables[c, :len(row)] = row
            np.add.at(self.refs, row, 1)
            self.ctx[c] = n
        return np.array([s for s, _ in pairs]), np.array([d for _, d in pairs]), np.array(forked)

    def free(self, seqs):
        for r in seqs:
            k = (int(self.ctx[r]) + 15) // 16
            np.subtract.at(self.refs, self.tables[r, :k], 1)
            self.ctx[r] = 0

    def compact(self):
        live = np.flatnonzero(self.refs > 0)
        L = len(live)
        src, dst = live[live >= L], np.flatnonzero(self.refs[:L] <= 0)
        remap = np.arange(len(self.refs))
        remap[src] = dst
        for r, n in enumerate(self.ctx):
            k = (n + 15) // 16
            self.tables[r, :k] = remap[self.tables[r, :k]]
        self.refs[dst] = self.refs[src]
        self.refs[src] = 0
        return src, dst, L, remap

    def device(self):
        return to_dev_i32(self.tables), to_dev_i32(self.ctx), to_dev_i32(self.refs)

    def equals(self, tables, ctx, refs):
        torch.cuda.synchronize()
        assert np.array_equal(ctx.cpu().numpy(), self.ctx)
        assert np.array_equal(refs.cpu().numpy(), self.refs)
        assert np.array_equal(tables.cpu().numpy(), self.tables)


def flags():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


POOLS = {
    "bf16": [(torch.bfloat16, (16, 2, 128))] * 2,
    "fp8": [(torch.uint8, (16, 2, 128)), (torch.uint8, (2, 128, 16)), (torch.uint8, (2,)),
            (torch.uint8, (2,))],
    "odd sizes": [(torch.uint8, (n,)) for n in (1, 3, 15, 16, 17, 31, 4095, 4096, 4097, 12345)],
    "eight heads": [(torch.bfloat16, (16, 8, 128)), (torch.uint8, (8,))],
}


@pytest.mark.parametrize("kind", list(POOLS))
@pytest.mark.parametrize("layers", [1, 37])
def test_copy_pages(ops, kind, layers):
    """Every pool kind, up to 370 pools (several launches), with skipped
    pairs, a device count and untouched pages."""
    g = torch.Generator(device="cuda").manual_seed(1)
    NB = 23
    pools = [torch.randint(0, 256, (NB,) + shape, generator=g, device="cuda").to(torch.uint8)
             if dt == torch.uint8 else
             torch.randn((NB,) + shape, generator=g, device="cuda").to(dt)
             for _ in range(layers) for dt, shape in POOLS[kind]]
    src = np.array([22, -1, 0, 5, 7, 7, 21], np.int32)
    dst = np.array([1, 2, 3, 4, 6, 8, 9], np.int32)
    for count in (None, 5, 0, 99, -3):
        want = [p.clone() for p in pools]
        n = len(src) if count is None else max(0, min(count, len(src)))
        for p in want:
            for s, d in zip(src[:n], dst[:n]):
                if s >= 0:
                    p[int(d)] = p[int(s)]
        err = flags()
        ops.copy_pages(ops.PagePools(pools), to_dev_i32(src), to_dev_i32(dst),
                       count=None if count is None else to_dev_i32([count, 7]), error_flags=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        for i, (a, b) in enumerate(zip(pools, want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (i, count)


def test_copy_pages_unaligned_pool_and_bad_pairs(ops):
    buf = torch.arange(4096 * 9 + 64, device="cuda").to(torch.uint8)
    pool = buf[3:3 + 4096 * 9].view(9, 4096)
    tiny = torch.arange(9 * 16, dtype=torch.uint8, device="cuda").view(9, 16)
    want, want_t = pool.clone(), tiny.clone()
    want[2], want_t[2] = pool[1], tiny[1]
    err = flags()
    ops.copy_pages(ops.PagePools([pool, tiny]), to_dev_i32([9, 1, 0, 3]), to_dev_i32([0, 2, -1, 9]),
                   error_flags=err)
    torch.cuda.synchronize()
    assert int(err.item()) == ops.DEVERR_BLOCK_INDEX
    assert torch.equal(pool, want) and torch.equal(tiny, want_t)


def test_copy_pages_large_pool_offsets(ops):
    """A pool past 4 GiB: page offsets need 64 bits."""
    pool = torch.empty((5, 1 << 30), dtype=torch.uint8, device="cuda")
    pool[4] = 9
    pool[4, ::4099] = 7
    ops.copy_pages(ops.PagePools([pool]), to_dev_i32([4]), to_dev_i32([0]))
    torch.cuda.synchronize()
    assert torch.equal(pool[0], pool[4])


def run_fork(ops, m, parents, children, expect=0):
    t, c, r = m.device()
    err = flags()
    src, dst, forked = ops.fork_pages(t, c, to_dev_i32(parents), to_dev_i32(children), r,
                                      error_flags=err)
    ws, wd, wf = m.fork(parents, children)
    torch.cuda.synchronize()
    assert np.array_equal(forked.cpu().numpy(), wf)
    assert np.array_equal(src.cpu().numpy(), ws) and np.array_equal(dst.cpu().numpy(), wd)
    m.equals(t, c, r)
    assert int(err.item()) == expect


@pytest.mark.parametrize("num_blocks", [60, 9000, 40001])
def test_fork(ops, num_blocks):
    """Full and part-filled last pages, empty parents, one parent many times."""
    rng = np.random.default_rng(num_blocks)
    m = Model(rng, [33, 48, 0, 1, 16, 200], 40, 14, num_blocks)
    run_fork(ops, m, [0, 1, 2, 3, 4, 5, 0, 0, 5], [10, 11, 12, 13, 14, 39, 6, 8, 7])
    run_fork(ops, m, [39, 7, 8], [20, 21, 22])


def test_fork_many(ops):
    """More forks than threads of a block, from a nearly full pool."""
    rng = np.random.default_rng(5)
    m = Model(rng, rng.integers(1, 100, 50), 2500, 7, 3000)
    m.refs[rng.permutation(np.flatnonzero(m.refs == 0))[2300:]] = 1
    parents = rng.integers(0, 50, 2300)
    run_fork(ops, m, list(parents), list(50 + rng.permutation(2450)[:2300]))


def test_fork_refusals(ops):
    """Rows out of range, parent = child, a child with pages, a child named
    twice, a context past the row; each refused, the others forked."""
    rng = np.random.default_rng(6)
    m = Model(rng, [33, 48, 20, 7], 12, 4, 40)
    m.ctx[11] = 65  # five pages, a row of four
    bad = 0x8
    run_fork(ops, m, [0, -1, 12, 1, 2, 3, 11, 0, 0, 1], [5, 6, 6, 1, 3, 5, 7, -1, 12, 8], bad)
    assert m.ctx[5] == 33 and m.ctx[8] == 48 and not m.ctx[6] and not m.ctx[7]


def test_fork_child_of_the_same_call_is_an_empty_parent(ops):
    rng = np.random.default_rng(7)
    m = Model(rng, [33], 6, 4, 20)
    run_fork(ops, m, [0, 2, 3], [2, 3, 4])
    assert list(m.ctx) == [33, 0, 33, 0, 0, 0]


def test_fork_without_free_pages(ops):
    """The pool runs out after two forks: the rest are refused and leave
    their children empty; forks that need no page still go through."""
    rng = np.random.default_rng(8)
    m = Model(rng, [33, 48], 12, 4, 8)
    run_fork(ops, m, [0, 0, 0, 1, 0], [2, 3, 4, 5, 6], 0x20)
    assert list(m.ctx[:7]) == [33, 48, 33, 33, 0, 48, 0]


def test_free(ops):
    """Shared and own pages, an empty row, a row named twice; a count that
    would fall below zero and bad entries are reported."""
    rng = np.random.default_rng(9)
    m = Model(rng, [33, 48, 20], 12, 4, 40)
    m.fork([0, 1, 0], [5, 6, 7])
    t, c, r = m.device()
    err = flags()
    ops.free_pages(t, c, to_dev_i32([5, 0, 3, 1]), r, error_flags=err)
    m.free([5, 0, 3, 1])
    m.equals(t, c, r)
    ops.free_pages(t, c, to_dev_i32([7, 7, 7]), r, error_flags=err)
    m.free([7])
    m.equals(t, c, r)
    assert int(err.item()) == 0
    ops.free_pages(t, c, to_dev_i32([12, -1]), r, error_flags=err)
    m.equals(t, c, r)
    assert int(err.item()) == ops.DEVERR_SHAPE
    err.zero_()
    t[2, 0] = int(np.flatnonzero(m.refs == 0)[0])  # held by nobody
    t[2, 1] = 40
    ops.free_pages(t, c, to_dev_i32([2]), r, error_flags=err)
    torch.cuda.synchronize()
    assert int(err.item()) == ops.DEVERR_PAGES | ops.DEVERR_BLOCK_INDEX
    want = m.refs.copy()
    assert np.array_equal(r.cpu().numpy(), want)


@pytest.mark.parametrize("num_blocks,rows", [(1, 1), (2, 1), (60, 5), (8192, 100), (8193, 100),
                                             (50001, 300)])
def test_compact(ops, num_blocks, rows):
    rng = np.random.default_rng(num_blocks)
    lens, left = [], num_blocks
    for _ in range(rows):
        n = int(rng.integers(0, 200))
        n = min(n, 16 * left)
        left -= (n + 15) // 16
        lens.append(n)
    m = Model(rng, lens, rows + 3, 13, num_blocks)
    if num_blocks > 50:
        m.fork([0, 1, 0], [rows, rows + 1, rows + 2])
    t, c, r = m.device()
    err = flags()
    src, dst, counts, remap = ops.compact_pages(t, c, r, error_flags=err)
    ws, wd, L, wr = m.compact()
    m.equals(t, c, r)
    assert int(err.item()) == 0
    assert counts.cpu().tolist() == [len(ws), L]
    assert np.array_equal(remap.cpu().numpy(), wr)
    pad = np.full(num_blocks // 2 - len(ws), -1)
    assert np.array_equal(src.cpu().numpy(), np.concatenate([ws, pad]))
    assert np.array_equal(dst.cpu().numpy(), np.concatenate([wd, pad]))
    assert np.all(m.refs[:L] > 0) and not np.any(m.refs[L:])


def test_compact_full_and_empty_pool(ops):
    rng = np.random.default_rng(11)
    for lens, L in (([64 * 16], 64), ([0], 0)):
        m = Model(rng, lens, 2, 64, 64)
        t, c, r = m.device()
        _, _, counts, _ = ops.compact_pages(t, c, r)
        m.equals(t, c, r)
        assert counts.cpu().tolist() == [0, L]


def test_tables_must_be_contiguous(ops):
    wide = torch.zeros((4, 9), dtype=torch.int32, device="cuda")
    c, r, one = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (4, 20, 1))
    for fn in (lambda: ops.fork_pages(wide[:, :5], c, one, one, r),
               lambda: ops.free_pages(wide[:, :5], c, one, r),
               lambda: ops.compact_pages(wide[:, :5], c, r)):
        with pytest.raises(ops.PagedAttentionError, match="contiguous"):
            fn()


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_serving_loop(ops, kind):
    """Prompts, a fork into beams, steps that store and decode, beams freed
    and forked anew, a compaction in between: every live sequence decodes to
    the same bits as one that was never moved or shared."""
    rng = np.random.default_rng(12)
    NB, Hkv, Hq, rows, stride = 64, 2, 12, 10, 6
    scale = 1 / np.sqrt(128)
    lens = [37, 16]
    m = Model(rng, lens, rows, stride, NB)
    t, c, r = m.device()
    if kind == "fp8":
        pools = [torch.from_numpy(a).cuda() for a in ref.random_cache(rng, NB, Hkv)]
    else:
        pools = [to_dev_bf16(normal_bits(rng, (NB, 16, Hkv, 128))) for _ in range(2)]
    handle = ops.PagePools(pools)
    history = {}  # row -> list of (k, v) appended after the prompt

    def store(rowset, k, v):
        """One token for each row of rowset, then its length grows."""
        lens = c.clone()
        lens[rowset] += 1
        ctx = lens.cpu().numpy()
        for row in rowset:  # a page for the new token where the last one is full
            if ctx[row] % 16 == 1:
                page = int(torch.nonzero(r <= 0)[0])
                t[row, (ctx[row] - 1) // 16] = page
                r[page] = 1
        c.copy_(lens)
        if kind == "fp8":
            ops.store_kv_fp8_block(k, v, *pools, to_dev_i32(np.arange(len(rowset) + 1)),
                                   t[rowset].contiguous(), c[rowset])
        else:
            slots = [int(t[row, (ctx[row] - 1) // 16]) * 16 + (ctx[row] - 1) % 16
                     for row in rowset]
            ops.store_kv(k, v, *pools, to_dev_i32(slots))

    def decode(pools, tables, ctx, q):
        fn = ops.decode_fp8_block if kind == "fp8" else ops.decode
        # one split: the summation order then depends on the sequence alone
        return fn(q, *pools, tables, ctx, scale, out_dtype=torch.float32, num_splits=1)

    # the same sequences kept apart: prompt pages copied out of the pool now
    kept = [p.clone() for p in pools]
    prompt_tables = t.clone()
    q = to_dev_bf16(normal_bits(rng, (1, Hq, 128)))
    ops.copy_pages(handle, *ops.fork_pages(t, c, to_dev_i32([0, 0, 1]), to_dev_i32([4, 5, 6]), r)[:2])
    origin = {0: 0, 1: 1, 4: 0, 5: 0, 6: 1}
    for row in origin:
        history[row] = []
    for step in range(24):
        live = sorted(origin)
        k, v = (to_dev_bf16(normal_bits(rng, (len(live), Hkv, 128))) for _ in range(2))
        store(live, k, v)
        for i, row in enumerate(live):
            history[row].append((k[i:i + 1], v[i:i + 1]))
        if step in (5, 13):  # drop a beam, fork another in its place
            ops.free_pages(t, c, to_dev_i32([5]), r)
            ops.copy_pages(handle, *ops.fork_pages(t, c, to_dev_i32([4]), to_dev_i32([5]), r)[:2])
            history[5] = list(history[4])
        if step in (9, 20):
            src, dst, counts, _ = ops.compact_pages(t, c, r)
            ops.copy_pages(handle, src, dst, count=counts)
    assert int((r < 0).sum()) == 0
    got = {row: decode(pools, t[row:row + 1], c[row:row + 1], q) for row in origin}
    # rebuild each sequence alone, appending the same tokens one by one
    for row, first in origin.items():
        own = [p.clone() for p in kept]
        n0 = lens[first]
        table = torch.full((1, stride), -1, dtype=torch.int32, device="cuda")
        k0 = (n0 + 15) // 16
        table[0, :k0] = prompt_tables[first, :k0]
        spare = [p for p in range(NB) if p not in table[0, :k0].tolist()]
        total = n0 + len(history[row])
        for j in range(k0, (total + 15) // 16):
            table[0, j] = spare.pop()
        for i, (k, v) in enumerate(history[row]):
            n = n0 + i + 1
            if kind == "fp8":
                ops.store_kv_fp8_block(k, v, *own, to_dev_i32([0, 1]), table, to_dev_i32([n]))
            else:
                slot = int(table[0, (n - 1) // 16]) * 16 + (n - 1) % 16
                ops.store_kv(k, v, *own, to_dev_i32([slot]))
        want = decode(own, table, to_dev_i32([total]), q)
        assert int(c[row]) == total
        assert torch.equal(got[row], want), row


def test_fork_and_copy_in_a_graph(ops):
    """Free, fork and copy captured once and replayed with other parents."""
    rng = np.random.default_rng(13)
    m = Model(rng, [33, 48, 90, 5], 8, 7, 50)
    t, c, r = m.device()
    pool = torch.randn((50, 300), device="cuda")
    parents, children = to_dev_i32([0, 1]), to_dev_i32([6, 7])
    free = ops.FreePagesCall(t, c, children, r, pdl=True)
    fork = ops.ForkPagesCall(t, c, parents, children, r, pdl=True)
    copy = ops.CopyPagesCall(ops.PagePools([pool]), fork.copy_src, fork.copy_dst, pdl=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        free()
        fork()
        copy()
    for pair in ([0, 1], [2, 3], [3, 3], [1, 0]):
        parents.copy_(to_dev_i32(pair))
        before = pool.clone()
        graph.replay()
        m.free([6, 7])
        src, dst, _ = m.fork(pair, [6, 7])
        m.equals(t, c, r)
        for s, d in zip(src, dst):
            if s >= 0:
                before[d] = before[s]
        assert torch.equal(pool, before)
