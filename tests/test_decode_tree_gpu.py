"""pa_decode_tree against the float64 definition: tree shapes, head layouts,
lengths, splits, masked values that are not finite, and bad inputs."""
import numpy as np
import pytest
import torch

from tests import tree_reference as ref
from tests.helpers import dev_to_f64, normal_bits, random_tables, to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu
SCALE = 1 / np.sqrt(128)


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


class Case:
    def __init__(self, seed, done, nodes, hq=12, hkv=2, arity=3, parents=None, amp=1.0, spare=3):
        rng = np.random.default_rng(seed)
        self.done, self.nodes = np.array(done), np.array(nodes)
        self.ctx = (self.done + self.nodes).astype(np.int32)
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        if parents is None:
            parents = [ref.random_parents(rng, n, arity) for n in nodes]
        self.parents = np.concatenate([*parents, np.zeros(0)]).astype(np.int32)
        NB = int(((self.ctx + 15) // 16).sum()) + spare
        self.tables = random_tables(rng, self.ctx, NB, pad=-7)
        # rows that no sequence holds are NaN
        self.k = np.full((NB, 16, hkv, 128), 0x7FC0, np.uint16)
        self.v = self.k.copy()
        for b, n in enumerate(self.ctx):
            pos = np.arange(n)
            self.k[self.tables[b, pos // 16], pos % 16] = normal_bits(rng, (n, hkv, 128))
            self.v[self.tables[b, pos // 16], pos % 16] = normal_bits(rng, (n, hkv, 128))
        self.T = int(self.cu[-1])
        self.q = normal_bits(rng, (self.T, hq, 128))
        if amp != 1.0:
            from paged_kv_continuous_gb300.synth import bf16_bits, bf16_to_f64
            self.q = bf16_bits((bf16_to_f64(self.q) * amp).astype(np.float32))

    def run(self, ops, out_dtype=torch.float32, scale=SCALE, check=True, **kw):
        d = dict(q=to_dev_bf16(self.q), cu=to_dev_i32(self.cu), par=to_dev_i32(self.parents),
                 k=to_dev_bf16(self.k), v=to_dev_bf16(self.v), t=to_dev_i32(self.tables),
                 c=to_dev_i32(self.ctx))
        ws = ops.tree_workspace(kw.get("num_splits", 0))
        out = torch.full(d["q"].shape, float("nan"), dtype=out_dtype, device="cuda")
        ops.decode_tree(d["q"], d["cu"], d["par"], d["k"], d["v"], d["t"], d["c"], scale,
                        max(1, int(self.nodes.max(initial=0))), out=out, workspace=ws, **kw)
        torch.cuda.synchronize()
        flags = ops.read_error_word(ws)
        if check:
            assert flags == 0
        return out if check else (out, flags)

    def reference(self, scale=SCALE):
        return ref.attention(self.q, self.k, self.v, self.tables, self.ctx, self.cu, self.parents,
                             scale)

    def check(self, out, scale=SCALE, refs=None, rows=None):
        want, a, big = refs or self.reference(scale)
        keys = int(self.ctx.max(initial=0))
        bound = ref.attention_bound(want, a, big, scale, keys, out.dtype == torch.bfloat16)
        err = np.abs(dev_to_f64(out) - want)
        bad = ~(err <= bound)
        if rows is not None:
            bad &= rows[:, None, None]
        assert not bad.any(), (int(bad.sum()), float(np.nanmax(err / bound)), np.argwhere(bad)[:3])


@pytest.mark.parametrize("done,nodes", [
    ([0], [1]), ([1], [1]), ([15], [1]), ([16], [1]), ([63], [1]), ([64], [1]), ([300], [8]),
    ([0], [5]), ([0], [64]), ([0], [65]), ([1], [63]), ([60], [9]), ([64], [64]), ([127], [2]),
    ([100, 0, 31], [7, 0, 1]), ([0, 0], [0, 3]), ([5, 700, 64], [33, 20, 16])])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_lengths(ops, done, nodes, out_dtype):
    c = Case(sum(done) + 7 * sum(nodes), done, nodes)
    c.check(c.run(ops, out_dtype))


@pytest.mark.parametrize("hkv", [1, 2, 4, 8])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 8])
def test_heads(ops, hkv, group):
    c = Case(10 * hkv + group, [90, 33], [23, 6], hkv * group, hkv)
    c.check(c.run(ops))


@pytest.mark.parametrize("kind", ["chain", "star", "forest", "random", "late"])
@pytest.mark.parametrize("n", [2, 40, 150])
def test_shapes_of_trees(ops, kind, n):
    rng = np.random.default_rng(n)
    par = {"chain": np.arange(n) - 1, "star": np.where(np.arange(n) > 0, 0, -1),
           "forest": np.full(n, -1), "random": ref.random_parents(rng, n, 2),
           # every node hangs on the one half way before it
           "late": np.where(np.arange(n) > 0, np.arange(n) // 2, -1)}[kind]
    if kind == "late":
        par[1:] = np.minimum(par[1:], np.arange(1, n) - 1)
    c = Case(n, [77], [n], 4, 1, parents=[par])
    c.check(c.run(ops))


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 64, 304, 1000])
def test_splits_agree(ops, splits):
    """Any number of CTAs gives the same attention, with pieces that end anywhere."""
    c = Case(3, [1500, 0, 200, 63], [25, 3, 1, 40], 6, 2)
    refs = c.reference()
    out = c.run(ops, num_splits=splits)
    c.check(out, refs=refs)
    again = c.run(ops, num_splits=splits)
    assert torch.equal(out, again)


@pytest.mark.parametrize("nodes,hq,hkv", [([300], 8, 1), ([45, 200, 64], 8, 2), ([86], 12, 2)])
@pytest.mark.parametrize("splits", [0, 1, 2, 5, 9])
def test_row_tiles_in_pairs(ops, nodes, hq, hkv, splits):
    """Row tiles in twos and left over, on an even or odd number of CTAs, both output types."""
    c = Case(sum(nodes), [130, 700, 3][:len(nodes)], nodes, hq, hkv)
    refs = c.reference()
    c.check(c.run(ops, num_splits=splits), refs=refs)
    c.check(c.run(ops, torch.bfloat16, num_splits=splits), refs=refs)


def test_both_output_types_of_long_and_short_pieces(ops):
    """fp32 rows of pieces around the length where a weight's third term ends."""
    for keys in (700, 768, 832, 1500):
        c = Case(keys, [keys - 5], [5], 4, 1)
        refs = c.reference()
        for splits in (1, 2):
            c.check(c.run(ops, num_splits=splits), refs=refs)


def test_many_sequences(ops):
    rng = np.random.default_rng(5)
    nodes = rng.integers(0, 4, 700)
    c = Case(5, rng.integers(0, 40, 700), nodes, 2, 1)
    c.check(c.run(ops))


def test_long_context(ops):
    c = Case(6, [20000, 9001], [6, 17], 8, 4)
    c.check(c.run(ops))
    c.check(c.run(ops, torch.bfloat16))


def test_the_longest_context(ops):
    """2^31 - 1 keys, all but the last pages the same one: offsets, tiles and windows at the end
    of an int.  K is zero and V one, so every row is one, but where a drafted node's NaN is
    seen: nodes 0 and 1 (its child) see node 0's, node 2 does not."""
    n = 2**31 - 1
    entries = (n + 15) // 16
    tables = torch.zeros((1, entries), dtype=torch.int32, device="cuda")
    tables[0, -1] = 1
    k = torch.zeros((2, 16, 1, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.ones((2, 16, 1, 128), dtype=torch.bfloat16, device="cuda")
    last = (n - 1) % 16
    v[1, last - 2, 0, 5] = float("nan")  # node 0
    v[1, last + 1:] = float("nan")  # past the end
    q = torch.randn((3, 1, 128), device="cuda").to(torch.bfloat16)
    ws = ops.tree_workspace()
    out = ops.decode_tree(q, to_dev_i32([0, 3]), to_dev_i32([-1, 0, -1]), k, v, tables,
                          to_dev_i32([n]), SCALE, 3, out_dtype=torch.float32, workspace=ws)
    assert ops.read_error_word(ws) == 0
    o = out[:, 0].cpu()
    nan = torch.zeros((3, 128), dtype=torch.bool)
    nan[:2, 5] = True
    assert torch.equal(torch.isnan(o), nan)
    # a part is some 2^31 / 304 = 7.1 million keys: its sums of ones are whole numbers below 2^24,
    # exact in fp32, and the merge adds 2^-20
    assert (o[~nan] - 1).abs().max() <= 2.0 ** -20


@pytest.mark.parametrize("scale", [-SCALE, 0.0, 1.0])
def test_scales(ops, scale):
    c = Case(8, [100], [20], 6, 2)
    c.check(c.run(ops, scale=scale), scale)


def test_large_scores(ops):
    """Scores far apart: the running reference moves, and most weights vanish."""
    c = Case(9, [400], [12], 4, 2, amp=6.0)
    c.check(c.run(ops))


def test_a_chain_is_a_causal_chunk(ops):
    c = Case(11, [333, 0, 64], [50, 9, 1], parents=[np.arange(50) - 1, np.arange(9) - 1, [-1]])
    tree = c.run(ops)
    chunk = ops.prefill_varlen(to_dev_bf16(c.q), to_dev_i32(c.cu), to_dev_bf16(c.k),
                               to_dev_bf16(c.v), to_dev_i32(c.tables), to_dev_i32(c.ctx), SCALE,
                               50, out_dtype=torch.float32)
    refs = c.reference()
    c.check(tree, refs=refs)
    c.check(chunk, refs=refs)


def test_one_node_is_a_decode(ops):
    c = Case(12, [333, 0, 64, 5000], [1] * 4)
    refs = c.reference()
    c.check(c.run(ops), refs=refs)
    c.check(ops.decode(to_dev_bf16(c.q), to_dev_bf16(c.k), to_dev_bf16(c.v), to_dev_i32(c.tables),
                       to_dev_i32(c.ctx), SCALE, out_dtype=torch.float32), refs=refs)


@pytest.mark.parametrize("value", [0x7FC0, 0x7F80, 0xFF80])  # NaN, inf, -inf
@pytest.mark.parametrize("which", ["v", "k"])
@pytest.mark.parametrize("splits", [0, 5])
def test_values_that_are_not_finite_stay_with_those_who_see_them(ops, value, which, splits):
    """One drafted node's row: the nodes below it, and itself, are the only ones."""
    c = Case(13, [130], [90], 6, 2)
    refs = c.reference()
    node, dim, head = 37, 77, 1
    pos = 130 + node
    getattr(c, which)[c.tables[0, pos // 16], pos % 16, head, dim] = value
    sees = np.array([node in ref.way(c.parents, i) for i in range(90)])
    out = dev_to_f64(c.run(ops, num_splits=splits))
    if which == "v":
        assert not np.isfinite(out[sees][:, 3:, dim]).any()
        clean = np.ones_like(out, bool)
        clean[np.ix_(sees, [3, 4, 5], [dim])] = False
    else:
        clean = np.ones_like(out, bool)
        clean[np.ix_(sees, [3, 4, 5])] = False
    want, a, big = refs
    bound = ref.attention_bound(want, a, big, SCALE, 220, False)
    assert (np.abs(out - want) <= bound)[clean].all()


def test_query_row_not_finite(ops):
    c = Case(14, [50], [10], 6, 2)
    refs = c.reference()
    c.q[4, 2, 9] = 0x7FC0
    out = dev_to_f64(c.run(ops))
    assert np.isnan(out[4, 2]).all()
    want, a, big = refs
    ok = np.abs(out - want) <= ref.attention_bound(want, a, big, SCALE, 60, False)
    ok[4, 2] = True
    assert ok.all()


def test_rows_behind_the_last_sequence_stay(ops):
    c = Case(15, [50, 20], [10, 4], 6, 2)
    refs = c.reference()
    T = c.T + 5
    q = torch.full((T, 6, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[:c.T] = to_dev_bf16(c.q)
    par = torch.full((T,), 99, dtype=torch.int32, device="cuda")
    par[:c.T] = to_dev_i32(c.parents)
    out = torch.full((T, 6, 128), 7.0, device="cuda")
    ws = ops.tree_workspace()
    ops.decode_tree(q, to_dev_i32(c.cu), par, to_dev_bf16(c.k), to_dev_bf16(c.v),
                    to_dev_i32(c.tables), to_dev_i32(c.ctx), SCALE, 10, out=out, workspace=ws)
    assert ops.read_error_word(ws) == 0
    c.check(out[:c.T], refs=refs)
    assert (out[c.T:] == 7.0).all()


def test_skipped_sequences_are_reported(ops):
    """Fewer keys than nodes, more nodes than max_q_len, a context past the table: each is
    skipped, the others are right."""
    c = Case(16, [50, 40, 30, 20], [3, 12, 2, 5], 6, 2)
    refs = c.reference()
    rows = np.concatenate([np.full(n, b == 3) for b, n in enumerate(c.nodes)])
    c.ctx[0], c.ctx[2] = 2, 16 * c.tables.shape[1] + 1
    ws = ops.tree_workspace()
    out = torch.full((c.T, 6, 128), 7.0, device="cuda")
    ops.decode_tree(to_dev_bf16(c.q), to_dev_i32(c.cu), to_dev_i32(c.parents), to_dev_bf16(c.k),
                    to_dev_bf16(c.v), to_dev_i32(c.tables), to_dev_i32(c.ctx), SCALE, 11, out=out,
                    workspace=ws)
    assert ops.read_error_word(ws, clear=True) == 8
    assert (out[:17] == 7.0).all()
    c.check(out, refs=refs, rows=rows)


@pytest.mark.parametrize("cu", [[0, 5, 3, 8], [-2, 3, 5, 8], [0, 3, 5, 9], [0, 2**31 - 1, 5, 8],
                                [5, -2**31, 3, 8]])
def test_bad_offsets_are_reported(ops, cu):
    c = Case(17, [50, 40, 30], [3, 2, 3], 6, 2)
    ws = ops.tree_workspace()
    ops.decode_tree(to_dev_bf16(c.q), to_dev_i32(cu), to_dev_i32(c.parents), to_dev_bf16(c.k),
                    to_dev_bf16(c.v), to_dev_i32(c.tables), to_dev_i32(c.ctx), SCALE, 8,
                    workspace=ws)
    assert ops.read_error_word(ws) & 8


@pytest.mark.parametrize("bad", [5, 6, 2**31 - 1, -2, -2**31])
def test_bad_parent_is_reported(ops, bad):
    c = Case(18, [50, 20], [10, 4], 6, 2)
    refs = c.reference()
    rows = np.array([5 not in ref.way(c.parents[:10], i) for i in range(10)] + [True] * 4)
    c.parents[5] = bad
    out, flags = c.run(ops, check=False)
    assert flags == 8
    c.check(out, refs=refs, rows=rows)


@pytest.mark.parametrize("bad", [-1, 10**6, 2**31 - 1, -2**31])
def test_bad_table_entry_is_reported(ops, bad):
    c = Case(19, [200, 50], [10, 4], 6, 2)
    refs = c.reference()
    c.tables[0, 3] = bad
    out, flags = c.run(ops, check=False)
    assert flags == 1
    c.check(out, refs=refs, rows=np.array([False] * 10 + [True] * 4))


def test_strided_tables_and_placement(ops):
    c = Case(20, [200, 50, 700], [10, 4, 30], 6, 2)
    out = c.run(ops)
    wide = torch.full((3, c.tables.shape[1] + 9), -3, dtype=torch.int32, device="cuda")
    wide[:, :c.tables.shape[1]] = to_dev_i32(c.tables)
    perm = np.random.default_rng(1).permutation(c.k.shape[0])
    k, v = np.empty_like(c.k), np.empty_like(c.v)
    k[perm], v[perm] = c.k, c.v
    moved = wide.clone()
    held = wide >= 0
    moved[held] = to_dev_i32(perm)[wide[held].long()]
    got = ops.decode_tree(to_dev_bf16(c.q), to_dev_i32(c.cu), to_dev_i32(c.parents),
                          to_dev_bf16(k), to_dev_bf16(v), moved, to_dev_i32(c.ctx), SCALE, 30,
                          out_dtype=torch.float32)
    assert torch.equal(got, out)


def test_streams_graphs_and_a_shared_workspace(ops):
    """Eager calls on two streams with workspaces of their own, and two captured graphs that
    share one, replayed in turn: the same bits everywhere."""
    a, b = Case(21, [900, 50], [30, 4], 6, 2), Case(22, [10, 2000, 64], [3, 9, 64], 8, 4)
    calls, want = [], []
    ws = ops.tree_workspace()
    for c in (a, b):
        args = (to_dev_bf16(c.q), to_dev_i32(c.cu), to_dev_i32(c.parents), to_dev_bf16(c.k),
                to_dev_bf16(c.v), to_dev_i32(c.tables), to_dev_i32(c.ctx), SCALE,
                int(c.nodes.max()))
        want.append(ops.decode_tree(*args))
        out = torch.empty_like(args[0])
        calls.append((ops.DecodeTreeCall(*args, out, workspace=ws), out, args))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [ops.decode_tree(*args, stream=s, pdl=True) for (_, _, args), s in zip(calls, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, want))
    graphs = []
    for call, _, _ in calls:
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
            call()
        graphs.append(g)
    for _ in range(3):
        for (_, out, _), g in zip(calls, graphs):
            out.fill_(float("nan"))
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, w) for (_, out, _), w in zip(calls, want))
    assert ops.read_error_word(ws) == 0
