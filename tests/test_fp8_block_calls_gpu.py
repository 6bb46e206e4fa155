"""Ways to call the block-scaled cache's entry points: programmatic chains with
early page requests, steps over 4 and 8 kv heads in a graph, outputs in pinned
host memory, nothing to do."""
import numpy as np
import pytest
import torch

from tests import fp8_block_reference as ref
from tests.helpers import normal_bits, random_tables, to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu
SCALE = 1 / np.sqrt(128)
LENS = {"short": [20, 1, 0, 33, 16], "one block each": [5] * 20, "one long": [9000],
        "mixed": [3000, 17, 0, 700, 1, 1500, 64], "many": [40] * 360}


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def layer(rng, ctx, Hq, Hkv):
    NB = int(((ctx + 15) // 16).sum()) + 2
    q = to_dev_bf16(normal_bits(rng, (len(ctx), Hq, 128)))

    def codes(*shape):  # any finite ones
        return dev(rng.integers(0, 0x70, shape, dtype=np.uint8) |
                   (rng.integers(0, 2, shape, dtype=np.uint8) << 7))

    scales = [dev(rng.integers(115, 123, (NB, Hkv)).astype(np.uint8)) for _ in range(2)]
    return q, [codes(NB, 16, Hkv, 128), codes(NB, Hkv, 128, 16), *scales], NB


@pytest.mark.parametrize("Hkv", [1, 2, 4, 8])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("num_splits", [0, 9])
def test_chain_of_layers_with_early_pages(ops, lens, Hkv, num_splits):
    """Decodes of three layers, each with its own pools, one behind the other:
    the same bits plain, with pdl, with early pages and as a replayed graph."""
    rng = np.random.default_rng(Hkv + len(lens))
    ctx = np.array(LENS[lens], np.int32)
    Hq = 3 * Hkv
    layers = [layer(rng, ctx, Hq, Hkv) for _ in range(3)]
    tables = random_tables(rng, np.maximum(ctx, 0), layers[0][2])
    td, cd = to_dev_i32(tables), to_dev_i32(ctx)
    ws = ops.decode_workspace(Hq, Hkv, num_splits, 128, "cuda")
    want = None
    for kw in ({}, dict(pdl=True), dict(pdl=True, early_kv=True)):
        outs = [torch.empty((len(ctx), Hq, 128), dtype=torch.float32, device="cuda")
                for _ in layers]
        chain = [ops.DecodeFp8BlockCall(q, *pools, td, cd, SCALE, o, num_splits=num_splits,
                                        workspace=ws, **kw)
                 for (q, pools, _), o in zip(layers, outs)]
        for _ in range(10):
            for call in chain:
                call()
        torch.cuda.synchronize()
        if want is None:
            want = [o.clone() for o in outs]
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for call in chain:
                call()
        for _ in range(5):
            for o in outs:
                o.fill_(7.0)
            graph.replay()
            assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert ops.read_error_word(ws) == 0


@pytest.mark.parametrize("Hkv", [4, 8])
def test_steps_over_many_heads(ops, Hkv):
    """A store and a decode per step, chained with pdl, eager and replayed, from
    one-block sequences on: the merge kernel with and without anything to merge
    behind stores that change the pages it was given."""
    rng = np.random.default_rng(Hkv)
    B, Hq, steps = 6, 2 * Hkv, 40
    start = np.array([1, 9, 15, 16, 3, 0])
    NB = int(((start + steps + 15) // 16).sum()) + 2
    tables = random_tables(rng, start + steps, NB)
    cache = ref.random_cache(rng, NB, Hkv)
    pools, want = [dev(a) for a in cache], [a.copy() for a in cache]
    first = [p.clone() for p in pools]
    k, v, q = (normal_bits(rng, (steps, B, h, 128)) for h in (Hkv, Hkv, Hq))
    kd, vd, qd = to_dev_bf16(k[0]), to_dev_bf16(v[0]), to_dev_bf16(q[0])
    rows = [to_dev_bf16(a) for a in (k, v, q)]
    td, cd, cu = to_dev_i32(tables), to_dev_i32(start), to_dev_i32(np.arange(B + 1))
    out = torch.empty((B, Hq, 128), dtype=torch.float32, device="cuda")
    store = ops.StoreKvFp8BlockCall(kd, vd, *pools, cu, td, cd, pdl=True)
    decode = ops.DecodeFp8BlockCall(qd, *pools, td, cd, SCALE, out, pdl=True)

    def load(t):
        for to, x in zip((kd, vd, qd), rows):
            to.copy_(x[t])
        cd.copy_(to_dev_i32(start + t + 1))

    eager = []
    for t in range(steps):
        load(t)
        store()
        decode()
        eager.append(out.clone())
        now = (start + t + 1).astype(np.int32)
        ref.store(k[t], v[t], *want, np.arange(B + 1), tables, now)
        if t % 8 == 7 or t < 3:
            w, mag, tiny = ref.attention(q[t], *want, tables, now, SCALE)
            err = np.abs(eager[-1].double().cpu().numpy() - w)
            assert np.all(err <= ref.tolerance(w, mag, tiny)), t
    for p, w in zip(pools, want):
        assert np.array_equal(p.cpu().numpy(), w)
    for p, s in zip(pools, first):
        p.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        store()
        decode()
    for t in range(steps):
        load(t)
        graph.replay()
        assert torch.equal(out, eager[t]), t
    assert ops.read_error_word(decode.workspace) == 0


@pytest.mark.parametrize("Hkv", [2, 8])
def test_output_in_pinned_host_memory(ops, Hkv):
    rng = np.random.default_rng(Hkv)
    ctx = np.array([300, 0, 17, 2000], np.int32)
    q, pools, NB = layer(rng, ctx, 4 * Hkv, Hkv)
    tables = random_tables(rng, ctx, NB)
    td, cd = to_dev_i32(tables), to_dev_i32(ctx)
    want = ops.decode_fp8_block(q, *pools, td, cd, SCALE)
    out = torch.empty(q.shape, dtype=torch.bfloat16).pin_memory()
    ops.decode_fp8_block(q, *pools, td, cd, SCALE, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want.cpu())


def test_nothing_to_do(ops):
    """No sequences, no tokens, no pairs, no forks, an empty pool to compact."""
    pools = ops.fp8_block_pools(4, 2, device="cuda")
    before = [p.clone() for p in pools]
    none = torch.zeros((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((0, 12, 128), dtype=torch.bfloat16, device="cuda")
    t, c = torch.zeros((0, 3), dtype=torch.int32, device="cuda"), to_dev_i32([])
    ops.store_kv_fp8_block(none, none, *pools, to_dev_i32([0]), t, c)
    ops.store_kv_fp8_block(none, none, *pools, to_dev_i32([0, 0]), to_dev_i32([[0, 1, 2]]),
                           to_dev_i32([7]))
    assert ops.decode_fp8_block(q, *pools, t, c, SCALE).shape == (0, 12, 128)
    assert ops.prefill_varlen_fp8_block(q, to_dev_i32([0]), *pools, t, c, SCALE, 0).shape == q.shape
    assert ops.prefill_varlen_fp8_block(q, to_dev_i32([0, 0]), *pools, to_dev_i32([[0, 1, 2]]),
                                        to_dev_i32([7]), SCALE, 4).shape == q.shape
    refs = to_dev_i32([1, 0, 1, 0])
    tables, ctx = to_dev_i32([[0, 2]]), to_dev_i32([20])
    ops.copy_pages(ops.PagePools(pools), c, c)
    assert [x.numel() for x in ops.fork_pages(tables, ctx, c, c, refs)] == [0, 0, 0]
    ops.free_pages(tables, ctx, c, refs)
    src, dst, counts, remap = ops.compact_pages(t, c, to_dev_i32([]))
    assert counts.tolist() == [0, 0] and not src.numel() and not remap.numel()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(pools, before))
    assert refs.tolist() == [1, 0, 1, 0] and ctx.tolist() == [20]
