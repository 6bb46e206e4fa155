"""Calls enqueued one behind another with nothing between them: what a call
writes must not reach the one before it.  A decode over 4 or 8 kv heads whose
sequences all lie in one split launches a merge kernel with nothing to merge,
and the page operators and the block-scaled append start as programmatic
dependents of that kernel."""
import numpy as np
import pytest
import torch

from tests import fp8_block_reference as ref
from tests.helpers import normal_bits, random_tables, to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu
SCALE = 1 / np.sqrt(128)
LENS = {"one short": [20], "one block": [16, 1, 9, 12, 16, 7, 2, 16],
        "two blocks": [17, 32, 25, 31, 18, 29] * 3 + [32], "empty beside": [0, 30, 0, 0, 17, 0],
        "all empty": [0, 0, 0]}


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def decoder(ops, kind, rng, ctx, tables, NB, hkv):
    """(pools, call): the pools' tensors and a call that enqueues the decode."""
    B, hq = len(ctx), 4 * hkv
    q, td, cd = to_dev_bf16(normal_bits(rng, (B, hq, 128))), to_dev_i32(tables), to_dev_i32(ctx)
    out = torch.empty((B, hq, 128), dtype=torch.float32, device="cuda")
    ws = ops.decode_workspace(hq, hkv, 0, 128, "cuda")
    if kind == "bf16":
        pools = [to_dev_bf16(normal_bits(rng, (NB, 16, hkv, 128))) for _ in range(2)]
        fn = lambda: ops.decode(q, *pools, td, cd, SCALE, out=out, workspace=ws)
    elif kind == "fp8":
        pools = [dev(a) for a in ref.random_cache(rng, NB, hkv)[:2]]
        one = torch.ones(hkv, device="cuda")
        fn = lambda: ops.decode_fp8(q, *pools, one, one, td, cd, SCALE, out=out, workspace=ws)
    else:
        pools = [dev(a) for a in ref.random_cache(rng, NB, hkv)]
        fn = ops.DecodeFp8BlockCall(q, *pools, td, cd, SCALE, out, workspace=ws)
    return pools, fn, out, ws


@pytest.mark.parametrize("kind", ["block", "fp8", "bf16"])
@pytest.mark.parametrize("hkv", [4, 8])
@pytest.mark.parametrize("lens", list(LENS))
def test_pages_overwritten_right_behind_a_decode(ops, lens, hkv, kind):
    """Every page that the decode reads is overwritten by the copy behind it."""
    rng = np.random.default_rng(hkv + len(lens))
    ctx = np.array(LENS[lens], np.int32)
    NB = 2 * (int(((ctx + 15) // 16).sum()) + 1)
    tables = random_tables(rng, ctx, NB // 2)
    pools, decode, out, ws = decoder(ops, kind, rng, ctx, tables, NB, hkv)
    start = [p.clone() for p in pools]
    half = np.arange(NB // 2)
    over = ops.CopyPagesCall(ops.PagePools(pools), to_dev_i32(half + NB // 2), to_dev_i32(half))
    decode()
    torch.cuda.synchronize()
    want = out.clone()
    for _ in range(100):
        for p, s in zip(pools, start):
            p.copy_(s)
        decode()
        over()
        assert torch.equal(out, want)
    assert ops.read_error_word(ws) == 0


@pytest.mark.parametrize("hkv", [4, 8])
def test_store_right_behind_a_decode(ops, hkv):
    """An append that grows the scale of the pages the decode reads."""
    rng = np.random.default_rng(hkv)
    ctx = np.array([17, 30, 25, 9, 15], np.int32)
    NB = 12
    tables = random_tables(rng, ctx, NB)
    pools, decode, out, ws = decoder(ops, "block", rng, ctx, tables, NB, hkv)
    start = [p.clone() for p in pools]
    big = to_dev_bf16(normal_bits(rng, (5, hkv, 128))) * 1024
    store = ops.StoreKvFp8BlockCall(big, big, *pools, to_dev_i32(np.arange(6)),
                                    to_dev_i32(tables), to_dev_i32(ctx + 1))
    decode()
    torch.cuda.synchronize()
    want = out.clone()
    for _ in range(100):
        for p, s in zip(pools, start):
            p.copy_(s)
        decode()
        store()
        assert torch.equal(out, want)
    assert ops.read_error_word(ws) == 0


def test_free_fork_and_copy_right_behind_a_decode(ops):
    """The rows a decode reads are freed and forked anew, their pages taken
    and copied over, while nothing waits for it."""
    rng = np.random.default_rng(3)
    hkv, rows, NB = 8, 6, 40
    ctx = np.array([20, 31, 0, 0, 0, 0], np.int32)
    tables = np.full((rows, 2), -1, np.int32)
    tables[:2] = [[0, 1], [2, 3]]
    refs = np.zeros(NB, np.int32)
    refs[:4] = 1
    pools, _, _, _ = decoder(ops, "block", rng, ctx, tables, NB, hkv)
    t, c, r = to_dev_i32(tables), to_dev_i32(ctx), to_dev_i32(refs)
    q = to_dev_bf16(normal_bits(rng, (rows, 4 * hkv, 128)))
    out = torch.empty((rows, 4 * hkv, 128), dtype=torch.float32, device="cuda")
    decode = ops.DecodeFp8BlockCall(q, *pools, t, c, SCALE, out)
    fork = ops.ForkPagesCall(t, c, to_dev_i32([0, 1]), to_dev_i32([4, 5]), r)
    free = ops.FreePagesCall(t, c, to_dev_i32([0, 1]), r)
    again = ops.ForkPagesCall(t, c, to_dev_i32([5, 4, 4]), to_dev_i32([0, 1, 2]), r)
    copies = [ops.CopyPagesCall(ops.PagePools(pools), f.copy_src, f.copy_dst)
              for f in (fork, again)]
    start = [x.clone() for x in (*pools, t, c, r)]
    outs = []
    for synchronised in [True] + [False] * 50:
        for x, s in zip((*pools, t, c, r), start):
            x.copy_(s)
        for step in (fork, copies[0], decode, free, again, copies[1], decode):
            step()
            if step is decode:
                outs.append(out.clone())
            if synchronised:
                torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, outs[i % 2]), i
