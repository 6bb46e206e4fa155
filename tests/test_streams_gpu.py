"""Default outputs and workspaces of calls on another stream than the current
one: right while the current stream is busy (with the fill of memory that the
allocator would hand out next), and not held up by it."""
import numpy as np
import pytest
import torch

from tests import fp8_block_reference as ref
from tests.helpers import normal_bits, random_tables, to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu
SCALE = 1 / np.sqrt(128)
LONG = 200_000_000  # cycles that the current stream sleeps, about 0.1 s


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


@pytest.fixture(scope="module")
def data(ops):
    rng = np.random.default_rng(1)
    ctx = np.array([3000, 700, 1, 1500], np.int32)
    NB = 400
    tables = random_tables(rng, ctx, NB)
    cache = [torch.from_numpy(a).cuda() for a in ref.random_cache(rng, NB, 2)]
    bf16 = [to_dev_bf16(normal_bits(rng, (NB, 16, 2, 128))) for _ in range(2)]
    q = to_dev_bf16(normal_bits(rng, (4, 12, 128)))
    return cache, bf16, q, to_dev_i32(tables), to_dev_i32(ctx)


def keep_busy(*tensors):
    """The current stream sleeps, then fills memory that it let go of: what it
    allocates next starts as garbage, late.  Returns the event of its end."""
    for _ in range(4):
        for n in (1 << 20, 1 << 22, 1 << 24):
            del_me = torch.empty(n, dtype=torch.uint8, device="cuda")
            del_me.fill_(255)
            del del_me
    torch.cuda._sleep(LONG)
    late = [torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    del late
    end = torch.cuda.Event()
    end.record()
    return end


def calls(ops, data):
    cache, bf16, q, td, cd = data
    one = torch.ones(2, device="cuda")
    cu = torch.arange(5, dtype=torch.int32, device="cuda")
    refs = torch.zeros(400, dtype=torch.int32, device="cuda")
    t2, c2 = td.clone(), cd.clone()
    return {
        "decode block": lambda s: ops.decode_fp8_block(q, *cache, td, cd, SCALE, stream=s),
        "prefill block": lambda s: ops.prefill_varlen_fp8_block(q, cu, *cache, td, cd, SCALE, 1,
                                                                stream=s),
        "decode fp8": lambda s: ops.decode_fp8(q, *cache[:2], one, one, td, cd, SCALE, stream=s),
        "decode": lambda s: ops.decode(q, *bf16, td, cd, SCALE, stream=s),
        "prefill": lambda s: ops.prefill_varlen(q, cu, *bf16, td, cd, SCALE, 1, stream=s),
        "compact": lambda s: ops.compact_pages(t2[:0], c2[:0], refs, stream=s)[3],
    }


NAMES = ["decode block", "prefill block", "decode fp8", "decode", "prefill", "compact"]


@pytest.mark.parametrize("name", NAMES)
def test_default_buffers_on_another_stream(ops, data, name):
    fn = calls(ops, data)[name]
    want = fn(None).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for turn in range(3):
        end = keep_busy()
        got = [fn(side) for _ in range(5)]
        side.synchronize()
        held_up = end.query()
        for g in got:
            g.record_stream(torch.cuda.current_stream())
            assert torch.equal(g, want)
        assert turn == 0 or not held_up  # (the first turn's allocations may synchronise)
        torch.cuda.synchronize()


def test_prepared_call_made_on_a_busy_stream(ops, data):
    """Its workspace is zeroed late there; another stream waits for that, and
    the memory outlives the object's last call."""
    cache, _, q, td, cd = data
    want = ops.decode_fp8_block(q, *cache, td, cd, SCALE)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        out = torch.empty_like(q)
        torch.cuda.synchronize()
        keep_busy()
        call = ops.DecodeFp8BlockCall(q, *cache, td, cd, SCALE, out)
        for _ in range(4):
            call(side)
        del call  # (its workspace stays its own until the side stream is done)
        other = torch.full((1 << 23,), 255, dtype=torch.uint8, device="cuda")
        side.synchronize()
        assert torch.equal(out, want)
        del other


def test_prepared_call_with_defaults_captured(ops, data):
    """Made on the current stream, captured on the graph's own, replayed."""
    cache, _, q, td, cd = data
    want = ops.decode_fp8_block(q, *cache, td, cd, SCALE)
    out = torch.empty_like(q)
    call = ops.DecodeFp8BlockCall(q, *cache, td, cd, SCALE, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(5):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    assert ops.read_error_word(call.workspace) == 0


def test_store_decode_call_made_on_a_busy_stream(ops):
    rng = np.random.default_rng(2)
    ctx = np.array([40, 900], np.int32)
    tables = random_tables(rng, ctx, 80)
    pools = [to_dev_bf16(normal_bits(rng, (80, 16, 2, 128))) for _ in range(2)]
    q, nk, nv = (to_dev_bf16(normal_bits(rng, (2, h, 128))) for h in (12, 2, 2))
    slots = to_dev_i32([tables[b, (n - 1) // 16] * 16 + (n - 1) % 16 for b, n in enumerate(ctx)])
    td, cd = to_dev_i32(tables), to_dev_i32(ctx)
    want = ops.store_decode(q, nk, nv, *pools, slots, td, cd, SCALE)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    keep_busy()
    call = ops.StoreDecodeCall(q, nk, nv, *pools, slots, td, cd, SCALE, out)
    call(side)
    side.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("name", NAMES)
def test_output_used_and_dropped_on_the_current_stream(ops, data, name):
    """The output of a call on another stream, read late by the current one and
    let go at once: later calls on that stream do not get its memory early."""
    fn = calls(ops, data)[name]
    want = fn(None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = fn(side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(LONG // 4)
        late = got.clone()  # runs when the sleep is over
        shape, dtype = got.shape, got.dtype
        del got
        with torch.cuda.stream(side):
            for _ in range(4):
                torch.full(shape, 1, dtype=dtype, device="cuda")
        side.synchronize()
        assert torch.equal(late, want)
