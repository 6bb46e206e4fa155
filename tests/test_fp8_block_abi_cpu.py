"""Argument checks of the block-scaled FP8 cache's and the page operators'
entry points that run before any CUDA call: nothing is launched here."""
import ctypes

import pytest

FAKE = 0x10000  # never dereferenced: every call fails, or has nothing to do, before a launch
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from paged_kv_continuous_gb300 import build
    build.build()
    from paged_kv_continuous_gb300 import ops
    return ops.lib


def caller(fn, **defaults):
    def call(**kw):
        assert not set(kw) - set(defaults)
        return fn(*{**defaults, **kw}.values())
    return call


def test_store_kv_fp8_block(lib):
    call = caller(lib.pa_store_kv_fp8_block, k=FAKE, v=FAKE, k_tok=256, k_head=128, v_tok=256,
                  v_head=128, cu=FAKE, num_seqs=2, total=4, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE,
                  num_blocks=8, bs=16, hkv=2, d=128, bt=FAKE, stride=4, ctx=FAKE, err=None,
                  flags=0, stream=None)
    for name in ("k", "v", "cu", "kc", "vc", "ks", "vs", "bt", "ctx"):
        assert call(**{name: None}) == INVALID, name
    assert call(num_seqs=0, k=None) == OK and call(total=0, bt=None) == OK
    assert call(num_seqs=-1) == INVALID and call(total=-1) == INVALID
    assert call(num_blocks=-1) == INVALID and call(stride=0) == INVALID
    assert call(k_tok=-1) == INVALID and call(v_head=-8) == INVALID
    assert call(d=64) == UNSUPPORTED and call(bs=32) == UNSUPPORTED
    assert call(hkv=0) == UNSUPPORTED and call(hkv=65) == UNSUPPORTED
    assert call(flags=2) == INVALID and call(flags=4) == INVALID
    assert call(kc=FAKE + 8) == INVALID and call(vc=FAKE + 1) == INVALID
    assert call(k=FAKE + 1) == INVALID


def test_decode_fp8_block(lib):
    call = caller(lib.pa_decode_fp8_block, out=FAKE, dt=0, q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE,
                  vs=FAKE, num_blocks=8, bt=FAKE, stride=4, ctx=FAKE, batch=2, hq=12, hkv=2,
                  d=128, bs=16, scale=0.1, splits=0, ws=FAKE, ws_bytes=1 << 30, flags=0,
                  stream=None)
    for name in ("out", "q", "kc", "vc", "ks", "vs", "bt", "ctx"):
        assert call(**{name: None}) == INVALID, name
    assert call(batch=0, q=None) == OK and call(batch=-1) == INVALID
    assert call(ks=FAKE + 4) == INVALID and call(vs=FAKE + 1) == INVALID
    assert call(dt=2) == INVALID and call(scale=float("inf")) == INVALID
    assert call(d=64) == UNSUPPORTED and call(bs=8) == UNSUPPORTED
    assert call(hkv=3, hq=3) == UNSUPPORTED and call(hq=18) == UNSUPPORTED
    assert call(splits=5000) == UNSUPPORTED and call(splits=-1) == INVALID
    assert call(flags=2) == INVALID and call(flags=8) == INVALID
    assert call(out=FAKE + 2) == INVALID and call(kc=FAKE + 8) == INVALID
    assert call(stride=0) == INVALID


def test_prefill_fp8_block(lib):
    call = caller(lib.pa_prefill_fp8_block, out=FAKE, dt=0, q=FAKE, cu=FAKE, num_seqs=2, total=4,
                  max_q=3, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, num_blocks=8, bt=FAKE, stride=4,
                  ctx=FAKE, hq=12, hkv=2, d=128, bs=16, scale=0.1, err=None, stream=None)
    for name in ("out", "q", "cu", "kc", "vc", "ks", "vs", "bt", "ctx"):
        assert call(**{name: None}) == INVALID, name
    for name in ("num_seqs", "total", "max_q"):
        assert call(**{name: 0}) == OK and call(**{name: -1}) == INVALID
    assert call(dt=5) == INVALID and call(scale=float("nan")) == INVALID
    assert call(d=64) == UNSUPPORTED and call(hkv=16, hq=16) == UNSUPPORTED
    assert call(hq=18) == UNSUPPORTED and call(hq=13) == UNSUPPORTED
    assert call(num_seqs=65536) == UNSUPPORTED and call(num_blocks=0) == INVALID
    assert call(q=FAKE + 8) == INVALID and call(vc=FAKE + 4) == INVALID
    assert call(stride=0) == INVALID


def test_copy_pages(lib):
    from paged_kv_continuous_gb300.ops import _PagePool
    pools = (_PagePool * 2)()
    for p in pools:
        p.base, p.page_bytes = FAKE, 4096
    call = caller(lib.pa_copy_pages, pools=ctypes.addressof(pools), n=2, num_blocks=8, src=FAKE,
                  dst=FAKE, pairs=3, count=None, err=None, flags=0, stream=None)
    for name in ("pools", "src", "dst"):
        assert call(**{name: None}) == INVALID, name
    assert call(n=0) == OK and call(pairs=0, src=None) == OK
    assert call(n=-1) == INVALID and call(pairs=-1) == INVALID and call(num_blocks=-1) == INVALID
    assert call(num_blocks=1 << 31) == INVALID and call(flags=2) == INVALID
    pools[1].page_bytes = 0
    assert call() == INVALID
    pools[1].page_bytes = (1 << 31) + 1
    assert call() == INVALID
    pools[1].page_bytes, pools[1].base = 16, None
    assert call() == INVALID


def test_fork_and_free_pages(lib):
    fork = caller(lib.pa_fork_pages, bt=FAKE, stride=4, ctx=FAKE, rows=8, parents=FAKE,
                  children=FAKE, n=2, refs=FAKE, num_blocks=16, bs=16, src=FAKE, dst=FAKE,
                  forked=FAKE, err=None, flags=0, stream=None)
    for name in ("bt", "ctx", "parents", "children", "refs", "src", "dst", "forked"):
        assert fork(**{name: None}) == INVALID, name
    assert fork(n=0, bt=None) == OK and fork(n=-1) == INVALID and fork(rows=-1) == INVALID
    assert fork(stride=0) == INVALID and fork(bs=32) == UNSUPPORTED and fork(flags=2) == INVALID
    assert fork(num_blocks=1 << 31) == INVALID and fork(refs=FAKE + 2) == INVALID
    free = caller(lib.pa_free_pages, bt=FAKE, stride=4, ctx=FAKE, rows=8, seqs=FAKE, n=2,
                  refs=FAKE, num_blocks=16, bs=16, err=None, flags=0, stream=None)
    for name in ("bt", "ctx", "seqs", "refs"):
        assert free(**{name: None}) == INVALID, name
    assert free(n=0, bt=None) == OK and free(n=-1) == INVALID and free(stride=0) == INVALID
    assert free(bs=32) == UNSUPPORTED and free(flags=4) == INVALID
    assert free(bt=FAKE + 1) == INVALID


def test_compact_pages(lib):
    call = caller(lib.pa_compact_pages, bt=FAKE, stride=4, ctx=FAKE, rows=8, refs=FAKE,
                  num_blocks=16, bs=16, src=FAKE, dst=FAKE, counts=FAKE, remap=FAKE, err=None,
                  flags=0, stream=None)
    for name in ("bt", "ctx", "refs", "src", "dst", "counts", "remap"):
        assert call(**{name: None}) == INVALID, name
    assert call(rows=-1) == INVALID and call(num_blocks=-1) == INVALID
    assert call(stride=0) == INVALID and call(bs=32) == UNSUPPORTED and call(flags=2) == INVALID
    assert call(remap=FAKE + 2) == INVALID


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    from paged_kv_continuous_gb300 import ops
    i32 = dict(dtype=torch.int32)
    k, v, ks, vs = ops.fp8_block_pools(4, 2)
    assert k.shape == (4, 16, 2, 128) and v.shape == (4, 2, 128, 16) and ks.shape == vs.shape == (4, 2)
    q = torch.zeros(1, 12, 128, dtype=torch.bfloat16)
    t, c = torch.zeros(1, 2, **i32), torch.zeros(1, **i32)
    with pytest.raises(ops.PagedAttentionError, match="CUDA"):
        ops.decode_fp8_block(q, k, v, ks, vs, t, c, 0.1)
    with pytest.raises(ops.PagedAttentionError, match="CUDA"):
        ops.store_kv_fp8_block(q, q, k, v, ks, vs, c, t, c)
    with pytest.raises(ops.PagedAttentionError, match="CUDA"):
        ops.prefill_varlen_fp8_block(q, c, k, v, ks, vs, t, c, 0.1, 1)
    with pytest.raises(ops.PagedAttentionError, match="CUDA"):
        ops.PagePools([k, v])
    with pytest.raises(ops.PagedAttentionError, match="at least one"):
        ops.PagePools([])
    for fn in (lambda: ops.fork_pages(t, c, c, c, c), lambda: ops.free_pages(t, c, c, c),
               lambda: ops.compact_pages(t, c, c)):
        with pytest.raises(ops.PagedAttentionError, match="CUDA"):
            fn()
