"""Argument checks of the speculative step's entry points that run before any
CUDA call: nothing is launched here."""
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


def test_workspace_size(lib):
    size = lib.pa_decode_tree_workspace_size
    assert size(0) == 0 and size(-1) == 0 and size(4097) == 0
    for s in (1, 7, 304, 4096):
        assert size(s) == 256 + s * (4 * 128 * 129 * 4 + 64)


def test_decode_tree(lib):
    call = caller(lib.pa_decode_tree, out=FAKE, dtype=0, q=FAKE, cu=FAKE, par=FAKE, num_seqs=2,
                  total=8, max_q=4, kc=FAKE, vc=FAKE, num_blocks=8, bt=FAKE, stride=4, ctx=FAKE,
                  hq=12, hkv=2, d=128, bs=16, scale=0.1, splits=4, ws=FAKE, bytes=1 << 30, flags=0,
                  stream=None)
    for name in ("out", "q", "cu", "par", "kc", "vc", "bt", "ctx"):
        assert call(**{name: None}) == INVALID, name
    assert call(ws=None) == WORKSPACE
    assert call(bytes=lib.pa_decode_tree_workspace_size(4) - 1) == WORKSPACE
    assert call(num_seqs=0, q=None) == OK and call(total=0, out=None) == OK
    assert call(max_q=0, ctx=None) == OK
    for name in ("num_seqs", "total", "max_q", "num_blocks", "splits"):
        assert call(**{name: -1}) == INVALID, name
    assert call(splits=4097) == INVALID and call(stride=0) == INVALID
    assert call(num_blocks=0) == INVALID and call(num_blocks=1 << 28) == INVALID
    assert call(dtype=2) == INVALID and call(flags=2) == INVALID and call(flags=4) == INVALID
    assert call(scale=float("nan")) == INVALID and call(scale=float("inf")) == INVALID
    assert call(d=64) == UNSUPPORTED and call(bs=32) == UNSUPPORTED
    assert call(hkv=3) == UNSUPPORTED and call(hq=13) == UNSUPPORTED
    assert call(hq=18) == UNSUPPORTED and call(hq=1) == UNSUPPORTED
    assert call(total=(1 << 26) + 1) == UNSUPPORTED
    # lists of tiles past an int: 1000 sequences of 2^27 table entries each
    assert call(num_seqs=1000, stride=1 << 27) == UNSUPPORTED
    for name in ("out", "q", "kc", "vc", "ws"):
        assert call(**{name: FAKE + 8}) == INVALID, name
    for name in ("cu", "par", "bt", "ctx"):
        assert call(**{name: FAKE + 2}) == INVALID, name


def test_verify_tree(lib):
    call = caller(lib.pa_verify_tree, accepted=FAKE, path=FAKE, out=FAKE, tokens=FAKE, par=FAKE,
                  cu=FAKE, num_seqs=2, total=8, max_q=4, p=FAKE, p_stride=100, q=FAKE, q_stride=100,
                  vocab=100, u=FAKE, last=FAKE, draws=0, err=None, flags=0, stream=None)
    for name in ("accepted", "path", "out", "tokens", "par", "cu", "p", "u", "last"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: FAKE + 2}) == INVALID, name
    assert call(q=FAKE + 1) == INVALID and call(err=FAKE + 1) == INVALID
    assert call(num_seqs=0, cu=None, p=None) == OK
    for name in ("num_seqs", "total", "max_q", "vocab"):
        assert call(**{name: -1}) == INVALID, name
    assert call(vocab=0, p_stride=0, q_stride=0) == INVALID
    assert call(p_stride=99) == INVALID and call(q_stride=99) == INVALID
    assert call(draws=2) == INVALID and call(draws=-1) == INVALID
    assert call(flags=2) == INVALID and call(flags=8) == INVALID
    assert call(vocab=(1 << 20) + 1, p_stride=1 << 21, q_stride=1 << 21) == UNSUPPORTED
    assert call(num_seqs=1 << 30) == UNSUPPORTED


class Pool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_int64)]


def test_commit_tree(lib):
    def pools(*pairs):
        return ctypes.addressof(keep.setdefault(pairs, (Pool * len(pairs))(*pairs)))
    keep = {}
    call = caller(lib.pa_commit_tree, pools=pools((FAKE, 8192)), n=1, num_blocks=8, bt=FAKE,
                  stride=4, ctx=FAKE, cu=FAKE, num_seqs=2, path=FAKE, width=4, accepted=FAKE,
                  refs=FAKE, bs=16, err=None, flags=0, stream=None)
    for name in ("pools", "bt", "ctx", "cu", "path", "accepted"):
        assert call(**{name: None}) == INVALID, name
    for name in ("bt", "ctx", "cu", "path", "accepted", "refs", "err"):
        assert call(**{name: FAKE + 2}) == INVALID, name
    assert call(num_seqs=0, bt=None) == OK
    for name in ("n", "num_blocks", "num_seqs", "width"):
        assert call(**{name: -1}) == INVALID, name
    assert call(num_blocks=0) == INVALID and call(num_blocks=1 << 28) == INVALID
    assert call(stride=0) == INVALID and call(flags=2) == INVALID
    assert call(bs=32) == UNSUPPORTED and call(num_seqs=1 << 30) == UNSUPPORTED
    for bad in ((None, 8192), (FAKE, 0), (FAKE, -16), (FAKE, 8200), (FAKE, (1 << 31) + 16)):
        assert call(pools=pools(bad)) == INVALID, bad
