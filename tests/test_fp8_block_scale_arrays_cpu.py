"""Where the scale arrays of the block-scaled decode may start.  No call gets
past its workspace check: nothing is launched."""
import pytest

FAKE = 0x10000
INVALID, WORKSPACE, DEVICE = 1, 3, 5


@pytest.fixture(scope="module")
def lib():
    from paged_kv_continuous_gb300 import build
    build.build()
    from paged_kv_continuous_gb300 import ops
    return ops.lib


@pytest.mark.parametrize("hkv", [1, 2, 4, 8])
def test_scale_arrays_are_aligned_to_a_blocks_bytes(lib, hkv):
    def call(k, v):
        return lib.pa_decode_fp8_block(FAKE, 0, FAKE, FAKE, FAKE, FAKE + k, FAKE + v, 8, FAKE, 4,
                                       FAKE, 2, 2 * hkv, hkv, 128, 16, 0.1, 0, FAKE, 0, 0, None)
    for at in range(16):
        if at % hkv:
            assert call(at, at) == INVALID, at
        else:
            assert call(at, at) in (WORKSPACE, DEVICE), at
        if at % 8:
            assert call(at, 0) == INVALID and call(8, at) == INVALID, at
