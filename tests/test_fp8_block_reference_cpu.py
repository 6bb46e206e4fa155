"""The reference's own pins: its codec against torch's conversions, its scale
rule against its definition, and its store against closed forms."""
import numpy as np
import torch

from paged_kv_continuous_gb300.synth import bf16_bits, bf16_to_f64
from tests import fp8_block_reference as ref


def test_codec_matches_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.VALUES, want, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 8, 20000),
                        ref.VALUES[:127], -ref.VALUES[:127],
                        (ref.VALUES[:126] + ref.VALUES[1:127]) / 2]).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(x), want)
    assert ref.encode(np.inf) == 0x7E and ref.encode(-1e9) == 0xFE and ref.encode(np.nan) == 0x7F


def test_scale_rule():
    assert ref.scale_exponent(448.0) == 0 and ref.scale_exponent(449.0) == 1
    assert ref.scale_exponent(224.0) == -1 and ref.scale_exponent(0.0) == -40
    assert ref.scale_exponent(1e30) == 40


def test_appending_one_by_one_equals_one_chunk_but_for_subnormals():
    """Powers of two: however the rows arrive, the codes are the same unless
    a re-coded one became subnormal, where it may be one step off."""
    rng = np.random.default_rng(1)
    n, H, D = 37, 2, 128
    rows = bf16_bits(rng.standard_normal((n, H, D)) * 2.0 ** rng.integers(-3, 4, (n, 1, 1)))
    tables = np.array([[2, 0, 1]], np.int32)
    pools = []
    for step in (n, 1):
        kc, vc = np.zeros((3, 16, H, D), np.uint8), np.zeros((3, H, D, 16), np.uint8)
        ks, vs = np.full((3, H), 99, np.uint8), np.full((3, H), 99, np.uint8)
        for t in range(0, n, step):
            ref.store(rows[t:t + step], rows[t:t + step], kc, vc, ks, vs, [0, step], tables,
                      [t + step])
        pools.append((kc, vc, ks, vs))
    (ka, va, sa, ta), (kb, vb, sb, tb) = pools
    assert np.array_equal(sa, sb) and np.array_equal(ta, tb)
    for a, b in ((ka, kb), (va, vb)):
        same = a == b
        assert np.all(same | (np.abs(ref.VALUES[a]) < 2.0 ** -6))
        assert np.max(np.abs(ref.VALUES[a] - ref.VALUES[b])) <= 2.0 ** -9
    wide = ref.widen(ka, va, sa, ta)[0].reshape(-1, H, D)
    at = tables[0].astype(int)
    got = np.concatenate([ref.widen(ka, va, sa, ta)[0][at[j]] for j in range(3)])[:n]
    x = bf16_to_f64(rows)
    top = np.array([np.abs(x[16 * j:16 * j + 16]).max((0, 2)) for j in range(3)])
    step = np.repeat(top, 16, 0)[:n, :, None] / 224 * 2.0 ** -10
    assert np.all(np.abs(got - x) <= np.abs(x) * 2.0 ** -4 + step)
    assert wide.shape[0] == 48
