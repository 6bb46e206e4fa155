"""The split of a query row into two E4M3 terms (the block-scaled prefill), by
enumeration of every bf16 magnitude that a scaled row can hold."""
import numpy as np

from paged_kv_continuous_gb300.synth import bf16_to_f64
from tests import fp8_block_reference as ref


def test_two_terms_of_every_bf16():
    """A row's largest magnitude a is scaled into (224, 448].  An element x is
    the sum of E4M3(x) and E4M3(x - E4M3(x)) exactly from 2^-9 a on (not from
    2^-10 a on), and within 2^-17 a below."""
    x = bf16_to_f64(np.arange(0x7F80, dtype=np.uint16))
    x = x[x <= 448]
    first = ref.VALUES[ref.encode(x)]
    err = np.abs(x - first - ref.VALUES[ref.encode(x - first)])
    smallest = x[x > 224].min()  # the least a: every bound is tightest there
    assert np.all(err[x >= 2.0 ** -9 * smallest] == 0)
    assert np.any(err[x >= 2.0 ** -10 * smallest] > 0)
    assert np.all(err <= 2.0 ** -17 * smallest)
