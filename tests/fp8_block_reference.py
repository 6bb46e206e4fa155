"""Plain NumPy float64 definitions of the block-scaled FP8 cache (test code):
the E4M3 codec, the appending store block by block, and the attention over
the widened pools.  Nothing here is shared with the library."""
from __future__ import annotations

import numpy as np

from paged_kv_continuous_gb300.synth import bf16_to_f64

BIAS, E_MIN, E_MAX = 127, -40, 40


def code_values():
    """float64 value of each of the 256 E4M3 codes."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = np.nan if (c & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = -mag if c & 128 else mag
    return v


VALUES = code_values()


def encode(x):
    """Nearest E4M3 code (ties to even), saturated to +-448; NaN -> 0x7F | sign."""
    x = np.asarray(x, np.float64)
    pos = VALUES[:127]  # ascending, code = index
    a = np.minimum(np.abs(x), 448.0)
    nan = np.isnan(x)
    a = np.where(nan, 0.0, a)
    hi = np.minimum(np.searchsorted(pos, a, side="left"), 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = pos[hi] - a, a - pos[lo]
    code = np.where(dh < dl, hi, np.where(dh > dl, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(a == pos[hi], hi, code)
    code = np.where(nan, 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_exponent(a):
    """Smallest e in [E_MIN, E_MAX] with a <= 448 * 2^e (E_MAX if none)."""
    for e in range(E_MIN, E_MAX):
        if a <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


def store(k, v, kc, vc, ks, vs, cu, tables, ctx):
    """Appends in place.  k, v uint16 [T, H, D]; kc [NB, 16, H, D], vc
    [NB, H, D, 16], ks / vs [NB, H] uint8."""
    for s in range(len(ctx)):
        q = int(cu[s + 1] - cu[s])
        first = int(ctx[s]) - q
        pos = np.arange(first, int(ctx[s]))
        for j in np.unique(pos // 16):
            page = int(tables[s, j])
            mine = pos[pos // 16 == j]
            rows = mine % 16
            tok = int(cu[s]) + mine - first
            r0 = int(rows[0])
            for new, cache, scale, dim_major in ((k, kc, ks, False), (v, vc, vs, True)):
                for h in range(new.shape[1]):
                    x = bf16_to_f64(new[tok, h])
                    fin = np.abs(x[np.isfinite(x)])
                    e = scale_exponent(fin.max() if fin.size else 0.0)
                    # [16 rows, D] view of this block and head
                    blk = cache[page, h].T if dim_major else cache[page, :, h]
                    if r0 > 0:
                        old = int(scale[page, h]) - BIAS
                        e = max(e, old)
                        if e > old:
                            blk[:r0] = encode(VALUES[blk[:r0]] * 2.0 ** (old - e))
                    blk[rows] = encode(x * 2.0 ** -e)
                    scale[page, h] = e + BIAS


def widen(kc, vc, ks, vs):
    """Values [NB, 16, H, D] of both pools."""
    ek = 2.0 ** (np.clip(ks.astype(int) - BIAS, E_MIN, E_MAX))
    ev = 2.0 ** (np.clip(vs.astype(int) - BIAS, E_MIN, E_MAX))
    return (VALUES[kc] * ek[:, None, :, None],
            (VALUES[vc] * ev[:, :, None, None]).transpose(0, 3, 1, 2))


def attention(q, kc, vc, ks, vs, tables, ctx, scale, cu=None):
    """(out, room) float64 [T, Hq, D]: the attention of the last q_len
    positions of each sequence (one each without cu), and what bounds the
    error of a computation with f16 weights (see ``tolerance``): sum of
    weight times |v|, and the number of keys times the largest V scale."""
    T, Hq, D = q.shape
    H = kc.shape[2]
    cu = np.arange(len(ctx) + 1) if cu is None else cu
    out, mag, tiny = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq, 1))
    qf = bf16_to_f64(q)
    for s in range(len(ctx)):
        n, m = int(ctx[s]), int(cu[s + 1] - cu[s])
        if n <= 0 or m == 0:
            continue
        pages = tables[s, :(n + 15) // 16].astype(int)
        kk, vv = widen(kc[pages], vc[pages], ks[pages], vs[pages])
        kk, vv = (a.reshape(-1, H, D)[:n] for a in (kk, vv))
        top = 2.0 ** (np.clip(vs[pages].astype(int) - BIAS, E_MIN, E_MAX)).max(0)
        for i in range(m):
            keys = n - m + i + 1
            for h in range(Hq):
                g = h * H // Hq
                sc = scale * (kk[:keys, g] @ qf[cu[s] + i, h])
                w = np.exp(sc - sc.max())
                w /= w.sum()
                out[cu[s] + i, h] = w @ vv[:keys, g]
                mag[cu[s] + i, h] = w @ np.abs(vv[:keys, g])
                tiny[cu[s] + i, h] = keys * top[g]
    return out, mag, tiny


def tolerance(ref, mag, tiny, bf16_out=False, score=64.0):
    """Bound of |got - ref| by arithmetic.  Each weight times V scale is
    rounded to f16: half a step, 2^-11 of it, or 2^-25 absolutely where it is
    subnormal, against a reference of at least 1 in units of the largest V
    scale, times a code of at most 448.  A score of magnitude ``score`` (base
    2) is rounded in fp32, a few times 2^-24 of it, which the exponential turns
    into as much of the weight, and so into at most that of both sums; fp32
    accumulation adds 2^-16 of the sum of magnitudes at these lengths."""
    exp_err = 2 * 4 * score * 2.0 ** -24
    bound = mag * (2.0 ** -11 + exp_err + 2.0 ** -16) + tiny * (448 * 2.0 ** -25) + 1e-30
    if bf16_out:
        bound = bound + (np.abs(ref) + bound) * 2.0 ** -8
    return bound


def random_cache(rng, NB, H, D=128, e_lo=-9, e_hi=-5):
    """Pools of random finite codes (N(0, 1) rows at each block's own scale)."""
    kc = encode(rng.standard_normal((NB, 16, H, D)) * 90)
    vc = encode(rng.standard_normal((NB, H, D, 16)) * 90)
    ks = rng.integers(e_lo, e_hi + 1, (NB, H)) + BIAS
    vs = rng.integers(e_lo, e_hi + 1, (NB, H)) + BIAS
    return kc, vc, ks.astype(np.uint8), vs.astype(np.uint8)
