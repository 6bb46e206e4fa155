"""NumPy float64 definitions of the speculative step: attention of a tree of
drafted nodes, their verification, and the commit of the accepted ones."""
from __future__ import annotations

import numpy as np

from paged_kv_continuous_gb300.synth import bf16_to_f64


def random_parents(rng, n, arity=3):
    """Parents of a random tree of n nodes (node 0 the root, parent -1)."""
    kids, par = np.zeros(n, int), [-1]
    for i in range(1, n):
        free = np.flatnonzero(kids[:i] < arity)
        j = int(free[max(rng.integers(len(free)), rng.integers(len(free)))])
        kids[j] += 1
        par.append(j)
    return np.array(par[:n], np.int32)


def way(parents, i):
    """Node i and those before it, up to the root."""
    out = []
    while i >= 0:
        out.append(i)
        i = int(parents[i])
    return out


def attention(q, k_pool, v_pool, tables, ctx, cu, parents, scale):
    """(out, a, s): the rows [T, Hq, D], the same sums over |V|, and the largest
    sum |q k| of each row's scores.  Bit patterns in, float64 out."""
    T, Hq, D = q.shape
    Hkv = k_pool.shape[2]
    G = Hq // Hkv
    qf = bf16_to_f64(q)
    out, a, big = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(len(cu) - 1):
        lo, n, done = int(cu[b]), int(cu[b + 1] - cu[b]), int(ctx[b] - (cu[b + 1] - cu[b]))
        if n == 0:
            continue
        pos = np.arange(ctx[b])
        slots = tables[b, pos // 16], pos % 16
        K, V = bf16_to_f64(k_pool[slots]), bf16_to_f64(v_pool[slots])
        for i in range(n):
            seen = np.concatenate([np.arange(done), done + np.array(sorted(way(parents[lo:lo + n], i)))])
            for h in range(Hq):
                kk, vv, x = K[seen, h // G], V[seen, h // G], qf[lo + i, h]
                s = scale * (kk @ x)
                w = np.exp(s - s.max())
                w /= w.sum()
                out[lo + i, h], a[lo + i, h] = w @ vv, w @ np.abs(vv)
                big[lo + i, h] = (np.abs(kk) @ np.abs(x)).max()
    return out, a, big


def attention_bound(out, a, big, scale, keys, bf16_out):
    """How far a row may be off, from its roundings, u = 2^-24:
    a score is a sum of 128 products in fp32, each addition off by at most 2 u (a
    truncating adder) of the sum of magnitudes; the scaling, the subtraction of the
    reference and the exponential (2^-22) add 2^-20 to a weight's relative
    error for scores up to 8 or so past the reference; the last of a weight's bf16
    terms is rounded, the second of two (at 2^-16 of the weight or less), or for
    fp32 rows of few keys the third of three; weights and products are added in fp32 (2 u for
    each of `keys` additions, numerator and denominator); the merge of pieces and the
    division add 2^-20.  The output is rounded by half a step."""
    score = abs(scale) * 128 * 2.0 ** -23 * big[..., None]
    # (up to 12 tiles of 64 keys a piece, of which 512 keys are eight at most)
    terms = 2.0 ** -16 if bf16_out or keys > 512 else 2.0 ** -24
    rel = 2 * score + terms + 2 * 2.0 ** -20 + 2 * keys * 2.0 ** -23
    return rel * a + (2.0 ** -8 if bf16_out else 2.0 ** -24) * np.abs(out) + 1e-30


LEAST = 2.0 ** -24


def verify(tokens, parents, p, q, u, u_last, again=False):
    """One tree: (path, tokens after it).  p, q: [n, V] (q None: looked up)."""
    n, V = p.shape
    path, new = [0], []
    while True:
        c = path[-1]
        row = p[c].astype(np.float64)
        beta, W, gone, found = 0.0, 1.0, 0.0, None
        for i in range(c + 1, n):
            x = int(tokens[i])
            if parents[i] != c or not 0 <= x < V:
                continue
            if q is None:
                if u[i] * W < row[x]:
                    found = i
                    break
                W, row[x] = max(W - row[x], 0.0), 0.0
                continue
            left, qx = max(1.0 - gone, LEAST), float(q[c, x])
            if u[i] * (qx / left) * W < float(p[c, x]) - beta * qx:
                found = i
                break
            beta += W / left
            if not again:
                gone += qx
            row = np.maximum(p[c].astype(np.float64) - beta * q[c].astype(np.float64), 0.0)
            W = row.sum()
        if found is None:
            break
        path.append(found)
        new.append(int(tokens[found]))
    if not row.sum() > 0:
        row = p[c].astype(np.float64)
    C = np.cumsum(row)
    if not C[-1] > 0:
        return path, new + [-1]
    over = np.flatnonzero((C > u_last * C[-1]) & (row > 0))
    return path, new + [int(over[0]) if len(over) else int(np.flatnonzero(row > 0)[-1])]


def verify_all(cu, tokens, parents, p, q, u, u_last, width, again=False):
    B = len(cu) - 1
    count = np.zeros(B, np.int32)
    path, new = np.full((B, width), -1, np.int32), np.full((B, width), -1, np.int32)
    for b in range(B):
        a, e = int(cu[b]), int(cu[b + 1])
        if a == e:
            continue
        w, t = verify(tokens[a:e], parents[a:e], p[a:e], None if q is None else q[a:e],
                      u[a:e].astype(np.float64), float(u_last[b]), again)
        count[b] = len(w)
        path[b, :len(w)], new[b, :len(t)] = w, t
    return count, path, new


def commit(pools, tables, ctx, cu, path, count, refs=None):
    """Changes the pools ([NB, 16, ...]), lengths and counts in place."""
    for b in range(len(ctx)):
        n = int(cu[b + 1] - cu[b])
        done = int(ctx[b]) - n
        src = done + path[b, :count[b]].astype(int)
        dst = done + np.arange(count[b])
        for x in pools:
            rows = x[tables[b, src // 16], src % 16].copy()
            x[tables[b, dst // 16], dst % 16] = rows
        new = done + int(count[b])
        if refs is not None and n:
            np.subtract.at(refs, tables[b, (new + 15) // 16:(ctx[b] + 15) // 16], 1)
        ctx[b] = new
