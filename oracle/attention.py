"""fp64 oracle of the softmax-attention operators (NumPy, row by row from the definitions).

For attention it also returns, per output element, sum_j w_ij |v_j|: the amount that a
relative error on each weight can move the output, which the tests' tolerances are made of.
"""
from __future__ import annotations

import numpy as np


def attend(q, k, v, last, scale):
    """q [r, D]; k, v [n, D]; row i sees keys 0 .. last[i]. Returns (out, weighted |v|, lse);
    a row that sees nothing gives zeros and -inf. Unseen rows of k and v are not touched."""
    r, D = q.shape
    out, mag, lse = np.zeros((r, D)), np.zeros((r, D)), np.full(r, -np.inf)
    for i in range(r):
        n = min(int(last[i]) + 1, k.shape[0])
        if n <= 0:
            continue
        s = scale * (k[:n] @ q[i])
        m = s.max()
        w = np.exp(s - m)
        lse[i] = m + np.log(w.sum())
        w /= w.sum()
        out[i], mag[i] = w @ v[:n], w @ np.abs(v[:n])
    return out, mag, lse


def sane_bounds(cu, T):
    """cu_seqlens with entries clamped to [0, T] and raised to the largest before them."""
    return np.maximum.accumulate(np.clip(np.asarray(cu, np.int64), 0, T))


def prefill(q, k, v, cu=None, scale=None):
    """q [T, H, D], k, v [T, Hk, D] -> (out, mag, lse, rows inside a sequence)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    T, H, D = q.shape
    G = H // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    cu = sane_bounds([0, T] if cu is None else cu, T)
    out, mag, lse = np.zeros((T, H, D)), np.zeros((T, H, D)), np.full((T, H), -np.inf)
    inside = np.zeros(T, bool)
    for b, e in zip(cu[:-1], cu[1:]):
        inside[b:e] = True
        for h in range(H):
            out[b:e, h], mag[b:e, h], lse[b:e, h] = attend(
                q[b:e, h], k[b:e, h // G], v[b:e, h // G], np.arange(e - b), scale)
    return out, mag, lse, inside


def gather(cache, table, n, length, h, page, shared):
    """Rows 0 .. length - 1 of sequence n's keys (or values) of key head h; the columns of
    the shared prefix come from the table's first row; pages that do not exist are zeros."""
    rows = np.zeros((length, cache.shape[3]))
    for j in range(0, length, page):
        p = int(table[0 if j < shared else n, j // page])
        if 0 <= p < cache.shape[0]:
            c = min(page, length - j)
            rows[j:j + c] = cache[p, h, :c]
    return rows


def decode(q, k_cache, v_cache, table, kv_lens, shared=0, scale=None):
    """q [N, n_q, H, D] -> (out, mag, lse)."""
    q, k_cache, v_cache = (np.asarray(x, np.float64) for x in (q, k_cache, v_cache))
    N, nq, H, D = q.shape
    _, Hk, page, _ = k_cache.shape
    G = H // Hk
    scale = D ** -0.5 if scale is None else scale
    out, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    for n in range(N):
        length = int(min(max(int(kv_lens[n]), 0), np.shape(table)[1] * page))
        last = np.arange(length - nq, length)
        for h in range(H):
            k = gather(k_cache, table, n, length, h // G, page, shared)
            v = gather(v_cache, table, n, length, h // G, page, shared)
            out[n, :, h], mag[n, :, h], lse[n, :, h] = attend(q[n, :, h], k, v, last, scale)
    return out, mag, lse


def front(x, H, Hk, D, q_weight=None, k_weight=None, eps=1e-6, rope=None, interleaved=False,
          cu=None, kv_lens=None, table=None, k_cache=None, v_cache=None):
    """x [T, (H + 2 Hk) D] -> (q, k, v, k_cache, v_cache, rows inside a sequence); the caches
    are copies with k and v appended."""
    x = np.asarray(x, np.float64).reshape(-1, H + 2 * Hk, D)
    T = x.shape[0]
    cu = np.asarray([0, T] if cu is None else cu, np.int64)
    kc = None if k_cache is None else np.array(k_cache, np.float64)
    vc = None if v_cache is None else np.array(v_cache, np.float64)
    out = np.zeros_like(x)
    inside = np.zeros(T, bool)

    def turned(y, w, row):
        if w is not None:
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
        if rope is not None:
            half = rope.shape[1] // 2
            c, s = row[:half], row[half:]
            a = np.arange(half) * (2 if interleaved else 1)
            b = a + (1 if interleaved else half)
            z = (y[:, a] + 1j * y[:, b]) * (c + 1j * s)
            y = y.copy()
            y[:, a], y[:, b] = z.real, z.imag
        return y

    for n in range(len(cu) - 1):
        for t in range(cu[n], cu[n + 1]):
            inside[t] = True
            pos = int(t - cu[n] if kv_lens is None else kv_lens[n] - (cu[n + 1] - t))
            row = None if rope is None else np.asarray(rope, np.float64)[
                min(max(pos, 0), rope.shape[0] - 1)]
            out[t, :H] = turned(x[t, :H], q_weight, row)
            out[t, H:H + Hk] = turned(x[t, H:H + Hk], k_weight, row)
            out[t, H + Hk:] = x[t, H + Hk:]
            if kc is not None and 0 <= pos < np.shape(table)[1] * kc.shape[2]:
                p = int(table[n, pos // kc.shape[2]])
                if 0 <= p < kc.shape[0]:
                    kc[p, :, pos % kc.shape[2]] = out[t, H:H + Hk]
                    vc[p, :, pos % kc.shape[2]] = out[t, H + Hk:]
    return out[:, :H], out[:, H:H + Hk], out[:, H + Hk:], kc, vc, inside
