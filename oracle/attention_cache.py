"""fp64 oracle of the long-conversation operators (NumPy, from the definitions): e4m3 caches with
a scale for each 16 tokens, the softmax weight that keys gather, eviction by it, and rotary
positions of several axes.
"""
from __future__ import annotations

import numpy as np

from . import attention as A

BLOCK = 16


def e4m3_values():
    """The value of each byte: sign, 4 bits of exponent (bias 7), 3 of fraction; 0x7F is NaN."""
    v = np.empty(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        x = np.nan if b & 127 == 127 else m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[b] = -x if b & 128 else x
    return v


VALUES = e4m3_values()


def to_e4m3(x):
    """Bytes of the nearest values (ties to the even byte); what is not finite becomes NaN. Finite
    x must lie within 448."""
    x = np.asarray(x, np.float64)
    assert (np.abs(x[np.isfinite(x)]) <= 448).all()
    pos = VALUES[:127]
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isfinite(x), code | np.where(np.signbit(x), 128, 0), 127)
    return code.astype(np.uint8)


def same_bytes(a, b):
    """Equal as values: zeros of either sign, and any NaN."""
    x, y = VALUES[np.asarray(a)], VALUES[np.asarray(b)]
    return (x == y) | (np.isnan(x) & np.isnan(y))


def held(cache, scale):
    """Values of a cache of bytes [pages, Hk, page, D] with scales [pages, Hk, page / 16]."""
    return VALUES[cache] * np.repeat(np.asarray(scale, np.float64), BLOCK, 2)[..., None]


def least_scale(top):
    s = 2.0 ** -100
    while top > 448 * s:
        s *= 2
    return s


def append8(x, cache, scale, table, kv_lens=None, cu=None):
    """x [T, Hk, D] into copies of cache (bytes) and scale; returns them."""
    x = np.asarray(x, np.float64)
    T, Hk, _ = x.shape
    cache, scale = cache.copy(), np.array(scale, np.float32)
    pages, _, page, _ = cache.shape
    cu = [0, T] if cu is None else [int(c) for c in cu]
    for n in range(len(cu) - 1):
        b, e = cu[n], cu[n + 1]
        end = e - b if kv_lens is None else int(kv_lens[n])
        first = end - (e - b)
        at = first
        while at < end:
            stop = min(at // BLOCK * BLOCK + BLOCK, end)
            rows = x[b + at - first:b + stop - first]
            p = int(table[n, at // page]) if 0 <= at < np.shape(table)[1] * page else -1
            if 0 <= p < pages:
                r = at % page
                had = at % BLOCK if at == first else 0
                for h in range(Hk):
                    fin = np.abs(rows[:, h][np.isfinite(rows[:, h])])
                    s = least_scale(fin.max(initial=0.0))
                    old = float(scale[p, h, r // BLOCK])
                    if had and old > s:
                        s = old
                    scale[p, h, r // BLOCK] = s
                    if had and s != old:
                        cache[p, h, r - had:r] = to_e4m3(VALUES[cache[p, h, r - had:r]] * (old / s))
                    cache[p, h, r:r + stop - at] = to_e4m3(rows[:, h] / s)
            at = stop
    return cache, scale


def row_weights(q, k, last, scale, lse=None):
    """Softmax weights [r, n] of rows q [r, D] over keys k [n, D], row i seeing keys 0 .. last[i]."""
    w = np.zeros((q.shape[0], k.shape[0]))
    for i in range(q.shape[0]):
        m = min(int(last[i]) + 1, k.shape[0])
        if m <= 0:
            continue
        s = scale * (k[:m] @ q[i])
        l = s.max() + np.log(np.exp(s - s.max()).sum()) if lse is None else lse[i]
        w[i, :m] = np.exp(s - l)
    return w


def decode_weights(q, k_cache, table, kv_lens, weights, scale=None):
    """q [N, n_q, H, D], k_cache values -> a copy of weights [pages, Hk, page] with the step's
    weights added (the last n_q tokens': set)."""
    q, k_cache = np.asarray(q, np.float64), np.asarray(k_cache, np.float64)
    w = np.array(weights, np.float64)
    N, nq, H, D = q.shape
    pages, Hk, page, _ = k_cache.shape
    G, scale = H // Hk, D ** -0.5 if scale is None else scale
    for n in range(N):
        length = int(min(max(int(kv_lens[n]), 0), np.shape(table)[1] * page))
        last = np.repeat(np.arange(length - nq, length), G)
        for h in range(Hk):
            k = A.gather(k_cache, table, n, length, h, page, 0)
            gain = row_weights(q[n, :, h * G:(h + 1) * G].reshape(nq * G, D), k, last, scale).sum(0)
            for j in range(length):
                p = int(table[n, j // page])
                if 0 <= p < pages:
                    w[p, h, j % page] = gain[j] + (0.0 if j >= length - nq else w[p, h, j % page])
    return w


def prefill_weights(q, k, lse, weights, table, cu=None, window=0, scale=None):
    """A copy of weights with those of the prompts' keys set."""
    q, k, lse = (np.asarray(x, np.float64) for x in (q, k, lse))
    w = np.array(weights, np.float64)
    T, H, D = q.shape
    pages, Hk, page = w.shape
    G, scale = H // Hk, D ** -0.5 if scale is None else scale
    cu = A.sane_bounds([0, T] if cu is None else cu, T)
    for n, (b, e) in enumerate(zip(cu[:-1], cu[1:])):
        i = np.arange(max(b, e - window) if window else b, e)
        for h in range(Hk):
            gain = np.zeros(e - b)
            for g in range(h * G, h * G + G):
                gain += row_weights(q[i, g], k[b:e, h], i - b, scale, lse[i, g]).sum(0)
            for j in range(e - b):
                p = int(table[n, j // page]) if j < np.shape(table)[1] * page else -1
                if 0 <= p < pages:
                    w[p, h, j % page] = gain[j]
    return w


def choose(weights, keep, recent):
    """Of a sequence's weights [len]: the places that stay, in order."""
    n = len(weights)
    if n <= keep:
        return list(range(n))
    rank = sorted(range(n - recent), key=lambda j: (not np.isnan(weights[j]),
                                                    0.0 if np.isnan(weights[j]) else -weights[j], j))
    return sorted(rank[:keep - recent]) + list(range(n - recent, n))


def evict(k_cache, v_cache, weights, table, kv_lens, new_table, keep, recent, k_scale=None, v_scale=None):
    """Copies of everything after the cut (caches as given: bytes with scales, or values), then the
    new lengths and the places kept."""
    src = [k_cache, v_cache, weights] + ([k_scale, v_scale] if k_scale is not None else [])
    dst = [np.array(x) for x in src]
    pages, Hk, page, _ = k_cache.shape
    N = len(kv_lens)
    lens, kept = np.zeros(N, np.int32), np.full((N, Hk, keep), -1, np.int32)
    for n in range(N):
        length = int(min(max(int(kv_lens[n]), 0), np.shape(table)[1] * page))
        lens[n] = min(length, keep)
        for h in range(Hk):
            def place(t, j):
                p = int(t[n, j // page])
                return (p, h, j % page) if 0 <= p < pages else None

            def weight(j):
                a = place(table, j)
                return 0.0 if a is None else float(weights[a])
            got = choose(np.array([weight(j) for j in range(length)]), keep, recent)
            kept[n, h, :len(got)] = got
            for i0 in range(0, len(got), BLOCK):
                block = got[i0:i0 + BLOCK]
                to = place(new_table, i0)
                if to is None:
                    continue
                at = [place(table, j) for j in block]
                for x in range(3):
                    for i, a in enumerate(at):
                        row = src[x][a] if a is not None else np.zeros_like(src[x][to])
                        if x < 2 and k_scale is not None:
                            scales = [float(src[3 + x][b[0], h, b[2] // BLOCK]) if b else 0.0 for b in at]
                            most = max(scales)
                            dst[3 + x][to[0], h, to[2] // BLOCK] = most
                            if scales[i] != most:
                                row = to_e4m3(VALUES[row] * (scales[i] / most))
                        dst[x][to[0], h, to[2] + i] = row
    return dst, lens, kept


def front_axes(x, H, Hk, D, q_weight, k_weight, eps, rope, interleaved, positions, axes):
    """q, k [T, heads, D] of the front end with positions [n_axes, T] and axes [rot / 2]."""
    x = np.asarray(x, np.float64).reshape(-1, H + 2 * Hk, D)[:, :H + Hk].copy()
    rope = np.asarray(rope, np.float64)
    half = rope.shape[1] // 2
    for w, part in ((q_weight, slice(0, H)), (k_weight, slice(H, H + Hk))):
        if w is not None:
            y = x[:, part]
            x[:, part] = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    for i in range(half):
        axis = 0 if axes is None else min(int(axes[i]), len(positions) - 1)
        row = np.clip(np.asarray(positions[axis], np.int64), 0, rope.shape[0] - 1)
        turn = (rope[row, i] + 1j * rope[row, half + i])[:, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        z = (x[..., a] + 1j * x[..., b]) * turn
        x[..., a], x[..., b] = z.real, z.imag
    return x[:, :H], x[:, H:]
