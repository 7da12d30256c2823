"""Plain fp64 definitions of the serving operators (numpy, one sequence at a
time): rotary positions, the paged-cache append and attention over the cache.
Test infrastructure only."""
from __future__ import annotations

import numpy as np


def rotate(x, pos, rot, axis, inv_freq, interleaved=False, inverse=False):
    """x [n, H, d] float64, pos [naxes, n]; axis and inv_freq per frequency.
    Returns (turned x, |a| + |b| of each element's pair: what an angle's error
    is multiplied by; 0 where nothing turns)."""
    x = np.asarray(x, np.float64)
    y, mag = x.copy(), np.zeros_like(x)
    F = rot // 2
    for f in range(F):
        i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + F)
        phi = np.asarray(pos[axis[f]], np.float64)[:, None] * inv_freq[f]
        if inverse:
            phi = -phi
        a, b = x[:, :, i], x[:, :, j]
        y[:, :, i] = a * np.cos(phi) - b * np.sin(phi)
        y[:, :, j] = a * np.sin(phi) + b * np.cos(phi)
        mag[:, :, i] = mag[:, :, j] = np.abs(a) + np.abs(b)
    return y, mag


def keys_of(cache, pages, n):
    """The first n rows of a page list: [n, Hkv, d] float64."""
    page = cache.shape[2]
    rows = [cache[pages[i // page], :, i % page] for i in range(n)]
    return np.asarray(rows, np.float64).reshape(n, cache.shape[1], cache.shape[3])


def attend(q, k_cache, v_cache, table, q_start, kv_len, prefix_pages, P):
    """q [Tq, Hq, d].  Returns per row O [Tq, Hq, d], lse [Tq, Hq], and what
    error bounds need: A = softmax-weighted mean of |v|, S = max over the keys
    seen of sum_d |q_d k_d| / sqrt(d), n = keys seen."""
    Tq, Hq, d = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    O, A = np.zeros((Tq, Hq, d)), np.zeros((Tq, Hq, d))
    lse, S, n = np.full((Tq, Hq), -np.inf), np.zeros((Tq, Hq)), np.zeros(Tq, int)
    pk, pv = keys_of(k_cache, prefix_pages, P), keys_of(v_cache, prefix_pages, P)
    for s in range(len(kv_len)):
        t0, t1, L = int(q_start[s]), int(q_start[s + 1]), int(kv_len[s])
        if t0 == t1:
            continue
        k = np.concatenate([pk, keys_of(k_cache, table[s], L)])
        v = np.concatenate([pv, keys_of(v_cache, table[s], L)])
        for t in range(t0, t1):
            seen = P + L - (t1 - t0) + (t - t0) + 1
            n[t] = seen
            for h in range(Hq):
                kk, vv = k[:seen, h // G], v[:seen, h // G]
                x = kk @ q[t, h] / np.sqrt(d)
                m = x.max()
                p = np.exp(x - m)
                z = p.sum()
                O[t, h], A[t, h] = p @ vv / z, p @ np.abs(vv) / z
                lse[t, h] = m + np.log(z)
                S[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() / np.sqrt(d)
    return O, lse, A, S, n
