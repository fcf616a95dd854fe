"""Attention from its definition in 64 bits, with a window in front of which the first keys stay visible, for the tests of
long caches."""
import math

import numpy as np


def attend64(q, q_lens, kv_lens, cu, rows, *, window=None, first=0, cap=None, causal=True, sinks=None, scale=None, Dv=None,
             step=None):
    """q [T, Hq, D] float64; rows(s) the K and V [keys, Hkv, D] of sequence s.  Returns o [T, Hq, Dv] and for each element the
    sum of |p v|, which the rounding of the probabilities is relative to; step(s) [keys, Hkv, D]: and the sum of p step."""
    T, Hq, D = q.shape
    Dv = Dv or D
    scale = scale or 1 / math.sqrt(D)
    o, size, steps = np.zeros((T, Hq, Dv)), np.zeros((T, Hq, Dv)), np.zeros((T, Hq, Dv))
    for s, (a, n) in enumerate(zip(q_lens, kv_lens)):
        if not a:
            continue
        K, V = rows(s)
        G = Hq // K.shape[1]
        t = slice(cu[s], cu[s] + a)
        pos = np.arange(n - a, n)[:, None]
        j = np.arange(n)[None]
        sees = (j <= pos) if causal else np.ones((a, n), bool)
        if window is not None:
            sees = sees & ((j > pos - window) | (j < first))
        for h in range(Hq):
            x = scale * q[t, h] @ K[:, h // G].T
            if cap:
                x = cap * np.tanh(x / cap)
            x = np.where(sees, x, -np.inf)
            m = x.max(1, keepdims=True)
            if sinks is not None:
                m = np.maximum(m, sinks[h])
            with np.errstate(invalid="ignore"):
                p = np.where(sees, np.exp(x - np.where(np.isfinite(m), m, 0)), 0.0)
            l = p.sum(1, keepdims=True)
            if sinks is not None:
                l = l + np.exp(sinks[h] - m)
            p = np.where(sees.any(1, keepdims=True), p / np.where(l > 0, l, 1), 0.0)
            o[t, h] = p @ V[:, h // G]
            size[t, h] = p @ np.abs(V[:, h // G])
            if step:
                steps[t, h] = p @ step(s)[:, h // G]
    return (o, size, steps) if step else (o, size)


def cached_rows(batch, cache, scale=1.0, latent=False):
    """rows(s) of a cache of 8- or 16-bit rows (float64 [N, ps, rows, D])."""
    def rows(s):
        page, at = batch.slots(s, np.arange(batch.kv_lens_list[s]))
        x = cache[page, at] * scale
        return (x, x[..., :512]) if latent else (x[:, 0::2], x[:, 1::2])

    return rows
