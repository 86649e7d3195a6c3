"""Float64 CPU oracle of the operators of serving in 8 bits.

TEST INFRASTRUCTURE. Only the test suite may import this module; it imports nothing from the product.

Each function follows the operator's definition directly. Codes come with the exact quotients they were
rounded from, so that a test can tell a border from a mistake.
"""

from __future__ import annotations

import numpy as np


def norm_quant(h, weight, eps):
    """h [n, d]: the sum as it is stored. Returns (codes, scales, y, quotients)."""
    h = np.asarray(h, dtype=np.float64)
    p = h if weight is None else h * np.asarray(weight, dtype=np.float64)
    n, d = h.shape
    codes, scales, y, quot = np.zeros((n, d)), np.zeros(n), np.zeros((n, d)), np.zeros((n, d))
    with np.errstate(all="ignore"):
        for i in range(n):
            ms = np.sum(h[i] * h[i]) / d + eps
            rho = 0.0 if ms == 0 else 1.0 / np.sqrt(ms)
            y[i] = p[i] * rho
            if not (np.all(np.isfinite(h[i])) and np.all(np.isfinite(p[i]))):
                scales[i] = np.nan
                continue
            top = np.max(np.abs(p[i]))
            scales[i] = top * rho / 127.0
            if top > 0:
                quot[i] = p[i] * 127.0 / top
                codes[i] = np.rint(quot[i])
    return codes, scales, y, quot


def byte_gemm(x, x_scales, w, w_scales, zeros):
    """(exact whole sums as int64, the product in float64)."""
    x = np.asarray(x, dtype=np.int64)
    w = np.asarray(w, dtype=np.int64)
    if zeros is not None:
        w = w - np.asarray(zeros, dtype=np.int64)[:, None]
    whole = x @ w.T
    out = whole.astype(np.float64)
    if x_scales is not None:
        out = out * np.asarray(x_scales, dtype=np.float64)[:, None]
    if w_scales is not None:
        out = out * np.asarray(w_scales, dtype=np.float64)
    return whole, out


def rotate(x, positions, inv_freq, pair_axis=None, interleaved=False):
    """x [n, heads, dh], positions [axes, n]."""
    out = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ax = 0 if pair_axis is None else min(max(int(pair_axis[i]), 0), positions.shape[0] - 1)
        t = positions[ax].astype(np.float64) * float(inv_freq[i])
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        u, v = out[..., a].copy(), out[..., b].copy()
        out[..., a], out[..., b] = u * c - v * s, v * c + u * s
    return out


def kv_append(x, cache, scales, table, start, past):
    """Appends x [n, heads, dh] (rotated already) token by page to float64 copies of cache [pages, page_size, heads,
    dh] and float32 scales [pages, heads]. Returns (cache, scales, quotients): quotients [pages, page_size, heads, dh]
    are the exact ones of codes that were rounded, NaN elsewhere."""
    x = np.asarray(x, dtype=np.float64)
    cache = np.array(cache, dtype=np.float64)
    scales = np.array(scales, dtype=np.float32)
    quot = np.full(cache.shape, np.nan)
    pages, ps, heads, _ = cache.shape
    n = x.shape[0]
    for s in range(len(past)):
        r0 = min(max(int(start[s]), 0), n)
        r1 = min(max(int(start[s + 1]), r0), n)
        t0 = min(max(int(past[s]), 0), table.shape[1] * ps)
        t1 = min(t0 + r1 - r0, table.shape[1] * ps)
        t = t0
        while t < t1:
            b, slot = t // ps, t % ps
            m = min(t1 - t, ps - slot)
            page = int(table[s, b])
            if 0 <= page < pages:
                rows = x[r0 + t - t0:r0 + t - t0 + m]
                for h in range(heads):
                    v = rows[:, h]
                    new = np.float32(np.max(np.abs(v)) / 127.0) if np.all(np.isfinite(v)) else np.float32(np.nan)
                    if slot > 0:
                        old = scales[page, h]
                        new = np.float32(np.nan) if np.isnan(new) or np.isnan(old) else max(new, old)
                        if new > old:
                            q = cache[page, :slot, h] * (np.float64(old)) / np.float64(new)
                            quot[page, :slot, h] = q
                            cache[page, :slot, h] = np.rint(q)
                    scales[page, h] = new
                    if new > 0 and np.isfinite(new):
                        q = v / np.float64(new)
                        quot[page, slot:slot + m, h] = q
                        cache[page, slot:slot + m, h] = np.clip(np.rint(q), -127, 127)
                    else:
                        cache[page, slot:slot + m, h] = 0
            t += m
    return cache, scales, quot


def kv_attention(q, k_cache, v_cache, k_scales, v_scales, table, q_start, lens, scale, causal=True, window=0,
                 softcap=0.0, slopes=None):
    """q [nq, hq, dh]. Returns (out, mag, spread, written): mag = sum p |v|, spread = the largest of scale * sum |q k|
    and |score| over the keys a query sees, written: the rows that belong to a sequence."""
    q = np.asarray(q, dtype=np.float64)
    nq, hq, dh = q.shape
    pages, ps, hk, _ = k_cache.shape
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    spread, written = np.zeros((nq, hq, 1)), np.zeros(nq, dtype=bool)
    for s in range(len(lens)):
        q0 = min(max(int(q_start[s]), 0), nq)
        q1 = min(max(int(q_start[s + 1]), q0), nq)
        n = min(max(int(lens[s]), 0), table.shape[1] * ps)
        written[q0:q1] = True
        if n == 0:
            continue
        ids = np.repeat(table[s, :-(-n // ps)].astype(np.int64), ps)[:n]
        slot = np.arange(n) % ps
        held = (ids >= 0) & (ids < pages)
        at = np.where(held, ids, 0)
        for g in range(hk):
            k = k_cache[at, slot, g].astype(np.float64) * np.where(held, k_scales[at, g], 0.0)[:, None]
            v = v_cache[at, slot, g].astype(np.float64) * np.where(held, v_scales[at, g], 0.0)[:, None]
            for i in range(q1 - q0):
                p = i + n - (q1 - q0)
                j = np.arange(n)
                seen = held.copy()
                if causal:
                    seen &= j <= p
                if window:
                    seen &= p - j < window
                if not seen.any():
                    continue
                for h in range(g * (hq // hk), (g + 1) * (hq // hk)):
                    z = k[seen] @ q[q0 + i, h] * scale
                    big = np.abs(k[seen]) @ np.abs(q[q0 + i, h]) * abs(scale)
                    if softcap:
                        z = softcap * np.tanh(z / softcap)
                    if slopes is not None:
                        z = z - float(slopes[h]) * np.abs(p - j[seen])
                    spread[q0 + i, h] = max(np.max(big), np.max(np.abs(z)))
                    e = np.exp(z - np.max(z))
                    e /= np.sum(e)
                    out[q0 + i, h] = e @ v[seen]
                    mag[q0 + i, h] = e @ np.abs(v[seen])
    return out, mag, spread, written
