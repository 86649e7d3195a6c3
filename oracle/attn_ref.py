"""Float64 CPU oracle of the attention-side operators and the adapters beside stored layers.

TEST INFRASTRUCTURE. Only the test suite may import this module; it imports nothing from the product.

Each function follows the operator's definition directly (loops over sequences and heads, complex
rotations) and also returns, where a tolerance needs them, the sums of magnitudes that rounding errors
scale with.
"""

from __future__ import annotations

import numpy as np


def norm_rotate(x, weight=None, positions=None, inv_freq=None, pair_axis=None, norm=True, eps=1e-6,
                interleaved=False):
    """x [n, heads, dh]; positions [axes, n]. Returns (out, mag): mag = |y_a| + |y_b| for rotated pairs, |y|
    for the other columns (y the normed head)."""
    x = np.asarray(x, dtype=np.float64)
    n, _, dh = x.shape
    y = x.copy()
    if norm:
        y = y / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
        if weight is not None:
            y = y * np.asarray(weight, dtype=np.float64)
    out, mag = y.copy(), np.abs(y)
    if inv_freq is not None:
        half = len(inv_freq)
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            ax = 0 if pair_axis is None else min(max(int(pair_axis[i]), 0), positions.shape[0] - 1)
            t = positions[ax].astype(np.float64) * float(inv_freq[i])
            z = (y[..., a] + 1j * y[..., b]) * np.exp(1j * t)[:, None]
            out[..., a], out[..., b] = z.real, z.imag
            mag[..., a] = mag[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, mag


def attention(q, k, v, seqs, scale, causal=True, softcap=0.0, slopes=None, q_doc=None, kv_doc=None, prefix=None):
    """q [nq, hq, dh], k and v [nk, hk, dh]; seqs: (q0, q1, k0, k1) per sequence. Returns (out, mag, spread):
    mag = sum p |v| and spread = the largest of scale * sum |q k| and |score| over the keys a query sees."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    nq, hq, dh = q.shape
    hk = k.shape[1]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    spread = np.zeros((nq, hq, 1))
    for s, (q0, q1, k0, k1) in enumerate(seqs):
        lq, lk = q1 - q0, k1 - k0
        for i in range(lq):
            p = i + lk - lq
            j = np.arange(lk)
            seen = np.ones(lk, dtype=bool) if not causal else (j <= p)
            if causal and prefix is not None:
                seen |= j < prefix[s]
            if q_doc is not None:
                seen &= (kv_doc[k0:k1] == q_doc[q0 + i]) & (q_doc[q0 + i] >= 0)
            j = j[seen]
            if j.size == 0:
                continue
            for h in range(hq):
                kk, vv = k[k0 + j, h * hk // hq], v[k0 + j, h * hk // hq]
                sc = scale * (kk @ q[q0 + i, h])
                if softcap:
                    sc = softcap * np.tanh(sc / softcap)
                if slopes is not None:
                    sc = sc - float(slopes[h]) * np.abs(p - j)
                w = np.exp(sc - sc.max())
                w /= w.sum()
                out[q0 + i, h] = w @ vv
                mag[q0 + i, h] = w @ np.abs(vv)
                spread[q0 + i, h] = max(abs(scale) * np.max(np.abs(kk) @ np.abs(q[q0 + i, h])), np.max(np.abs(sc)))
    return out, mag, spread


def lora(x, A, B, index, scales=None, ranks=None, base=None):
    """Returns (y, mag): mag = |base| + |s| (|x| |A|^T) |B|^T."""
    x, A, B = (np.asarray(t, dtype=np.float64) for t in (x, A, B))
    na, r, _ = A.shape
    y = np.zeros((x.shape[0], B.shape[1])) if base is None else np.asarray(base, dtype=np.float64).copy()
    mag = np.abs(y)
    for i, a in enumerate(index):
        if 0 <= a < na:
            ra = r if ranks is None else min(max(int(ranks[a]), 0), r)
            s = 1.0 if scales is None else float(scales[a])
            y[i] += s * (B[a][:, :ra] @ (A[a][:ra] @ x[i]))
            mag[i] += abs(s) * (np.abs(B[a][:, :ra]) @ (np.abs(A[a][:ra]) @ np.abs(x[i])))
    return y, mag


def block_forward(X, W, hidden, heads, kv_heads, seqs, seq_len, eps=1e-6, qk_norm=False, q_norm=None, k_norm=None,
                  norm_eps=1e-6, inv_freq=None, positions=None, pair_axis=None, interleaved=False, scale=None,
                  softcap=0.0, slopes=None, doc=None, prefix=None, causal=True):
    """The decoder block of gptq_quantize_block_attn: RMSNorm, q/k/v, per-head norm and rotation, attention, o,
    residual, RMSNorm, gated MLP, residual. Returns the four stage inputs and the output."""
    X = np.asarray(X, dtype=np.float64)
    n, dh = seqs * seq_len, hidden // heads

    def rms(x):
        return x / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps)

    xa = rms(X)
    q = (xa @ W[0].T).reshape(n, heads, dh)
    k, v = ((xa @ W[i].T).reshape(n, kv_heads, dh) for i in (1, 2))
    pos = None if positions is None else np.atleast_2d(positions)
    if qk_norm or inv_freq is not None:
        q, _ = norm_rotate(q, q_norm, pos, inv_freq, pair_axis, qk_norm, norm_eps, interleaved)
        k, _ = norm_rotate(k, k_norm, pos, inv_freq, pair_axis, qk_norm, norm_eps, interleaved)
    ranges = [(s * seq_len, (s + 1) * seq_len) * 2 for s in range(seqs)]
    o, _, _ = attention(q, k, v, ranges, dh ** -0.5 if scale is None else scale, causal, softcap, slopes, doc, doc,
                        prefix)
    o = o.reshape(n, hidden)
    h1 = X + o @ W[3].T
    xm = rms(h1)
    g = xm @ W[4].T
    down = g / (1.0 + np.exp(-g)) * (xm @ W[5].T)
    return dict(inputs=[xa, o, xm, down], out=h1 + down @ W[6].T)
