"""Serving in 8 bits where its roundings decide: sums bit for bit, values rounded once, scales and queries of very
different sizes.

Tolerances count roundings, h half a step of the output's type and u = 2^-24. For kv_attention:
* the output's own rounding, h |out| (and 2^-25 for subnormal fp16);
* a probability times its value's scale is kept to 2^-22 of itself or 2^-30 of the largest such product of the query's
  keys: 2^-22 sum p |v| + n 2^-30 * 127 max p vs for n keys; that largest product is at most the sum of all of them,
  which is the output where every code is 127;
* a score's fp32 error is at most (head_dim + 8) u times the sum of |q k| scale (or the score itself) and a query's
  rounding to 22 bits adds 4 u more, which moves numerator and denominator each; sums over keys add at most 64 u.
Nothing is added for scales of pages that a query does not see.
"""

import numpy as np
import pytest

from gpu_util import torch_cuda
from oracle import serve_ref
from test_serving_gpu import DT, U, _dtype, _g, _half_step, _ints, _np, _pool, _rand, _starts, _table

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------ kv_attention

def _attend(dtype, q, kc, vc, ks, vs, table, news, lens, split=True, **kw):
    """Runs the call, and checks every row within the bound above."""
    torch = torch_cuda()
    g = _g()
    start = _starts(news)
    dh, pages = q.shape[2], kc.shape[0]
    scale = dh ** -0.5
    work = None if split else torch.empty(0, dtype=torch.uint8, device="cuda:0")
    out = g.gptq_kv_attention(q, kc, vc, ks, vs, _ints(table), _ints(lens), q_start=_ints(start), work=work,
                              causal=kw.get("causal", True), window=kw.get("window", 0), softcap=kw.get("cap", 0.0),
                              slopes=kw.get("slopes"))
    torch.cuda.synchronize()
    slopes = kw.get("slopes")
    args = (np.asarray(table), start, lens, scale, kw.get("causal", True), kw.get("window", 0), kw.get("cap", 0.0),
            None if slopes is None else _np(slopes))
    k8, v8, ksn, vsn = (t.cpu().numpy() for t in (kc, vc, ks, vs))
    want, mag, spread, written = serve_ref.kv_attention(_np(q), k8, v8, ksn, vsn, *args)
    most = serve_ref.kv_attention(_np(q), k8, np.full_like(v8, 127), ksn, np.abs(vsn), *args)[0]
    assert written.all()
    bound = _half_step(dtype) * np.abs(want) + (2.0 ** -22 + (2 * (dh + 12) * spread + 64) * U) * mag \
        + max(lens) * 2.0 ** -30 * most + 2.0 ** -25 * (dtype == "f16")
    got = _np(out)
    held = np.abs(want) < 65000.0 if dtype == "f16" else np.ones(want.shape, dtype=bool)
    err = np.abs(got - want)
    worst = float(np.max(np.where(held, err / np.maximum(bound, 1e-300), 0.0)))
    assert np.all(err[held] <= bound[held]), worst
    return out, want


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("news,lens", [([1, 1], [1000, 130]), ([70], [200]), ([5, 3], [64, 900])], ids=str)
def test_probabilities_keep_fp32s_accuracy(news, lens, dtype):
    """Values that nearly cancel: every second one is the negative of the one before, and all probabilities are much
    alike, so that their roundings are what an output's error is made of."""
    hq, hk, dh, ps = 4, 2, 128, 16
    most = max(-(-n // ps) for n in lens)
    pages = len(lens) * most
    kc, ks = _pool(pages, ps, hk, dh, 13)
    vc, vs = _pool(pages, ps, hk, dh, 14)
    vc[:, 1::2] = -vc[:, 0::2]
    table = _table(len(lens), most, pages, 15)
    q = _rand((sum(news), hq, dh), 16, dtype, 0.02)
    for kw in ({}, dict(causal=False), dict(cap=20.0)):
        _attend(dtype, q, kc, vc, ks, vs, table, news, lens, **kw)
