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
from test_serving_gpu import (DT, U, _check_gemm, _dtype, _g, _gemm_inputs, _half_step, _ints, _np, _pool, _rand, _starts,
                              _table)

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
@pytest.mark.parametrize("ratio", [1e3, 1e6, 1e9, 1e12, 1e25], ids=str)
@pytest.mark.parametrize("where", ["later", "before", "half"])
def test_value_scales_of_unseen_pages_take_no_part(where, ratio, dtype):
    """A page whose values are far larger, which some rows see and others do not: after a row's position, before its window
    (and 128 keys before others that it sees), in the other half of 32 keys that it sees."""
    torch = torch_cuda()
    print(f"unseen scales {(where, ratio, dtype)}", flush=True)
    hq, hk, dh, ps = 2, 2, 64, 16
    news, lens, kw, page = {"later": ([32], [32], {}, 1), "before": ([100], [500], dict(window=200), 13),
                            "half": ([64], [64], {}, 3)}[where]
    pages = -(-lens[0] // ps)
    kc, ks = _pool(pages, ps, hk, dh, 1)
    vc, vs = _pool(pages, ps, hk, dh, 2)
    table = _table(1, pages, pages, 3)
    vs[int(table[0, page])] *= ratio
    q = _rand((news[0], hq, dh), 4, dtype)
    for split in (True, False):
        _attend(dtype, q, kc, vc, ks, vs, table, news, lens, split=split, **kw)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("split", [True, False])
def test_values_far_apart_weigh_by_their_products(split, dh, dtype):
    """Early pages with values 2^40 times the others', whose probabilities are smaller by as much or by far more."""
    torch = torch_cuda()
    print(f"far values {(split, dh, dtype)}", flush=True)
    hq, hk, ps, n = 4, 2, 32, 1700
    pages = -(-n // ps)
    kc, ks = _pool(pages, ps, hk, dh, 5)
    vc, vs = _pool(pages, ps, hk, dh, 6)
    table = _table(1, pages, pages, 7)
    order = [int(p) for p in table[0]]
    slopes = torch.tensor([1.0, 0.5, 0.02, 0.0], device="cuda:0")
    q = _rand((3, hq, dh), 8, dtype, 0.5)
    for early in (pages - 2, pages - 3, pages // 2, 1):
        v2 = vs.clone()
        v2[order[:early]] *= 2.0 ** 40 if dtype != "f16" else 2.0 ** 20
        _attend(dtype, q, kc, vc, ks, v2, table, [3], [n], split=split, slopes=slopes)


@pytest.mark.parametrize("dtype", DT)
def test_value_scales_of_zero_and_of_either_sign(dtype):
    hq, hk, dh, ps = 4, 2, 64, 16
    kc, ks = _pool(13, ps, hk, dh, 9)
    vc, vs = _pool(13, ps, hk, dh, 10)
    table = _table(1, 13, 13, 11)
    for i, p in enumerate(int(p) for p in table[0]):
        vs[p] *= [1.0, 0.0, -1.0, 1e-30, -1e4][i % 5]
    q = _rand((50, hq, dh), 12, dtype)
    _attend(dtype, q, kc, vc, ks, vs, table, [50], [200])
    vs.zero_()
    out, _ = _attend(dtype, q, kc, vc, ks, vs, table, [50], [200])
    assert (out == 0).all()


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


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("news", [1, 40])
def test_queries_with_a_channel_far_larger(news, dtype):
    """A channel of a query that is far larger than the others, where the keys hold zeros: fp32's others keep their 22
    bits down to 2^-18 of it, bf16's are exact down to 2^-31, fp16's always."""
    torch = torch_cuda()
    print(f"large channel {(news, dtype)}", flush=True)
    hq, hk, dh, ps, n = 4, 2, 64, 16, 300
    pages = -(-n // ps)
    kc, ks = _pool(pages, ps, hk, dh, 17)
    vc, vs = _pool(pages, ps, hk, dh, 18)
    kc[..., 5] = 0
    r = np.random.default_rng(19)
    q = r.uniform(0.5, 1.0, (news, hq, dh)) * r.choice([-1.0, 1.0], (news, hq, dh))
    q[..., 5] = {"f32": 2.0 ** 16, "f16": 2.0 ** 15, "bf16": 2.0 ** 29}[dtype]
    q = torch.from_numpy(q).to(_dtype(dtype)).cuda()
    for kw in ({}, dict(cap=8.0)):
        _attend(dtype, q, kc, vc, ks, vs, _table(1, pages, pages, 20), [news], [n], **kw)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("power", [18, 22, 23, 24, 25, 26, 27, 28, 30, 36, 40])
@pytest.mark.parametrize("any_score", [False, True])
def test_scores_so_large_that_fp32_counts_in_steps(any_score, power, dtype):
    """Scores of 2^18 to 2^40 and more, exact in fp32, of which a row's best is one key's or two keys': the output is
    that key's value, or the two's average, whatever the sizes of the values' scales."""
    torch = torch_cuda()
    print(f"large scores {(any_score, power, dtype)}", flush=True)
    hq, hk, dh, ps, n = 2, 1, 64, 16, 160
    pages = n // ps
    r = np.random.default_rng(60)
    kc = torch.zeros(pages, ps, hk, dh, dtype=torch.int8, device="cuda:0")
    order = r.permutation(n) % 100 + 20       # 20 .. 79 stand twice
    kc[..., 3] = torch.from_numpy(order.reshape(pages, ps, 1).astype(np.int8)).cuda()
    kc[9, 15, 0, 3] = 127
    kc[4, 2, 0, 3] = 126
    vc, _ = _pool(pages, ps, hk, dh, 61)
    top = 400.0 if dtype == "f16" else 3e7
    vs = torch.tensor([top, 1e-3, top, 1.0, top, 2.0, 1e-6, top, 0.0, top], device="cuda:0")[:, None].contiguous()
    ks = torch.full((pages, hk), 2.0 ** (power - 10), device="cuda:0")
    q = torch.zeros(3, hq, dh, device="cuda:0")
    q[:, 0, 3], q[:, 1, 3] = 64.0, -64.0                 # scores 2^(power - 7) times the code, or less
    slopes = torch.zeros(hq, device="cuda:0") if any_score else None
    table = np.arange(pages, dtype=np.int32)[None]
    for split in (True, False):
        work = None if split else torch.empty(0, dtype=torch.uint8, device="cuda:0")
        out = _g().gptq_kv_attention(q.to(_dtype(dtype)), kc, vc, ks, vs, _ints(table), _ints([n]), slopes=slopes, work=work)
        torch.cuda.synchronize()
        want, mag, _, _ = serve_ref.kv_attention(_np(q), kc.cpu().numpy(), vc.cpu().numpy(), ks.cpu().numpy(), vs.cpu().numpy(),
                                                 table, [0, 3], [n], 0.125, True, 0, 0.0, None)
        bound = _half_step(dtype) * np.abs(want) + (2.0 ** -22 + 64 * U) * mag + 2.0 ** -25 * (dtype == "f16")
        err = np.abs(_np(out) - want)
        assert np.all(err <= bound), float(np.max(err / np.maximum(bound, 1e-300)))


# -------------------------------------------------------------------------------------- norm_quant

SIZES = [(1, 1), (3, 2), (5, 7), (2, 8), (9, 63), (4, 64), (7, 255), (3, 512), (6, 513), (5, 1000), (3, 1024), (2, 2049),
         (3, 4097), (2, 8200), (2, 11008), (1, 16389), (1, 40001), (1, 65535), (3000, 97), (2500, 1030)]


def _same_bits(got, want):
    torch = torch_cuda()
    kind = torch.int32 if got.dtype == torch.float32 else torch.int16
    return torch.equal(got.contiguous().view(kind), want.contiguous().view(kind))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,d", SIZES)
def test_sums_bit_for_bit(n, d, dtype):
    """The sum is x + residual rounded once, into a new array, a range of a wider one (what lies beside is left as it
    was), over either input; without a residual it is x."""
    torch = torch_cuda()
    print(f"sums {(n, d, dtype)}", flush=True)
    g = _g()
    x, r = _rand((n, d), 31, dtype, 3.0), _rand((n, d), 32, dtype)
    want = (x.float() + r.float()).to(x.dtype)
    _, _, total = g.gptq_norm_quant(x, r)
    torch.cuda.synchronize()
    assert _same_bits(total, want)
    base = torch.full((n + 2, d + 9), 7.0, dtype=x.dtype, device="cuda:0")
    g.gptq_norm_quant(x, r, sum_out=base[1:n + 1, 4:4 + d])
    alone = torch.full((n + 2, d + 9), 7.0, dtype=x.dtype, device="cuda:0")
    g.gptq_norm_quant(x, sum_out=alone[1:n + 1, 3:3 + d])
    torch.cuda.synchronize()
    for got, at, held in ((base, 4, want), (alone, 3, x)):
        assert _same_bits(got[1:n + 1, at:at + d], held)
        got[1:n + 1, at:at + d] = 7.0
        assert torch.all(got == 7.0)
    x2, r2 = x.clone(), r.clone()
    g.gptq_norm_quant(x2, r, sum_out=x2)
    g.gptq_norm_quant(x, r2, sum_out=r2)
    torch.cuda.synchronize()
    assert _same_bits(x2, want) and _same_bits(r2, want)


@pytest.mark.parametrize("dtype", DT)
def test_sums_that_are_not_finite(dtype):
    torch = torch_cuda()
    x, r = _rand((4, 600), 33, dtype), _rand((4, 600), 34, dtype)
    x[1, 599], r[2, 0], x[3, 8], r[3, 8] = float("inf"), float("nan"), float("inf"), -float("inf")
    want = (x.float() + r.float()).to(x.dtype)
    _, _, total = _g().gptq_norm_quant(x, r)
    torch.cuda.synchronize()
    gone = want.isnan()
    assert torch.equal(total.isnan(), gone) and torch.equal(total[~gone], want[~gone])


def _round_to(dtype, v):
    """float64 numbers to the nearest of the type, ties to even, in one step, as float64; and where they are within 2^-40
    of a tie: 64-bit sums of up to 4096 squares and a few roundings more do not decide those."""
    bits, low = {"f16": (11, -24), "bf16": (8, -133), "f32": (24, -149)}[dtype]
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - bits, low))
    q = v / step
    return np.rint(q) * step, np.abs(q - np.floor(q) - 0.5) < np.ldexp(1.0, bits - 40)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d,size", [(96, 1.0), (4096, 1.0), (1001, 1e-5)])
def test_normed_rows_are_rounded_once(d, size, dtype):
    """y is the rounding of the 64-bit result: many elements, since a second rounding shows in one of some ten thousand."""
    torch = torch_cuda()
    n = (1 << 21) // d
    x = _rand((n, d), 35, dtype)
    w = _rand((d,), 36, "f32", size)
    y = torch.empty_like(x)
    _g().gptq_norm_quant(x, None, w, eps=1e-5, y=y)
    torch.cuda.synchronize()
    h, wn = _np(x), _np(w)
    v = h * wn / np.sqrt((h * h).sum(1, keepdims=True) / d + 1e-5)
    want, unclear = _round_to(dtype, v)
    off = (_np(y) != want) & ~unclear
    assert not off.any(), int(off.sum())


# --------------------------------------------------------------------------------------- kv_append

@pytest.mark.parametrize("tokens", [3, 40])
@pytest.mark.parametrize("dh", [32, 6])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_keys_whose_rotation_passes_fp32s_largest(dtype, dh, tokens):
    """Finite keys near fp32's largest, rotated to up to sqrt(2) times it: their page's scale is the 127th of that, finite,
    and the codes stand on it. An infinity or NaN still makes the scale NaN."""
    torch = torch_cuda()
    print(f"large keys {(dtype, dh, tokens)}", flush=True)
    g = _g()
    pages = -(-tokens // 16)
    k = _rand((tokens, 2, dh), 40, dtype)
    k[1:3] = 3.3e38 * torch.sign(k[1:3])
    v = _rand((tokens, 2, dh), 41, dtype)
    f = torch.from_numpy((10000.0 ** (-np.arange(dh // 2) * 2 / dh)).astype(np.float32)).cuda()
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda:0")
    table = np.arange(pages, dtype=np.int32)[None]

    def run(keys):
        kc, vc = (torch.zeros(pages, 16, 2, dh, dtype=torch.int8, device="cuda:0") for _ in range(2))
        ks, vs = (torch.zeros(pages, 2, device="cuda:0") for _ in range(2))
        g.gptq_kv_append(keys, v, kc, vc, ks, vs, _ints(table), _ints([0]), positions=pos, inv_freq=f)
        torch.cuda.synchronize()
        return kc, ks

    kc, ks = run(k)
    turned = serve_ref.rotate(_np(k), pos.cpu().numpy()[None], _np(f))
    assert np.abs(turned).max() > float(torch.finfo(torch.float32).max)
    want, sc, quot = serve_ref.kv_append(turned, np.zeros((pages, 16, 2, dh)), np.zeros((pages, 2), np.float32), table,
                                         [0, tokens], [0])
    assert np.isfinite(sc).all() and np.array_equal(ks.cpu().numpy(), sc)
    got = kc.cpu().numpy().astype(np.float64)
    off = got != want
    assert np.all(np.abs(quot - np.floor(quot) - 0.5)[off] < 1e-9)
    k[2, 1, dh - 1] = float("inf")
    _, ks = run(k)
    assert torch.isnan(ks[0, 1]) and torch.isfinite(ks[0, 0]) and torch.isfinite(ks[1:]).all()


# --------------------------------------------------------------------------------------- byte_gemm

@pytest.mark.parametrize("m,rows", [(256, 4096), (256, 4097), (257, 2048), (513, 1280), (129, 4224), (1000, 1030)])
@pytest.mark.parametrize("stored", [False, True])
def test_products_on_both_sides_of_strips_and_tiles(stored, m, rows):
    """16 tiles of 256 x 256 and a few more, with a last partial stage of columns."""
    torch = torch_cuda()
    print(f"strips and tiles {(m, rows, stored)}", flush=True)
    x, xs, w, ws, z = _gemm_inputs(m, 400, rows, stored, seed=50)
    y = _g().gptq_byte_gemm(x, xs, w, ws, z, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    _check_gemm(x, xs, w, ws, z, y)


# ---------------------------------------------------------------------------------------- no tokens

def test_no_tokens_in_any_layout():
    """Tensors without an element pass in whatever strides where serving in 8 bits takes them; attention over packed
    sequences and norm with rotation refuse columns that are not side by side, as ever."""
    torch = torch_cuda()
    g = _g()
    z = torch.empty_strided((0, 2, 32), (0, 0, 0), dtype=torch.float16, device="cuda:0")
    kc, ks = _pool(2, 16, 2, 32, 1)
    t, n = _ints([[0], [1]]), _ints([0, 0])
    before = kc.clone()
    g.gptq_kv_append(z, z, kc, kc.clone(), ks, ks.clone(), t, n)
    assert g.gptq_kv_attention(z, kc, kc, ks, ks, t, n).shape == (0, 2, 32)
    torch.cuda.synchronize()
    assert torch.equal(kc, before)
    with pytest.raises(ValueError, match="unit stride"):
        g.gptq_norm_rotate(z)
    with pytest.raises(ValueError, match="unit stride"):
        g.gptq_attention(z, z, z)
