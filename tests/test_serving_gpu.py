"""gptq_norm_quant, gptq_byte_gemm, gptq_kv_append and gptq_kv_attention against their float64 oracle.

Tolerances count roundings. h is half a step of the type the values are stored in (torch.finfo.eps / 2) and
u = 2^-24 half a step of fp32:
* norm_quant: the sum is one fp32 addition and one rounding, bit for bit; codes are those of the exact quotient
  (unless it is within 1e-9 of a half, where 64-bit roundings decide); scales are one fp32 rounding of a 64-bit
  number, u (and 2^-149 below fp32's normal range); y one to fp32 and one to its type.
* byte_gemm: whole sums are exact, the fp32 chain sum, product, product, rounding is repeated bit for bit.
* kv_append: as norm_quant's codes, against the fp32 scale that was written, which is bit for bit.
* kv_attention: each probability is rounded once to 11 bits (fp16 and bf16 queries; 22 with fp32), 2^-11 sum p |v|
  (2^-21), and the result once, h |out|; a score's fp32 error d is at most (head_dim + 8) u times the sum of
  |q k| scale (or the score itself), which moves numerator and denominator by a factor 1 + d each; sums over keys
  add at most 64 u, as for gptq_attention. A query's own rounding to 22 bits (fp32) moves a score by 2^-22 of
  sum |q k| scale: 4 u more. Subnormal fp16 results add 2^-25, subnormal probabilities 2^-24 of the largest |v|.
"""

import numpy as np
import pytest

from gpu_util import torch_cuda
from oracle import serve_ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = ["f32", "f16", "bf16"]


def _g():
    import post_weight_quantization_20_amd as g
    return g


def _dtype(name):
    torch = torch_cuda()
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _half_step(name):
    torch = torch_cuda()
    return float(torch.finfo(_dtype(name)).eps) / 2


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _rand(shape, seed, dtype, scale=1.0):
    torch = torch_cuda()
    r = np.random.default_rng(seed)
    return torch.from_numpy(r.standard_normal(shape) * scale).to(_dtype(dtype)).to("cuda:0")


def _ints(a):
    torch = torch_cuda()
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda:0")


def _codes_match(got, want, quot):
    """Codes equal, but where the exact quotient is a border to 64 bits."""
    off = got != want
    if off.any():
        d = np.abs(quot - np.floor(quot) - 0.5)
        assert np.all(d[off] < 1e-9) and np.all(np.abs(got - want)[off] <= 1), int(off.sum())


# -------------------------------------------------------------------------------------- norm_quant

def _check_norm(dtype, x, r, w, eps, codes, scales, total, y=None):
    torch = torch_cuda()
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    if total is not None:
        assert torch.equal(total, h) or torch.equal(total.isnan(), h.isnan())
    want, sc, yy, quot = serve_ref.norm_quant(_np(h), _np(w), eps)
    got = codes.cpu().numpy().astype(np.float64)
    _codes_match(got, want, quot)
    s = _np(scales)
    assert np.array_equal(np.isnan(s), np.isnan(sc))
    ok = ~np.isnan(sc)
    assert np.all(np.abs(s - sc)[ok] <= U * 1.0001 * np.abs(sc[ok]) + 2.0 ** -149)
    if y is not None:
        o = _np(y)
        assert np.array_equal(np.isnan(o), np.isnan(yy))
        f = np.isfinite(yy)
        bound = (_half_step(dtype) * (1 + 2.0 ** -10) + U) * np.abs(yy) + 2.0 ** -25 * (dtype == "f16") + 2.0 ** -133
        assert np.all(np.abs(o - yy)[f] <= bound[f])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,d", [(1, 1), (3, 2), (5, 7), (2, 8), (9, 63), (4, 64), (7, 255), (3, 512), (6, 513), (5, 1000),
                                 (3, 1024), (2, 2048), (2, 2049), (3, 4096), (2, 4097), (1, 8192), (2, 11008), (1, 16389),
                                 (1, 40000), (1, 65536), (1, 65535)])
def test_norm_quant_sizes(n, d, dtype):
    torch = torch_cuda()
    print(f"norm_quant {(n, d, dtype)}", flush=True)
    x, r = _rand((n, d), 1, dtype, 3.0), _rand((n, d), 2, dtype)
    w = _rand((d,), 3, ["f32", "f16", "bf16"][d % 3])
    y = torch.empty_like(x)
    codes, scales, total = _g().gptq_norm_quant(x, r, w, eps=1e-5, y=y)
    torch.cuda.synchronize()
    _check_norm(dtype, x, r, w, 1e-5, codes, scales, total, y)
    codes, scales, total = _g().gptq_norm_quant(x)
    torch.cuda.synchronize()
    assert total is None
    _check_norm(dtype, x, None, None, 1e-6, codes, scales, None)


@pytest.mark.parametrize("dtype", DT)
def test_norm_quant_many_rows(dtype):
    torch = torch_cuda()
    x, r, w = _rand((1037, 96), 1, dtype), _rand((1037, 96), 2, dtype, 10.0), _rand((96,), 3, dtype)
    codes, scales, total = _g().gptq_norm_quant(x, r, w)
    torch.cuda.synchronize()
    _check_norm(dtype, x, r, w, 1e-6, codes, scales, total)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d", [96, 1030])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_norm_quant_strides_and_in_place(into, d, dtype):
    """Column ranges of wider arrays at odd offsets, the sum over an input, and what lies beside left as it was."""
    torch = torch_cuda()
    n, ld = 11, d + 5
    bx, br = _rand((n, ld), 4, dtype), _rand((n, ld), 5, dtype)
    x, r = bx[:, 3:3 + d], br[:, 1:1 + d]
    kx, kr = bx.clone(), br.clone()
    bc = torch.full((n, ld), 55, dtype=torch.int8, device="cuda:0")
    codes = bc[:, 2:2 + d]
    x0, r0 = x.clone(), r.clone()
    c, s, total = _g().gptq_norm_quant(x, r, None, codes=codes, sum_out=x if into == "x" else r)
    torch.cuda.synchronize()
    assert c is codes and total.data_ptr() == (x if into == "x" else r).data_ptr()
    _check_norm(dtype, x0, r0, None, 1e-6, codes, s, total)
    assert torch.all(bc[:, :2] == 55) and torch.all(bc[:, 2 + d:] == 55)
    (bx if into == "x" else br)[:, (3 if into == "x" else 1):][:, :d] = (x0 if into == "x" else r0)
    assert torch.equal(bx, kx) and torch.equal(br, kr)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_quant_ranges(dtype):
    """Zeros, rows whose squares leave fp32's range, ties, infinities and NaN each in their own row."""
    torch = torch_cuda()
    x = _rand((9, 260), 6, dtype)
    x[0] = 0
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3] = 1.0                       # codes of 127
    x[4] = 0.5
    x[4, 0] = 1.0                    # a tie: 63.5 is 64
    x[5, 7] = float("inf")
    x[6, 9] = float("nan")
    x[7, 1:] = 0.0
    w = torch.ones(260, device="cuda:0") * 1e3
    y = torch.empty_like(x)
    for eps in (0.0, 1e-6):
        codes, scales, _ = _g().gptq_norm_quant(x, None, w, eps=eps, y=y)
        torch.cuda.synchronize()
        _check_norm(dtype, x, None, w, eps, codes, scales, None, y)
        assert torch.all(codes[0] == 0) and scales[0] == 0 and torch.all(y[0] == 0)
        assert torch.all(codes[3] == 127) and torch.all(codes[4, 1:] == 64)
        assert torch.isnan(scales[5:7]).all() and torch.all(codes[5:7] == 0) and torch.isfinite(scales[7:]).all()
    w[3] = float("inf")
    codes, scales, _ = _g().gptq_norm_quant(x, None, w)
    torch.cuda.synchronize()
    assert torch.isnan(scales).all() and torch.all(codes == 0)


def test_norm_quant_norm_alone():
    """Without codes: the C entry takes y alone."""
    import ctypes
    from post_weight_quantization_20_amd import _lib
    torch = torch_cuda()
    x = _rand((5, 300), 7, "f16")
    y = torch.empty_like(x)
    a = _lib.gptq_norm_quant_t(5, 300, 300, 0, 0, 300, 0, 1e-6, 1, 0)
    st = _lib.lib().gptq_norm_quant(ctypes.byref(a), x.data_ptr(), None, None, None, y.data_ptr(), None, None,
                                    torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    _, _, yy, _ = serve_ref.norm_quant(_np(x), None, 1e-6)
    assert np.all(np.abs(_np(y) - yy) <= (2.0 ** -11 * 1.001 + U) * np.abs(yy) + 2.0 ** -25)


# --------------------------------------------------------------------------------------- byte_gemm

def _gemm_inputs(m, d, rows, stored, seed=1, top=127):
    torch = torch_cuda()
    r = np.random.default_rng(seed)
    x = torch.from_numpy(r.integers(-top, top + 1, (m, d)).astype(np.int8)).cuda()
    xs = torch.from_numpy(r.uniform(0.001, 0.1, m).astype(np.float32)).cuda()
    ws = torch.from_numpy(r.uniform(0.001, 0.1, rows).astype(np.float32)).cuda()
    if stored:
        w = torch.from_numpy(r.integers(0, 256, (rows, d)).astype(np.uint8)).cuda()
        z = _ints(r.integers(90, 160, rows))
    else:
        w, z = torch.from_numpy(r.integers(-128, 128, (rows, d)).astype(np.int8)).cuda(), None
    return x, xs, w, ws, z


def _check_gemm(x, xs, w, ws, z, y):
    torch = torch_cuda()
    # whole sums below 2^53: float64 products are exact
    wd = w.double() if z is None else w.double() - z.double()[:, None]
    whole = torch.matmul(x.double(), wd.T)
    v = whole.float()
    if xs is not None:
        v = v * xs[:, None]
    if ws is not None:
        v = v * ws
    want = v.to(y.dtype)
    assert torch.equal(y, want), float((y.double() - want.double()).abs().max())


GEMM = [(1, 1, 1), (1, 16, 16), (2, 31, 3), (3, 64, 17), (5, 100, 33), (8, 128, 64), (16, 256, 100), (17, 512, 16),
        (31, 1000, 65), (32, 1024, 48), (33, 4096, 129), (64, 333, 257), (65, 2048, 128), (100, 96, 1000),
        (128, 1024, 256), (129, 80, 131), (255, 640, 300), (256, 512, 512), (257, 4096, 513), (1000, 72, 520),
        (513, 1001, 700), (1, 11008, 4096), (4, 4096, 11008), (700, 4096, 1024)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("stored", [False, True])
@pytest.mark.parametrize("m,d,rows", GEMM)
def test_byte_gemm_sizes(m, d, rows, stored, dtype):
    torch = torch_cuda()
    print(f"byte_gemm {(m, d, rows, stored, dtype)}", flush=True)
    x, xs, w, ws, z = _gemm_inputs(m, d, rows, stored)
    y = _g().gptq_byte_gemm(x, xs, w, ws, z, dtype=_dtype(dtype))
    torch.cuda.synchronize()
    _check_gemm(x, xs, w, ws, z, y)
    if dtype == "f32":
        plain = _g().gptq_byte_gemm(x, None, w, None, z)
        torch.cuda.synchronize()
        _check_gemm(x, None, w, None, z, plain)


def test_byte_gemm_against_the_oracle():
    torch = torch_cuda()
    for stored in (False, True):
        x, xs, w, ws, z = _gemm_inputs(7, 300, 40, stored, seed=3)
        y = _g().gptq_byte_gemm(x, xs, w, ws, z)
        torch.cuda.synchronize()
        _, want = serve_ref.byte_gemm(x.cpu().numpy(), _np(xs), w.cpu().numpy(), _np(ws),
                                      None if z is None else z.cpu().numpy())
        assert np.all(np.abs(_np(y) - want) <= 3.01 * U * np.abs(want))


@pytest.mark.parametrize("m", [1, 40, 300])
@pytest.mark.parametrize("stored", [False, True])
def test_byte_gemm_strides(stored, m):
    """Column ranges at odd offsets, pitched outputs, and what lies beside left as it was."""
    torch = torch_cuda()
    d, rows = 150, 70
    x, xs, w, ws, z = _gemm_inputs(m, d + 7, rows, stored, seed=5)
    x, w = x[:, 3:3 + d], w[:, 5:5 + d]
    base = torch.full((m, rows + 9), 3.0, device="cuda:0")
    y = base[:, 4:4 + rows]
    _g().gptq_byte_gemm(x, xs, w, ws, z, y=y)
    torch.cuda.synchronize()
    _check_gemm(x, xs, w, ws, z, y)
    assert torch.all(base[:, :4] == 3.0) and torch.all(base[:, 4 + rows:] == 3.0)


@pytest.mark.parametrize("m", [2, 64, 300])
def test_byte_gemm_largest_sums(m):
    """The longest rows of extreme values, with zeros far outside the codes."""
    torch = torch_cuda()
    d, rows = 131071, 20
    x = torch.full((m, d), -128, dtype=torch.int8, device="cuda:0")
    w = torch.full((rows, d), -128, dtype=torch.int8, device="cuda:0")
    x[1::2] = 127
    w[1::3] = 127
    y = _g().gptq_byte_gemm(x, None, w, None)
    torch.cuda.synchronize()
    _check_gemm(x, None, w, None, None, y)
    wu = torch.full((rows, d), 255, dtype=torch.uint8, device="cuda:0")
    wu[::2] = 0
    z = _ints([0, 255, -1000000, 1000000, 2 ** 31 - 1, -2 ** 31, 128, 1 << 28, 1, 254] * 2)
    y = _g().gptq_byte_gemm(x, None, wu, None, z)
    torch.cuda.synchronize()
    _check_gemm(x, None, wu, None, z, y)


def test_byte_gemm_not_a_number_stays_in_its_row():
    torch = torch_cuda()
    x, xs, w, ws, z = _gemm_inputs(40, 256, 50, False)
    xs[3], ws[7] = float("nan"), float("inf")
    y = _g().gptq_byte_gemm(x, xs, w, ws)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[3], want[:, 7] = True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("sym", [0, 1])
def test_byte_gemm_takes_stored_layers(sym):
    """A layer quantized to 8 bits with one group per row: its codes and gptq_pack's words give one product, that of
    gptq_dequant_gemm."""
    torch = torch_cuda()
    g = _g()
    rows, d = 96, 256
    W, X = _rand((rows, d), 1, "f16", 0.02), _rand((1024, d), 2, "f16")
    p = g.Params(bits=8, group_size=0, block_size=128, sym=bool(sym))
    res = g.quantize_layer(W, [X], p)
    out = res.quant
    packed = g.gptq_pack(out.codes, 8)
    x = X[:48]
    codes, scales, _ = g.gptq_norm_quant(x, eps=0.0)
    a = g.gptq_byte_gemm(codes, scales, out.codes, out.scales, out.zeros)
    b = g.gptq_byte_gemm(codes, scales, packed.view(rows, d // 4), out.scales, out.zeros)
    xv = codes.float() * scales[:, None]
    c = g.gptq_dequant_gemm(xv, packed, out.scales, out.zeros, d, group_size=0, bits=8)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    _check_gemm(codes, scales, out.codes, out.scales.reshape(-1), out.zeros.reshape(-1), a)
    wd = (out.codes.double() - out.zeros.reshape(rows, 1).double()) * out.scales.reshape(rows, 1).double()
    mag = xv.double().abs() @ wd.abs().T
    assert torch.all((a.double() - c.double()).abs() <= (d + 16) * U * mag)


# --------------------------------------------------------------------------------------- kv_append

def _pool(pages, ps, hk, dh, seed, layout="slots"):
    """(cache, scales): random codes and scales; layout: slots outside heads or heads outside slots."""
    torch = torch_cuda()
    r = np.random.default_rng(seed)
    c = torch.from_numpy(r.integers(-127, 128, (pages, ps, hk, dh)).astype(np.int8)).cuda()
    if layout == "heads":
        c = c.transpose(1, 2).contiguous().transpose(1, 2)
    return c, torch.from_numpy(r.uniform(0.004, 0.04, (pages, hk)).astype(np.float32)).cuda()


def _table(seqs, max_pages, pages, seed):
    """Distinct pages in random order."""
    r = np.random.default_rng(seed)
    assert seqs * max_pages <= pages
    return r.permutation(pages)[:seqs * max_pages].reshape(seqs, max_pages).astype(np.int32)


def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _run_append(dtype, news, pasts, hk, dh, ps=16, rd=None, inter=False, axes=1, positions=None, layout="slots",
                max_pages=None, table=None, start=None, kscale=1.0, even=False, seed=1, data=None):
    torch = torch_cuda()
    print(f"kv_append {(dtype, news, pasts, hk, dh, ps, rd, inter, axes, layout)}", flush=True)
    rd = dh // 2 * 2 if rd is None else rd
    n = sum(news)
    seqs = len(news)
    max_pages = max_pages or max(1, max(-(-(a + b) // ps) for a, b in zip(news, pasts)))
    pages = seqs * max_pages + 3
    kc, ksc = _pool(pages, ps, hk, dh, seed, layout)
    vc, vsc = _pool(pages, ps, hk, dh, seed + 1, layout)
    table = _table(seqs, max_pages, pages, seed + 2) if table is None else table
    if data is None:
        qkv = _rand((n, 2 * hk, dh), seed + 3, dtype, kscale)
        k, v = qkv[:, :hk], qkv[:, hk:]
    else:
        k, v = data
    start = _starts(news) if start is None else start
    r = np.random.default_rng(seed + 4)
    f = pos = axis = None
    if rd:
        f = torch.from_numpy((10000.0 ** (-np.arange(rd // 2) * 2 / rd)).astype(np.float32)).cuda()
        if positions is not None:
            pos = _ints(r.integers(-positions, positions, (axes, n)))
            axis = _ints(r.integers(-1, axes + 1, rd // 2)) if axes > 1 else None
    before = [t.cpu().numpy() for t in (kc, vc, ksc, vsc)]
    _g().gptq_kv_append(k, v, kc, vc, ksc, vsc, _ints(table), _ints(pasts), start=None if even else _ints(start),
                        positions=pos, inv_freq=f, pair_axis=axis, interleaved=inter)
    torch.cuda.synchronize()
    kd = _np(k)
    if rd:
        if pos is None:
            place = np.zeros((1, n), dtype=np.int64)
            for s in range(seqs):
                place[0, start[s]:start[s + 1]] = pasts[s] + np.arange(start[s + 1] - start[s])
        else:
            place = pos.cpu().numpy()
        kd = serve_ref.rotate(kd, place, _np(f), None if axis is None else axis.cpu().numpy(), inter)
    for x, cache, scales, c0, s0 in ((kd, kc, ksc, before[0], before[2]), (_np(v), vc, vsc, before[1], before[3])):
        want, ws, quot = serve_ref.kv_append(x, c0, s0, np.asarray(table), start, pasts)
        got = scales.cpu().numpy()
        assert np.array_equal(got, ws, equal_nan=True), float(np.nanmax(np.abs(got - ws)))
        _codes_match(cache.cpu().numpy().astype(np.float64), want, quot)
    return kc, vc, ksc, vsc


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("news,pasts", [
    ([1], [0]), ([1], [1]), ([1], [15]), ([1], [16]), ([5], [13]), ([16], [0]), ([17], [0]), ([33], [15]), ([0, 3], [4, 0]),
    ([1, 1, 1, 1], [0, 7, 15, 31]), ([100, 0, 1, 37], [3, 5, 47, 16]), ([2] * 70, list(range(70))), ([400], [9]),
], ids=str)
def test_kv_append_lengths(news, pasts, dtype):
    _run_append(dtype, news, pasts, 2, 64)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("hk,dh,rd,inter", [
    (1, 1, 0, False), (1, 2, 2, True), (3, 7, 4, False), (2, 20, 20, True), (1, 16, 8, False), (5, 72, 36, False),
    (8, 128, 128, False), (8, 128, 64, True), (4, 80, 80, True), (9, 96, 0, False), (2, 256, 256, False),
    (1, 1024, 1024, True), (17, 33, 32, False), (1, 1023, 1022, False)], ids=str)
def test_kv_append_heads(hk, dh, rd, inter, dtype):
    _run_append(dtype, [19, 1, 4], [5, 0, 30], hk, dh, rd=rd, inter=inter)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("ps", [16, 32, 48, 112, 256, 1024])
def test_kv_append_page_sizes(ps, dtype):
    for layout in ("slots", "heads"):
        _run_append(dtype, [1, 300, ps, 2 * ps + 1], [ps - 1, 7, 0, 1], 2, 32, ps=ps, layout=layout)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_kv_append_positions(dtype):
    _run_append(dtype, [40, 3], [100, 0], 2, 64, positions=1 << 20)
    _run_append(dtype, [40, 3], [100, 0], 2, 96, rd=48, axes=3, positions=300, inter=True)
    _run_append(dtype, [3, 3], [1000000, 12], 2, 64, max_pages=62503, table=np.tile(np.arange(2, dtype=np.int32)[:, None],
                                                                                 (1, 62503)))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kscale", [1e-3, 1e-30, 0.0, 1e3])
def test_kv_append_scales_grow_or_stay(kscale, dtype):
    _run_append(dtype, [3, 1, 20], [5, 18, 12], 3, 48, kscale=kscale if dtype != "f16" or kscale > 1e-20 else 1e-7)


def test_kv_append_out_of_the_table():
    """Pages outside the pool, tokens past the table's end, ranges that leave the rows, lengths that leave the table."""
    table = np.array([[0, 9999, 2], [-1, 4, 5], [6, 7, 8]], dtype=np.int32)
    _run_append("f32", [40, 30, 10], [2, 10, 45], 2, 32, table=table, max_pages=3)
    _run_append("f32", [5, 6, 4], [48, 0, 1000], 2, 32, table=table, max_pages=3)
    _run_append("f32", [5, 6, 4], [3, -7, 2], 2, 32, table=table, max_pages=3, start=np.array([0, 5, 11, 1 << 30], np.int32),
                positions=50)
    _run_append("f32", [5, 6, 4], [3, 7, 2], 2, 32, table=table, max_pages=3, start=np.array([4, 2, 9, 9], np.int32),
                positions=50)


def test_kv_append_equal_ranges_and_again():
    """Without start: equal ranges. The same tokens again change nothing."""
    torch = torch_cuda()
    kc, vc, ks, vs = _run_append("f16", [4, 4, 4], [13, 0, 31], 2, 64, even=True)
    g = _g()
    k, v = _rand((6, 2, 64), 50, "f16", 5.0), _rand((6, 2, 64), 51, "f16")
    t = _ints([[0, 1], [2, 3]])
    args = (k, v, kc, vc, ks, vs, t, _ints([13, 4]))
    g.gptq_kv_append(*args)
    kept = [x.clone() for x in (kc, vc, ks, vs)]
    g.gptq_kv_append(*args)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, (kc, vc, ks, vs)))


@pytest.mark.parametrize("bad", ["inf", "nan"])
def test_kv_append_not_a_number(bad):
    """An infinity or NaN makes its page's scale of its head NaN until the page is begun again."""
    torch = torch_cuda()
    data = (_rand((20, 2, 32), 60, "f32"), _rand((20, 2, 32), 61, "f32"))
    data[0][2, 1, 3] = float(bad)
    data[1][17, 0, 5] = float(bad)
    kc, vc, ks, vs = _run_append("f32", [20], [3], 2, 32, data=data, table=np.array([[0, 1]], np.int32), max_pages=2)
    assert torch.isnan(ks[0, 1]) and torch.isfinite(ks[0, 0]) and torch.isnan(vs[1, 0]) and torch.isfinite(vs[1, 1])
    g = _g()
    k = _rand((1, 2, 32), 62, "f32")
    g.gptq_kv_append(k, k, kc, vc, ks, vs, _ints([[0, 1]]), _ints([5]))
    torch.cuda.synchronize()
    assert torch.isnan(ks[0, 1])
    g.gptq_kv_append(k, k, kc, vc, ks, vs, _ints([[0, 1]]), _ints([0]))
    torch.cuda.synchronize()
    assert torch.isfinite(ks[0]).all()


def test_kv_append_keys_and_values_in_one_array():
    """Keys and values interleaved by page and by head."""
    torch = torch_cuda()
    g = _g()
    k, v = _rand((21, 2, 32), 70, "bf16"), _rand((21, 2, 32), 71, "bf16")
    t = _ints([[1, 0]])
    ref = [torch.zeros(2, 16, 2, 32, dtype=torch.int8, device="cuda:0") for _ in range(2)]
    sc = [torch.zeros(2, 2, device="cuda:0") for _ in range(4)]
    g.gptq_kv_append(k, v, *ref, *sc[:2], t, _ints([0]))
    both = torch.zeros(2, 2, 16, 2, 32, dtype=torch.int8, device="cuda:0")
    g.gptq_kv_append(k, v, both[:, 0], both[:, 1], *sc[2:], t, _ints([0]))
    torch.cuda.synchronize()
    assert torch.equal(both[:, 0], ref[0]) and torch.equal(both[:, 1], ref[1])
    pairs = torch.zeros(2, 16, 2, 64, dtype=torch.int8, device="cuda:0")
    g.gptq_kv_append(k, v, pairs[..., :32], pairs[..., 32:], *sc[2:], t, _ints([0]))
    torch.cuda.synchronize()
    assert torch.equal(pairs[..., :32], ref[0]) and torch.equal(pairs[..., 32:], ref[1])
    assert torch.equal(sc[0], sc[2]) and torch.equal(sc[1], sc[3])


# ------------------------------------------------------------------------------------ kv_attention

def _check_kv(dtype, q, caches, table, start, lens, out, scale, causal, window, cap, slopes, fill):
    dh = q.shape[2]
    kc, vc, ks, vs = (t.cpu().numpy() for t in caches)
    want, mag, spread, written = serve_ref.kv_attention(_np(q), kc, vc, ks, vs, np.asarray(table), start, lens, scale,
                                                        causal, window, cap, _np(slopes))
    got = _np(out)
    assert np.all(got[~written] == fill)
    rounding = 2.0 ** -11 if dtype != "f32" else 2.0 ** -21
    vmax = 127.0 * float(np.nanmax(np.where(np.isfinite(vs), vs, 0.0)))
    bound = _half_step(dtype) * np.abs(want) + (rounding + (2 * (dh + 12) * spread + 64) * U) * mag \
        + 2.0 ** -25 * (dtype == "f16") + 2.0 ** -24 * vmax * (mag > 0)
    err = np.abs(got - want)[written]
    assert np.all(err <= bound[written]), float(np.max(err / np.maximum(bound[written], 1e-300)))


def _run_kv(dtype, hq, hk, dh, seqs, ps=16, scale=None, causal=True, window=0, cap=0.0, bias=False, work=True, layout="slots",
            table=None, max_pages=None, even=False, extra=0, seed=1, qs=1.0, strided=False):
    """seqs: (queries, cached tokens) of each."""
    torch = torch_cuda()
    print(f"kv_attention {(dtype, hq, hk, dh, seqs[:6], ps, causal, window, cap, bias, work, layout)}", flush=True)
    news, lens = [a for a, _ in seqs], [b for _, b in seqs]
    nq = sum(news) + extra
    max_pages = max_pages or max(1, max(-(-b // ps) for b in lens))
    pages = len(seqs) * max_pages + 5
    kc, ks = _pool(pages, ps, hk, dh, seed, layout)
    vc, vs = _pool(pages, ps, hk, dh, seed + 1, layout)
    table = _table(len(seqs), max_pages, pages, seed + 2) if table is None else np.asarray(table, np.int32)
    # pages that no sequence names hold scales of nothing, and what stands behind a sequence's last page no page
    used = set()
    for row, n in zip(table, lens):
        used |= {int(p) for p in row[:-(-n // ps)]}
    for p in range(pages):
        if p not in used:
            ks[p], vs[p] = float("nan"), float("inf")
    if strided:
        q = _rand((nq, hq + 3, dh), seed + 3, dtype, qs)[:, 1:1 + hq]
        out = torch.full((hq, nq, dh), 7.0, dtype=q.dtype, device="cuda:0").transpose(0, 1)
    else:
        q = _rand((nq, hq, dh), seed + 3, dtype, qs)
        out = torch.full((nq, hq, dh), 7.0, dtype=q.dtype, device="cuda:0")
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device="cuda:0") if bias else None
    start = _starts(news)
    g = _g()
    w = None if work else torch.empty(0, dtype=torch.uint8, device="cuda:0")
    g.gptq_kv_attention(q, kc, vc, ks, vs, _ints(table), _ints(lens), scale=scale, causal=causal,
                        q_start=None if even else _ints(start), window=window, softcap=cap, slopes=slopes, out=out, work=w)
    torch.cuda.synchronize()
    _check_kv(dtype, q, (kc, vc, ks, vs), table, start, lens, out, dh ** -0.5 if scale is None else scale, causal,
              window, cap, slopes, 7.0)
    return q, (kc, vc, ks, vs), table, out


KV = {
    "one": [(1, 1)], "two": [(2, 2)], "15": [(1, 15)], "16": [(1, 16)], "17": [(1, 17)], "31": [(3, 31)], "32": [(1, 32)],
    "33": [(1, 33)], "prompt": [(70, 70)], "prompts": [(5, 5), (0, 0), (130, 130), (1, 1), (33, 33)], "long": [(257, 257)],
    "tokens": [(1, 300), (1, 1), (1, 64), (1, 129)], "chunk": [(7, 200), (40, 41), (3, 3)], "nokeys": [(3, 0), (4, 4)],
    "noqueries": [(0, 5), (2, 9)], "more_queries": [(9, 4), (70, 2)], "chunks": [(150, 400), (1, 300), (64, 64)],
}


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lens", list(KV), ids=str)
def test_kv_attention_lengths(lens, dtype):
    _run_kv(dtype, 4, 2, 64, KV[lens], extra=2)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("dh", [1, 7, 8, 16, 20, 32, 48, 64, 72, 80, 96, 112, 128, 136, 192, 200, 256, 260, 1024])
def test_kv_attention_head_widths(dh, dtype):
    _run_kv(dtype, 2, 1, dh, [(70, 70), (1, 90)])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (7, 1), (6, 2), (40, 8), (33, 1), (130, 1), (16, 16)])
def test_kv_attention_shared_heads(hq, hk, dtype):
    _run_kv(dtype, hq, hk, 32, [(35, 35), (1, 70), (2, 3)])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kw", [
    dict(causal=False), dict(window=1), dict(window=17), dict(window=64), dict(window=64, causal=False), dict(window=1000),
    dict(window=2 ** 31 - 1), dict(cap=2.0), dict(cap=50.0, causal=False), dict(cap=5000.0), dict(bias=True),
    dict(bias=True, causal=False), dict(bias=True, cap=3.0, window=40), dict(scale=-0.3), dict(scale=0.0),
    dict(scale=-0.3, cap=3.0), dict(cap=1e-6), dict(cap=1e7, bias=True)], ids=str)
def test_kv_attention_masks(kw, dtype):
    _run_kv(dtype, 4, 2, 64, [(9, 9), (200, 200), (66, 140), (1, 333)], **kw)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("ps", [16, 32, 48, 80, 128, 1024])
def test_kv_attention_page_sizes(ps, dtype):
    for layout in ("slots", "heads"):
        _run_kv(dtype, 4, 2, 64, [(3, 200), (1, 1500), (90, 130)], ps=ps, layout=layout)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("work", [True, False])
def test_kv_attention_long_caches(work, dtype):
    """Few queries against long key ranges: split across workgroups with the workspace, whole without it."""
    _run_kv(dtype, 8, 2, 128, [(1, 9001), (2, 700), (1, 1), (5, 4097)], work=work)
    _run_kv(dtype, 4, 4, 80, [(1, 5000)], cap=20.0, work=work, ps=48)
    _run_kv(dtype, 2, 1, 64, [(3, 3000), (1, 0)], bias=True, causal=False, work=work)
    _run_kv(dtype, 2, 1, 64, [(3, 8000), (40, 5000)], window=900, work=work)


@pytest.mark.parametrize("dtype", DT)
def test_kv_attention_pages_left_out(dtype):
    """Pages outside the pool are not seen; a query all of whose pages are is a row of zeros; shared pages."""
    table = [[3, -1, 4, 9999], [3, 1, 2, 0], [-1, -5, 77777, -1]]
    q, _, _, out = _run_kv(dtype, 4, 2, 64, [(5, 60), (2, 50), (3, 64)], table=table, max_pages=4)
    assert (out[7:] == 0).all()
    _run_kv(dtype, 4, 2, 64, [(50, 60), (2, 50), (40, 64)], table=table, max_pages=4, window=20)


@pytest.mark.parametrize("dtype", DT)
def test_kv_attention_strides(dtype):
    _run_kv(dtype, 4, 2, 64, [(1, 100), (2, 40)], strided=True, layout="heads")
    _run_kv(dtype, 6, 2, 40, [(90, 100), (2, 40)], strided=True)
    _run_kv(dtype, 4, 2, 64, [(3, 100), (3, 40)], even=True)


@pytest.mark.parametrize("dtype", DT)
def test_kv_attention_many_sequences(dtype):
    r = np.random.default_rng(3)
    _run_kv(dtype, 2, 2, 32, [(1, int(b)) for b in r.integers(0, 60, 300)])
    _run_kv(dtype, 4, 1, 32, [(int(a), int(a + b)) for a, b in zip(r.integers(0, 30, 150), r.integers(0, 40, 150))])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_kv_attention_large_scores(dtype):
    _run_kv(dtype, 2, 2, 64, [(150, 150), (1, 200)], qs=300.0)
    _run_kv(dtype, 2, 2, 64, [(150, 150), (1, 200)], qs=1e-20)


@pytest.mark.parametrize("dtype", DT)
def test_kv_attention_value_scales_far_apart(dtype):
    """Pages whose value scales differ by powers of ten."""
    torch = torch_cuda()
    q, (kc, vc, ks, vs), table, out = _run_kv(dtype, 4, 2, 64, [(1, 200), (40, 100)])
    for i in range(vs.shape[0]):
        if torch.isfinite(vs[i]).all():
            vs[i] *= 10.0 ** (i % 7 - 3)
    lens = [200, 100]
    _g().gptq_kv_attention(q, kc, vc, ks, vs, _ints(table), _ints(lens), q_start=_ints([0, 1, 41]), out=out)
    torch.cuda.synchronize()
    _check_kv(dtype, q, (kc, vc, ks, vs), table, [0, 1, 41], lens, out, 0.125, True, 0, 0.0, None, 7.0)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("news", [2, 60])
def test_kv_attention_not_a_number(news, dtype):
    """A query that holds a NaN gives NaN in its own rows alone; a page whose value scale is NaN in the rows that see
    it; scales of unseen pages change nothing."""
    torch = torch_cuda()
    q, (kc, vc, ks, vs), table, out = _run_kv(dtype, 4, 2, 64, [(news, 200)])
    kept = out.clone()
    q[1, 2, 5] = float("nan")
    t, n = _ints(table), _ints([200])
    got = _g().gptq_kv_attention(q, kc, vc, ks, vs, t, n)
    torch.cuda.synchronize()
    assert torch.isnan(got[1, 2]).all()
    got[1, 2] = kept[1, 2]
    assert torch.equal(got, kept)
    q[1, 2, 5] = 0.0
    page = int(table[0, 8])          # keys 128 .. 143
    base = _g().gptq_kv_attention(q, kc, vc, ks, vs, t, n, window=40)
    vs[page] = float("nan")
    got = _g().gptq_kv_attention(q, kc, vc, ks, vs, t, n, window=40)
    torch.cuda.synchronize()
    p = 200 - news + np.arange(news)
    sees = (p - 143 < 40) & (p >= 128)
    for i in range(news):
        assert torch.isnan(got[i]).all() if sees[i] else torch.equal(got[i], base[i])


def test_kv_attention_offsets_past_32_bits():
    """Pages further than 4 GiB from the cache's start."""
    torch = torch_cuda()
    g = _g()
    ps, hk, dh = 1024, 8, 128
    pages = (5 << 30) // (ps * hk * dh)
    kc, vc = (torch.zeros(pages, ps, hk, dh, dtype=torch.int8, device="cuda:0") for _ in range(2))
    ks, vs = (torch.zeros(pages, hk, device="cuda:0") for _ in range(2))
    t = _ints([[pages - 1, 1, pages - 3]])
    k, v = _rand((2100, hk, dh), 1, "bf16"), _rand((2100, hk, dh), 2, "bf16")
    g.gptq_kv_append(k, v, kc, vc, ks, vs, t, _ints([5]))
    small = [torch.zeros(3, ps, hk, dh, dtype=torch.int8, device="cuda:0") for _ in range(2)]
    ss = [torch.zeros(3, hk, device="cuda:0") for _ in range(2)]
    g.gptq_kv_append(k, v, *small, *ss, _ints([[0, 1, 2]]), _ints([5]))
    torch.cuda.synchronize()
    at = [pages - 1, 1, pages - 3]
    assert torch.equal(kc[at], small[0]) and torch.equal(vc[at], small[1]) and torch.equal(ks[at], ss[0])
    for nq in (1, 100):
        q = _rand((nq, 16, dh), 3, "bf16")
        a = g.gptq_kv_attention(q, kc, vc, ks, vs, t, _ints([2105]))
        b = g.gptq_kv_attention(q, *small, *ss, _ints([[0, 1, 2]]), _ints([2105]))
        torch.cuda.synchronize()
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------- streams and graphs

def _step(g, s):
    """One serving step: norm, projections, append, attention, projection."""
    codes, sc, h = g.gptq_norm_quant(s["x"], s["r"], s["w"], sum_out=s["h"], codes=s["codes"], scales=s["sc"])
    n, hq, hk, dh = s["dims"]
    q = g.gptq_byte_gemm(codes, sc, s["wq"], s["wqs"], s["wqz"], y=s["q"])
    kv = g.gptq_byte_gemm(codes, sc, s["wkv"], s["wkvs"], y=s["kv"])
    q3 = q.view(n, hq, dh)
    g.gptq_norm_rotate(q3, None, s["pos"], s["f"], norm=False, q_out=q3)
    kv3 = kv.view(n, 2 * hk, dh)
    g.gptq_kv_append(kv3[:, :hk], kv3[:, hk:], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["past"],
                     start=s["start"], inv_freq=s["f"])
    g.gptq_kv_attention(q3, s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], q_start=s["start"], out=s["o"],
                        work=s["work"])
    oc, osc, _ = g.gptq_norm_quant(s["o"].view(n, hq * dh), codes=s["oc"], scales=s["osc"])
    g.gptq_byte_gemm(oc, osc, s["wo"], s["wos"], y=s["y"])


def _state(news, pasts, seed=1):
    torch = torch_cuda()
    g = _g()
    n, hq, hk, dh, d = sum(news), 8, 2, 64, 512
    r = np.random.default_rng(seed)
    s = {"dims": (n, hq, hk, dh)}
    s["x"], s["r"], s["w"] = _rand((n, d), seed, "bf16"), _rand((n, d), seed + 1, "bf16"), _rand((d,), seed + 2, "bf16")

    def i8(*shape):
        return torch.from_numpy(r.integers(-127, 128, shape).astype(np.int8)).cuda()

    def sc(*shape):
        return torch.from_numpy(r.uniform(0.0005, 0.001, shape).astype(np.float32)).cuda()

    s["wq"] = torch.from_numpy(r.integers(0, 256, (hq * dh, d)).astype(np.uint8)).cuda()
    s["wqs"], s["wqz"] = sc(hq * dh), _ints(r.integers(120, 136, hq * dh))
    s["wkv"], s["wkvs"] = i8(2 * hk * dh, d), sc(2 * hk * dh)
    s["wo"], s["wos"] = i8(d, hq * dh), sc(d)
    ps = 16
    maxp = max(-(-(a + b) // ps) for a, b in zip(news, pasts)) + 1
    s["kc"], s["ks"] = _pool(len(news) * maxp, ps, hk, dh, seed + 5)
    s["vc"], s["vs"] = _pool(len(news) * maxp, ps, hk, dh, seed + 6)
    s["table"] = _ints(_table(len(news), maxp, len(news) * maxp, seed + 7))
    s["past"], s["lens"] = _ints(pasts), _ints([a + b for a, b in zip(news, pasts)])
    s["start"] = _ints(_starts(news))
    s["f"] = torch.from_numpy((10000.0 ** (-np.arange(dh // 2) * 2 / dh)).astype(np.float32)).cuda()
    s["pos"] = _ints(np.concatenate([b + np.arange(a) for a, b in zip(news, pasts)]))
    bf = torch.bfloat16
    for name, shape, dt in (("h", (n, d), bf), ("codes", (n, d), torch.int8), ("sc", (n,), torch.float32),
                            ("q", (n, hq * dh), bf), ("kv", (n, 2 * hk * dh), bf), ("o", (n, hq, dh), bf),
                            ("oc", (n, hq * dh), torch.int8), ("osc", (n,), torch.float32), ("y", (n, d), bf)):
        s[name] = torch.zeros(shape, dtype=dt, device="cuda:0")
    nb = g.gptq_kv_attention_workspace_bytes(s["o"], s["kc"], s["table"])
    s["work"] = torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda:0")
    return s


@pytest.mark.parametrize("news,pasts", [([1, 1, 1], [40, 3, 15]), ([30, 1, 77], [0, 400, 20])], ids=str)
def test_a_serving_step(news, pasts):
    """The operators in the order of a decoder layer's attention half, each checked on what it was given."""
    torch = torch_cuda()
    s = _state(news, pasts)
    n, hq, hk, dh = s["dims"]
    before = [t.cpu().numpy() for t in (s["kc"], s["vc"], s["ks"], s["vs"])]
    _step(_g(), s)
    torch.cuda.synchronize()
    _check_norm("bf16", s["x"], s["r"], s["w"], 1e-6, s["codes"], s["sc"], s["h"])
    _check_gemm(s["codes"], s["sc"], s["wkv"], s["wkvs"], None, s["kv"])
    kv = _np(s["kv"].view(n, 2 * hk, dh))
    k = serve_ref.rotate(kv[:, :hk], s["pos"].cpu().numpy()[None], _np(s["f"]))
    start = _starts(news)
    table = s["table"].cpu().numpy()
    for x, c, sc, c0, s0 in ((k, s["kc"], s["ks"], before[0], before[2]), (kv[:, hk:], s["vc"], s["vs"], before[1],
                                                                           before[3])):
        want, ws, quot = serve_ref.kv_append(x, c0, s0, table, start, pasts)
        assert np.array_equal(sc.cpu().numpy(), ws)
        _codes_match(c.cpu().numpy().astype(np.float64), want, quot)
    # the rotated queries the attention was given
    lens = [a + b for a, b in zip(news, pasts)]
    _check_kv("bf16", s["q"].view(n, hq, dh), (s["kc"], s["vc"], s["ks"], s["vs"]), table, start, lens, s["o"], dh ** -0.5,
              True, 0, 0.0, None, 0.0)
    _check_norm("bf16", s["o"].view(n, hq * dh), None, None, 1e-6, s["oc"], s["osc"], None)
    _check_gemm(s["oc"], s["osc"], s["wo"], s["wos"], None, s["y"])


def test_a_captured_step_on_changing_inputs():
    """A decode step in a graph, replayed on new inputs and growing caches, with eager work in between; two graphs
    with their own workspaces."""
    torch = torch_cuda()
    g = _g()
    s, e = _state([1, 1, 1], [40, 3, 15]), _state([1, 1, 1], [40, 3, 15])
    names = ("h", "codes", "sc", "q", "kv", "o", "oc", "osc", "y", "kc", "vc", "ks", "vs")
    side = torch.cuda.Stream()
    kept = {k: s[k].clone() for k in names}
    with torch.cuda.stream(side):
        _step(g, s)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        s["work"] = torch.empty_like(s["work"])
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            _step(g, s)
        graphs.append((gr, s["work"]))
    for k in names:
        s[k].copy_(kept[k])
    for i in range(6):
        x = _rand(tuple(s["x"].shape), 100 + i, "bf16")
        for t in (s, e):
            t["x"].copy_(x)
            if i:
                for k in ("past", "lens", "pos"):
                    t[k].add_(1)
        graphs[i % 2][0].replay()
        _step(g, e)
        torch.cuda.synchronize()
        for k in names:
            assert torch.equal(s[k], e[k]), (i, k)


def test_calls_on_two_streams_at_once():
    torch = torch_cuda()
    g = _g()
    states = [_state([1, 20, 1], [300, 3, 15], seed=s) for s in (1, 2)]
    want = [_state([1, 20, 1], [300, 3, 15], seed=s) for s in (1, 2)]
    for w in want:
        _step(g, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(3):
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                _step(g, s)
    torch.cuda.synchronize()
    for s, w in zip(states, want):
        assert all(torch.equal(s[k], w[k]) for k in ("y", "o", "kc", "vc", "ks", "vs"))


def test_the_stream_argument():
    torch = torch_cuda()
    g = _g()
    st = torch.cuda.Stream()
    x = _rand((3, 64), 1, "f16")
    torch.cuda.synchronize()
    codes, sc, _ = g.gptq_norm_quant(x, stream=st)
    w = torch.ones(16, 64, dtype=torch.int8, device="cuda:0")
    torch.cuda.synchronize()
    y = g.gptq_byte_gemm(codes, sc, w, None, stream=st)
    st.synchronize()
    _check_norm("f16", x, None, None, 1e-6, codes, sc, None)
    _check_gemm(codes, sc, w, None, None, y)


def test_empty_calls():
    torch = torch_cuda()
    g = _g()
    codes, sc, _ = g.gptq_norm_quant(_rand((0, 64), 1, "f16"))
    assert codes.shape == (0, 64)
    w = torch.ones(16, 64, dtype=torch.int8, device="cuda:0")
    assert g.gptq_byte_gemm(codes, sc, w, None).shape == (0, 16)
    kc, ks = _pool(2, 16, 2, 32, 1)
    z = _rand((0, 2, 32), 1, "f16")
    g.gptq_kv_append(z, z, kc, kc.clone(), ks, ks.clone(), _ints([[0], [1]]), _ints([0, 0]))
    assert g.gptq_kv_attention(z, kc, kc, ks, ks, _ints([[0], [1]]), _ints([0, 0])).shape == (0, 2, 32)
    # a cache without pages: nothing is seen
    none, nos = torch.empty(0, 16, 2, 32, dtype=torch.int8, device="cuda:0"), torch.empty(0, 2, device="cuda:0")
    q = _rand((2, 4, 32), 1, "f16")
    out = g.gptq_kv_attention(q, none, none, nos, nos, _ints([[0], [1]]), _ints([5, 0]))
    torch.cuda.synchronize()
    assert torch.all(out == 0)


# -------------------------------------------------------------------------------------------- edges

@pytest.mark.parametrize("m,d,rows,stored", [((1 << 20) + 300, 16, 3, False), (2, 16, (1 << 18) + 70, True),
                                             (200, 32, (1 << 18) + 70, False)])
def test_byte_gemm_more_than_one_launch_takes(m, d, rows, stored):
    torch = torch_cuda()
    x, xs, w, ws, z = _gemm_inputs(m, d, rows, stored, seed=9)
    y = _g().gptq_byte_gemm(x, xs, w, ws, z, dtype=torch.float16)
    torch.cuda.synchronize()
    _check_gemm(x, xs, w, ws, z, y)


@pytest.mark.parametrize("tiles", [(2, 16), (4, 20), (8, 30), (8, 33), (17, 17)], ids=str)
def test_byte_gemm_rounds_of_tiles(tiles):
    """Less than a round of the CUs, parts of one, and a part past whole ones; the last tile of each edge is narrow."""
    torch = torch_cuda()
    m, rows = 256 * tiles[0] - 97, 256 * tiles[1] - 130
    for stored in (False, True):
        x, xs, w, ws, z = _gemm_inputs(m, 208, rows, stored, seed=10)
        y = _g().gptq_byte_gemm(x, xs, w, ws, z, dtype=torch.bfloat16)
        torch.cuda.synchronize()
        _check_gemm(x, xs, w, ws, z, y)


@pytest.mark.parametrize("m", [7, 300])
def test_byte_gemm_and_norm_in_a_graph(m):
    torch = torch_cuda()
    g = _g()
    x, r = _rand((m, 320), 1, "f16"), _rand((m, 320), 2, "f16")
    w = _rand((320,), 3, "f16")
    _, _, b, ws, z = _gemm_inputs(1, 320, 500, True)
    codes = torch.empty(m, 320, dtype=torch.int8, device="cuda:0")
    sc, y = torch.empty(m, device="cuda:0"), torch.empty(m, 500, device="cuda:0")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=side):
        g.gptq_norm_quant(x, r, w, sum_out=r, codes=codes, scales=sc)      # the residual in place
        g.gptq_byte_gemm(codes, sc, b, ws, z, y=y)
    for i in range(4):
        x.copy_(_rand((m, 320), 10 + i, "f16"))
        before = r.clone()
        gr.replay()
        torch.cuda.synchronize()
        _check_norm("f16", x, before, w, 1e-6, codes, sc, r)
        _check_gemm(codes, sc, b, ws, z, y)


@pytest.mark.parametrize("dtype", DT)
def test_norm_quant_more_rows_than_workgroups(dtype):
    """Rows in turn: zeros, infinities and rows beyond fp32's squares between ordinary ones, in one workgroup's list."""
    torch = torch_cuda()
    n, d = 9000, 520
    x = _rand((n, d), 11, dtype)
    x[5::7] = 0
    x[4096 + 3, 9] = float("inf")
    if dtype != "f16":
        x[2048 + 5] *= 1e25
        x[4096 + 5] *= 1e-25
    w = _rand((d,), 12, dtype)
    codes, scales, _ = _g().gptq_norm_quant(x, None, w)
    torch.cuda.synchronize()
    _check_norm(dtype, x, None, w, 1e-6, codes, scales, None)


def test_norm_quant_values_next_to_halves():
    """Quotients at and beside halves: ties go to the even code, neighbours to their own."""
    torch = torch_cuda()
    k = torch.arange(0, 127, device="cuda:0", dtype=torch.float64)
    half = (k + 0.5) / 127.0
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        row = torch.cat([half, -half, torch.ones(1, device="cuda:0", dtype=torch.float64)]) * 127.0 * 8
        x = torch.stack([row.to(dtype), torch.nextafter(row.float(), torch.zeros_like(row.float())).to(dtype),
                         torch.nextafter(row.float(), 2 * row.float()).to(dtype)])
        codes, scales, _ = _g().gptq_norm_quant(x)
        torch.cuda.synchronize()
        h = _np(x)
        want = np.rint(h * 127.0 / np.abs(h).max(1, keepdims=True))
        assert np.array_equal(codes.cpu().numpy(), want)


def test_kv_append_after_a_page_of_zeros():
    """Earlier tokens of scale zero: their codes stay zero when the scale begins."""
    torch = torch_cuda()
    zeros = torch.zeros(5, 2, 32, device="cuda:0")
    kc, vc, ks, vs = _run_append("f32", [5], [0], 2, 32, data=(zeros, zeros), table=np.array([[0]], np.int32), max_pages=1)
    assert torch.all(ks[0] == 0) and torch.all(kc[0, :5] == 0)
    k = _rand((3, 2, 32), 5, "f32")
    _g().gptq_kv_append(k, k, kc, vc, ks, vs, _ints([[0]]), _ints([5]))
    torch.cuda.synchronize()
    assert torch.all(kc[0, :5] == 0) and torch.all(ks[0] > 0)
    want = np.rint(_np(k) / _np(ks)[0][None, :, None])
    assert np.array_equal(kc[0, 5:8].cpu().numpy(), want)


def test_calls_between_devices_and_layouts_are_refused():
    torch = torch_cuda()
    g = _g()
    x = torch.ones(4, 32, dtype=torch.int8, device="cuda:0")
    with pytest.raises(ValueError):
        g.gptq_byte_gemm(x, None, x.cpu(), None)
    with pytest.raises(ValueError):
        g.gptq_byte_gemm(x, None, x.to(torch.uint8), None)          # codes without zeros
    with pytest.raises(ValueError):
        g.gptq_byte_gemm(x, None, x.t().contiguous().t(), None)     # columns not side by side
    with pytest.raises(ValueError):
        g.gptq_byte_gemm(x, torch.ones(3, device="cuda:0"), x, None)
    with pytest.raises(ValueError):
        g.gptq_norm_quant(torch.ones(2, 8, device="cuda:0"), torch.ones(2, 7, device="cuda:0"))
    kc, ks = _pool(2, 16, 2, 32, 1)
    q = _rand((1, 4, 32), 1, "f16")
    t, n = _ints([[0, 1]]), _ints([5])
    with pytest.raises(ValueError):
        g.gptq_kv_attention(q, kc, kc, ks, ks, t.long(), n)
    with pytest.raises(ValueError):
        g.gptq_kv_attention(q[:, :3], kc, kc, ks, ks, t, n)
    with pytest.raises(ValueError):
        g.gptq_kv_append(q[:, :1], q[:, :1], kc, kc.clone(), ks, ks.clone(), t, n)
    with pytest.raises(g.GPTQError):
        g.gptq_kv_append(q[:, :2], q[:, :2], kc, kc, ks, ks.clone(), t, n)   # keys and values in one place
