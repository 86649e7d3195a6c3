"""gptq_norm_rotate, gptq_attention and gptq_lora_gemm against their float64 oracle.

Tolerances count roundings. h is half a step of the type the values are stored in (torch.finfo.eps / 2) and
u = 2^-24 half a step of fp32:
* norm_rotate: one rounding of the result, h |out|, and fp32 arithmetic on the pair's two values: the sum of
  squares (at most 16 products per lane and six levels of a butterfly, halved by the root), the root, the
  quotient, the weight, cos and sin (2 u each beyond their angle's half step) and two products and a sum: fewer
  than 32 roundings of magnitude |y_a| + |y_b|.
* attention: each probability is rounded once to a 16-bit type before its product with v, h sum p |v|, and
  the result once, h |out|; a score's fp32 error d is at most (head_dim + 8) u times the sum of |q k| scale
  (or the score itself), which moves numerator and denominator by a factor 1 + d each; sums over keys add at
  most 64 u (fp32 sums run over 16-key steps and tiles, whose relative errors grow with the root of the
  length at most: 16 steps of 4096 keys).
* lora: sums of d and then rank products in fp32: at most (d + rank + 8) u of the sum of magnitudes.
Subnormal fp16 results add 2^-25.
"""

import numpy as np
import pytest

from gpu_util import torch_cuda
from oracle import attn_ref

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


# ------------------------------------------------------------------------------------- norm_rotate

def _check_rotate(dtype, q, k, qo, ko, qw, kw, pos, f, axis, norm, eps, inter):
    p = None if pos is None else np.atleast_2d(pos.cpu().numpy())
    ax = None if axis is None else axis.cpu().numpy()
    h = _half_step(dtype)
    for x, w, o in ((q, qw, qo), (k, kw, ko)):
        if x is None:
            continue
        want, mag = attn_ref.norm_rotate(_np(x), _np(w), p, _np(f), ax, norm, eps, inter)
        err = np.abs(_np(o) - want)
        bound = h * np.abs(want) + 32 * U * mag + 2.0 ** -25 * (dtype == "f16")
        assert np.all(err <= bound), float(np.max(err / bound))


ROT = [   # n, hq, hk, dh, rd, axes, interleaved, norm
    (1, 1, 0, 2, 2, 1, False, True), (1, 4, 4, 128, 128, 1, False, True), (5, 32, 8, 128, 128, 1, False, True),
    (3, 3, 1, 64, 32, 1, True, True), (17, 2, 2, 80, 80, 3, False, True), (7, 5, 1, 72, 36, 2, True, False),
    (9, 2, 1, 7, 4, 1, False, True), (9, 2, 1, 7, 4, 1, True, True), (4, 1, 1, 1, 0, 1, False, True),
    (33, 7, 7, 256, 256, 1, True, True), (6, 2, 1, 1024, 1024, 1, False, True), (6, 1, 1, 1023, 510, 4, True, True),
    (1300, 2, 1, 96, 48, 1, False, True), (2100, 8, 8, 128, 64, 1, True, True), (40, 1, 0, 1000, 2, 1, False, False),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,hq,hk,dh,rd,axes,inter,norm", ROT)
def test_norm_rotate(n, hq, hk, dh, rd, axes, inter, norm, dtype):
    torch = torch_cuda()
    print(f"norm_rotate {(n, hq, hk, dh, rd, axes, inter, norm, dtype)}", flush=True)
    q = _rand((n, hq, dh), 1, dtype, 2.0)
    k = _rand((n, hk, dh), 2, dtype, 0.5) if hk else None
    qw = _rand((dh,), 3, "f32") if norm else None
    kw = _rand((dh,), 4, "f32") if norm and hk and n % 2 else None
    r = np.random.default_rng(5)
    f = pos = axis = None
    if rd:
        f = torch.from_numpy((10000.0 ** (-np.arange(rd // 2) * 2 / rd)).astype(np.float32)).cuda()
        pos = _ints(r.integers(-5, 1 << 20, (axes, n)))
        axis = _ints(r.integers(-1, axes + 1, rd // 2)) if axes > 1 else None
    qo, ko = _g().gptq_norm_rotate(q, k, pos, f, axis, qw, kw, norm=norm, eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    assert (ko is None) == (k is None)
    _check_rotate(dtype, q, k, qo, ko, qw, kw, pos, f, axis, norm, 1e-5, inter)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_norm_rotate_views_and_in_place(dtype, shift):
    """Column ranges of one fused projection (at odd offsets too), head-major arrays, in place, and columns
    beside them left as they were."""
    torch = torch_cuda()
    n, hq, hk, dh = 37, 6, 2, 64
    base = _rand((n, shift + (hq + 2 * hk) * dh), 7, dtype)
    kept = base.clone()
    fused = base[:, shift:].unflatten(1, (hq + 2 * hk, dh))
    q, k = fused[:, :hq], fused[:, hq:hq + hk]
    f = torch.rand(dh // 2, device="cuda:0")
    pos = _ints(np.arange(n))
    q0, k0 = q.clone(), k.clone()
    qo = torch.empty(hq, n, dh, dtype=q.dtype, device="cuda:0").transpose(0, 1)     # head-major output
    _, ko = _g().gptq_norm_rotate(q, k, pos, f, q_out=qo)
    torch.cuda.synchronize()
    _check_rotate(dtype, q0, k0, qo, ko, None, None, pos, f, None, True, 1e-6, False)
    _g().gptq_norm_rotate(q, k, pos, f, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko)
    edge = shift + (hq + hk) * dh
    assert torch.equal(base[:, :shift], kept[:, :shift]) and torch.equal(base[:, edge:], kept[:, edge:])


def test_norm_rotate_special_values():
    """A head of zeros stays zero, eps keeps tiny heads small, and an infinity or NaN stays in its own head."""
    torch = torch_cuda()
    q = _rand((4, 3, 32), 8, "f32")
    q[0, 0] = 0
    q[1, 1] = 1e-20
    q[2, 2, 5] = float("inf")
    q[3, 0, 7] = float("nan")
    f = torch.rand(16, device="cuda:0")
    o, _ = _g().gptq_norm_rotate(q, None, _ints([1, 2, 3, 4]), f)
    torch.cuda.synchronize()
    o = o.cpu()
    assert torch.all(o[0, 0] == 0) and o[1, 1].abs().max() < 1e-16
    bad = ~torch.isfinite(o)
    assert bad[2, 2].any() and bad[3, 0].all()
    bad[2, 2] = bad[3, 0] = False
    assert not bad.any()


# --------------------------------------------------------------------------------------- attention

def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _check_attention(dtype, q, k, v, out, seqs, scale, **kw):
    want, mag, spread = attn_ref.attention(_np(q), _np(k), _np(v), seqs, scale, **kw)
    got = _np(out)
    dh = q.shape[2]
    p_step = 0.0 if dtype == "f32" else _half_step(dtype)
    bound = _half_step(dtype) * np.abs(want) + (p_step + (2 * (dh + 8) * spread + 64) * U) * mag \
        + 2.0 ** -25 * (dtype == "f16")
    err = np.abs(got - want)
    covered = np.zeros(len(got), dtype=bool)
    for q0, q1, _, _ in seqs:
        covered[q0:q1] = True
    ok = err <= bound
    assert np.all(ok[covered]), (float(np.nanmax(np.where(bound > 0, err / np.where(bound > 0, bound, 1), err))),
                                 int(np.count_nonzero(~ok[covered])), np.argwhere(~ok)[:4].tolist())


def _run_attention(dtype, hq, hk, dh, lens, seed=1, scale=None, causal=True, softcap=0.0, bias=False, docs=None,
                   prefix=None, work=True, qs=1.5):
    torch = torch_cuda()
    lq, lk = [a for a, _ in lens], [b for _, b in lens]
    q0, k0 = _starts(lq), _starts(lk)
    q = _rand((q0[-1], hq, dh), seed, dtype, qs)
    k, v = _rand((k0[-1], hk, dh), seed + 1, dtype), _rand((k0[-1], hk, dh), seed + 2, dtype)
    slopes = torch.tensor([2.0 ** (-h - 1) for h in range(hq)], device="cuda:0") if bias else None
    r = np.random.default_rng(seed + 3)
    qd = kd = None
    if docs:
        kd = np.sort(r.integers(0, docs, k0[-1])) if docs > 0 else r.integers(-1, -docs, k0[-1])
        qd = np.concatenate([kd[b - min(a, b - e):b] if a <= b - e else
                             np.concatenate([np.full(a - (b - e), -1), kd[e:b]])
                             for a, e, b in zip(lq, k0[:-1], k0[1:])]) if len(lens) else kd
    scale = scale or dh ** -0.5
    out = torch.full((q0[-1], hq, dh), 7.0, dtype=q.dtype, device="cuda:0")
    print(f"attention {(dtype, hq, hk, dh, lens[:4], causal, softcap, bias, docs, prefix, work)}", flush=True)
    _g().gptq_attention(q, k, v, scale, causal, q_start=_ints(q0), kv_start=_ints(k0), softcap=softcap, slopes=slopes,
                        q_doc=None if qd is None else _ints(qd), kv_doc=None if kd is None else _ints(kd),
                        prefix=None if prefix is None else _ints(prefix), out=out,
                        work=None if work else torch.empty(0, dtype=torch.uint8, device="cuda:0"))
    torch.cuda.synchronize()
    seqs = list(zip(q0[:-1], q0[1:], k0[:-1], k0[1:]))
    _check_attention(dtype, q, k, v, out, seqs, scale, causal=causal, softcap=softcap, slopes=_np(slopes), q_doc=qd,
                     kv_doc=kd, prefix=prefix)
    return out


LENS = {
    "one": [(1, 1)], "two": [(2, 2)], "edge63": [(63, 63)], "edge64": [(64, 64)], "edge65": [(65, 65)],
    "uneven": [(5, 5), (0, 0), (130, 130), (1, 1), (33, 33)], "long": [(257, 257)],
    "tokens": [(1, 300), (1, 1), (1, 64), (1, 129)], "chunk": [(7, 200), (40, 41), (3, 3)],
    "nokeys": [(3, 0), (4, 4)], "noqueries": [(0, 5), (2, 9)], "more_queries": [(9, 4), (70, 2)],
}


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lens", list(LENS), ids=str)
def test_attention_lengths(lens, dtype):
    _run_attention(dtype, 4, 2, 64, LENS[lens])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("dh", [1, 7, 16, 20, 32, 48, 72, 80, 96, 112, 128, 136, 192, 200, 256, 260, 1024])
def test_attention_head_widths(dh, dtype):
    _run_attention(dtype, 2, 1, dh, [(70, 70), (1, 90)])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (7, 1), (6, 2), (40, 8), (33, 1), (130, 1)])
def test_attention_shared_heads(hq, hk, dtype):
    _run_attention(dtype, hq, hk, 32, [(35, 35), (1, 70), (2, 3)])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kw", [
    dict(causal=False), dict(softcap=2.0), dict(softcap=50.0, causal=False), dict(bias=True),
    dict(bias=True, causal=False), dict(docs=3), dict(docs=-3), dict(docs=-3, causal=False),
    dict(docs=4, softcap=5.0, bias=True), dict(prefix=[0, 150, 20]), dict(prefix=[9, 500, -4], bias=True),
    dict(prefix=[5, 5, 5], docs=2, softcap=1.0), dict(prefix=[5, 5, 5], causal=False), dict(scale=-0.3),
    dict(softcap=256.0), dict(softcap=5000.0), dict(softcap=1e7, bias=True), dict(softcap=1e-6),
    dict(scale=-0.3, softcap=3.0), dict(scale=-0.3, bias=True), dict(docs=70), dict(docs=-70, causal=False),
], ids=str)
def test_attention_masks(kw, dtype):
    _run_attention(dtype, 4, 2, 64, [(9, 9), (200, 200), (66, 140)], **kw)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("work", [True, False])
def test_attention_long_caches(work, dtype):
    """Few queries against long key ranges: split across workgroups with the workspace, whole without it."""
    _run_attention(dtype, 8, 2, 128, [(1, 9001), (2, 700), (1, 1), (5, 4097)], work=work)
    _run_attention(dtype, 4, 4, 80, [(1, 5000)], docs=9, softcap=20.0, work=work)
    _run_attention(dtype, 2, 1, 64, [(3, 3000), (1, 0)], bias=True, causal=False, work=work)


@pytest.mark.parametrize("dtype", DT)
def test_attention_documents_over_many_blocks(dtype):
    """Keys beyond one scan of 64 tiles, documents that skip whole scans, recur and end inside tiles."""
    n = 9300
    r = np.random.default_rng(2)
    torch = torch_cuda()
    h, dh = 1, 32
    q, k, v = (_rand((n, h, dh), s, dtype) for s in (1, 2, 3))
    doc = np.repeat(np.arange(6), [3000, 70, 1, 4300, 1500, 429])
    doc[100:130] = 4                 # an early piece of a late document
    doc[8000:8040] = -1
    d = _ints(doc)
    rows = np.unique(np.concatenate([r.integers(0, n, 60), [0, 99, 100, 129, 130, 2999, 3000, 3070, 3071, 7999, 8000,
                                                            8039, 8040, 8870, 9299]]))
    out = _g().gptq_attention(q, k, v, q_doc=d, kv_doc=d)
    torch.cuda.synchronize()
    got = _np(out)[rows]
    # the same rows one by one: a sequence of the first i + 1 keys, whose last token is the row
    want, mag, spread = attn_ref.attention(np.repeat(_np(q)[rows], 1, 0), np.concatenate([_np(k)[:i + 1] for i in rows]),
                                           np.concatenate([_np(v)[:i + 1] for i in rows]),
                                           [(j, j + 1, *(int(x) for x in e)) for j, e in enumerate(
                                               zip(_starts(rows + 1)[:-1], _starts(rows + 1)[1:]))],
                                           dh ** -0.5, q_doc=doc[rows], kv_doc=np.concatenate([doc[:i + 1] for i in rows]))
    p_step = 0.0 if dtype == "f32" else _half_step(dtype)
    bound = _half_step(dtype) * np.abs(want) + (p_step + (2 * (dh + 8) * spread + 64) * U) * mag + 2.0 ** -25
    assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("dh", [64, 128, 256])
def test_attention_nan_everywhere(dh, dtype):
    """All-NaN keys or values give NaN in every row that sees one, zeros in rows that see none."""
    torch = torch_cuda()
    n = 70
    q, k, v = (_rand((n, 2, dh), s, dtype) for s in (1, 2, 3))
    doc = np.zeros(n, dtype=np.int32)
    doc[:5] = -1
    for bad in (k, v):
        kk, vv = (torch.full_like(t, float("nan")) if t is bad else t for t in (k, v))
        o = _g().gptq_attention(q, kk, vv, q_doc=_ints(doc), kv_doc=_ints(doc))
        torch.cuda.synchronize()
        assert torch.all(o[:5] == 0) and torch.isnan(o[5:]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_attention_infinite_scores_in_split_ranges(dtype):
    """An infinity in one value that a long range sees shows in its column alone, split or not."""
    torch = torch_cuda()
    q, k, v = _rand((1, 2, 64), 1, dtype), _rand((6000, 1, 64), 2, dtype), _rand((6000, 1, 64), 3, dtype)
    v[4000, 0, 9] = float("inf")
    for work in (None, torch.empty(0, dtype=torch.uint8, device="cuda:0")):
        o = _g().gptq_attention(q, k, v, work=work)
        torch.cuda.synchronize()
        bad = ~torch.isfinite(o)
        assert torch.all(o[:, :, 9] == float("inf")) and bad.sum() == 2


@pytest.mark.parametrize("dtype", DT)
def test_attention_many_sequences(dtype):
    r = np.random.default_rng(3)
    lens = [(int(a), int(a)) for a in r.integers(0, 12, 300)]
    _run_attention(dtype, 2, 2, 32, lens)
    lens = [(int(a), int(a + b)) for a, b in zip(r.integers(0, 60, 150), r.integers(0, 40, 150))]
    _run_attention(dtype, 4, 1, 32, lens, docs=5, prefix=[3] * 150)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_large_scores(dtype):
    """Scores of hundreds: the running maximum keeps every exponent at or below zero."""
    _run_attention(dtype, 2, 2, 64, [(150, 150)], qs=300.0)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("case", ["causal", "documents", "padding", "last"])
def test_attention_masked_places_hold_anything(case, dtype):
    """Infinities and NaN in the keys and values that a query does not see leave its output bit for bit."""
    torch = torch_cuda()
    n, h, dh = 150, 2, 64
    q, k, v = (_rand((n, h, dh), s, dtype) for s in (1, 2, 3))
    doc = np.zeros(n, dtype=np.int32)
    kw = dict(causal=True)
    if case == "causal":
        bad, rows = [140], slice(0, 140)
    elif case == "documents":
        doc[70:] = 1
        bad, rows, kw = [3, 20, 69], slice(70, n), dict(causal=False)
    elif case == "padding":
        doc[100:] = -1
        bad, rows, kw = [100, 120, 149], slice(0, n), dict(causal=False)
    else:
        bad, rows = [149], slice(0, 149)
    d = _ints(doc)
    clean = _g().gptq_attention(q, k, v, q_doc=d, kv_doc=d, **kw)
    k2, v2 = k.clone(), v.clone()
    for i, b in enumerate(bad):
        k2[b, :, i % 3] = [float("inf"), float("nan"), -float("inf")][i % 3]
        v2[b, :, (i + 1) % 5] = [float("nan"), float("inf"), float("nan")][i % 3]
    got = _g().gptq_attention(q, k2, v2, q_doc=d, kv_doc=d, **kw)
    torch.cuda.synchronize()
    h_ = _half_step(dtype)
    a, b = _np(clean)[rows], _np(got)[rows]
    # the same values up to the roundings of either evaluation
    mag = np.max(np.abs(_np(v)))
    p_step = 0.0 if dtype == "f32" else h_
    assert np.all(np.isfinite(b))
    assert np.all(np.abs(a - b) <= 2 * (h_ * np.abs(a) + (p_step + 2 * 72 * 16 * U) * mag))
    if case == "padding":
        assert np.all(b[100:] == 0)


def test_attention_nan_that_is_seen_shows():
    torch = torch_cuda()
    q, k, v = (_rand((100, 1, 64), s, "f16") for s in (1, 2, 3))
    v[50, 0, 3] = float("nan")
    o = _g().gptq_attention(q, k, v)
    torch.cuda.synchronize()
    bad = torch.isnan(o).cpu()
    assert bad[50:, 0, 3].all() and not bad[:50].any() and not bad[:, :, 4:].any() and not bad[:, :, :3].any()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_attention_views(dtype):
    """Column ranges of a fused projection at odd offsets, head-major tensors, heads shared by stride 0, an
    output inside a wider array; rows and columns that are not the output's stay."""
    torch = torch_cuda()
    n, h, dh = 90, 3, 40
    seqs = [(0, n, 0, n)]
    for shift in (0, 1, 8):
        f = _rand((n, shift + 3 * h * dh), 11 + shift, dtype)[:, shift:].unflatten(1, (3 * h, dh))
        q, k, v = f[:, :h], f[:, h:2 * h], f[:, 2 * h:]
        wide = torch.full((n + 2, h + 1, dh + shift), 3.0, dtype=q.dtype, device="cuda:0")
        out = wide[1:n + 1, :h, :dh]
        _g().gptq_attention(q, k, v, out=out)
        torch.cuda.synchronize()
        _check_attention(dtype, q, k, v, out, seqs, dh ** -0.5)
        rest = wide.clone()
        rest[1:n + 1, :h, :dh] = 3.0
        assert torch.all(rest == 3.0)
    qh, kh, vh = (_rand((h, n, dh), s, dtype).transpose(0, 1) for s in (20, 21, 22))
    _check_attention(dtype, qh, kh, vh, _g().gptq_attention(qh, kh, vh), seqs, dh ** -0.5)
    kb = kh[:, :1].expand(n, h, dh)
    _check_attention(dtype, qh, kb, vh, _g().gptq_attention(qh, kb, vh), seqs, dh ** -0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_rows_behind_the_last_sequence(dtype):
    torch = torch_cuda()
    q, k, v = (_rand((100, 2, 64), s, dtype) for s in (1, 2, 3))
    out = torch.full_like(q, 5.0)
    _g().gptq_attention(q, k, v, q_start=_ints([4, 30, 77]), kv_start=_ints([0, 26, 90]), out=out)
    torch.cuda.synchronize()
    assert torch.all(out[:4] == 5.0) and torch.all(out[77:] == 5.0)
    _check_attention(dtype, q, k, v, out, [(4, 30, 0, 26), (30, 77, 26, 90)], 64 ** -0.5)


def test_attention_offsets_are_clamped():
    """Offsets beyond the arrays end at their last row; the result is that of the clamped ranges."""
    torch = torch_cuda()
    q, k, v = (_rand((60, 2, 64), s, "f16") for s in (1, 2, 3))
    got = _g().gptq_attention(q, k, v, q_start=_ints([-9, 40, 1 << 30]), kv_start=_ints([-5, 40, 1 << 30]))
    want = _g().gptq_attention(q, k, v, q_start=_ints([0, 40, 60]), kv_start=_ints([0, 40, 60]))
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_attention_equal_ranges_without_offsets():
    torch = torch_cuda()
    q, k, v = (_rand((96, 2, 64), s, "bf16") for s in (1, 2, 3))
    a = _g().gptq_attention(q, k, v, seqs=3)
    b = _g().gptq_attention(q, k, v, q_start=_ints([0, 32, 64, 96]), kv_start=_ints([0, 32, 64, 96]))
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_attention_offsets_past_32_bits():
    """A cache of more than 2^31 elements: queries that match one key each get its value."""
    torch = torch_cuda()
    n, hk, dh = 2_200_003, 8, 128
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(1)
    k = torch.randn(n, hk, dh, generator=gen, device="cuda:0", dtype=torch.bfloat16)
    v = torch.randn(n, hk, dh, generator=gen, device="cuda:0", dtype=torch.bfloat16)
    at = [10, 2 ** 31 // (hk * dh) + 3, n - 1]
    q = k[at].repeat_interleave(2, 1).contiguous() * 4
    for work in (None, torch.empty(0, dtype=torch.uint8, device="cuda:0")):
        o = _g().gptq_attention(q, k, v, causal=False, work=work)
        torch.cuda.synchronize()
        # each match's score is 4 |k|^2 / sqrt(dh), about 45, against about 4 for the others: e^-41 times their number
        assert torch.all((o - v[at].repeat_interleave(2, 1)).abs().float() <= 2 ** -6 * (1 + o.abs().float()))


def test_norm_rotate_large_sizes():
    """More than 2^31 elements, and more tokens than one launch takes: rows equal those of small calls."""
    torch = torch_cuda()
    f = torch.rand(32, device="cuda:0")
    for n, h, dh in ((270_001, 64, 128), ((1 << 22) + 77, 1, 64)):
        q = torch.empty(n, h, dh, dtype=torch.bfloat16, device="cuda:0").uniform_(-1, 1)
        pos = torch.arange(n, dtype=torch.int32, device="cuda:0")
        o, _ = _g().gptq_norm_rotate(q, None, pos, f)
        for a in (0, n // 2, min(n, 1 << 22) - 9, n - 40):
            p, _ = _g().gptq_norm_rotate(q[a:a + 40], None, pos[a:a + 40].contiguous(), f)
            torch.cuda.synchronize()
            assert torch.equal(o[a:a + 40], p)


# -------------------------------------------------------------------------------------------- lora

LORA = [  # m, d, rows, adapters, rank
    (1, 8, 8, 1, 1), (1, 4096, 4096, 3, 16), (3, 100, 37, 4, 5), (16, 256, 512, 2, 64), (17, 1000, 1000, 40, 8),
    (65, 129, 63, 3, 33), (130, 512, 300, 7, 256), (257, 64, 128, 1, 16), (700, 96, 100, 5, 24), (5, 1, 1, 2, 2),
    (40, 11008, 64, 3, 12),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("m,d,rows,na,r", LORA)
def test_lora(m, d, rows, na, r, dtype):
    torch = torch_cuda()
    print(f"lora {(m, d, rows, na, r, dtype)}", flush=True)
    x, A, B = _rand((m, d), 1, dtype), _rand((na, r, d), 2, dtype, d ** -0.5), _rand((na, rows, r), 3, dtype, 0.3)
    rr = np.random.default_rng(4)
    idx = rr.integers(-1, na + 1, m)
    ranks = rr.integers(-1, r + 2, na)
    s = torch.from_numpy(rr.uniform(-2, 2, na).astype(np.float32)).cuda()
    base = _rand((m, rows), 5, "f32")
    for kw in (dict(base=base, scales=s), dict(ranks=_ints(ranks)), dict(base=base, scales=s, ranks=_ints(ranks))):
        y = _g().gptq_lora_gemm(x, A, B, _ints(idx), **kw)
        torch.cuda.synchronize()
        want, mag = attn_ref.lora(_np(x), _np(A), _np(B), idx, _np(kw.get("scales")),
                                  ranks if "ranks" in kw else None, _np(kw.get("base")))
        err = np.abs(_np(y) - want)
        assert np.all(err <= (d + r + 8) * U * mag), float(np.max(err))
        none = (idx < 0) | (idx >= na)
        assert np.array_equal(_np(y)[none], _np(kw["base"])[none] if "base" in kw else np.zeros_like(want[none]))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("runs", [False, True], ids=["mixed", "runs"])
@pytest.mark.parametrize("m,d,rows,na,r", [(8, 4096, 4100, 5, 16), (200, 1024, 1030, 12, 20), (1100, 512, 700, 3, 64)])
def test_lora_exact_on_whole_numbers(m, d, rows, na, r, runs, dtype):
    """Small whole numbers make every product and sum exact in fp32: the result is equal, not close."""
    torch = torch_cuda()
    rr = np.random.default_rng(6)
    x, A, B = rr.integers(-2, 3, (m, d)), rr.integers(-1, 2, (na, r, d)), rr.integers(-2, 3, (na, rows, r))
    idx = rr.integers(0, na, m)
    if runs:
        idx = np.sort(idx)
    to = lambda a: torch.from_numpy(a.astype(np.float32)).to(_dtype(dtype)).cuda()   # noqa: E731
    y = _g().gptq_lora_gemm(to(x), to(A), to(B), _ints(idx))
    torch.cuda.synchronize()
    want = attn_ref.lora(x, A, B, idx)[0]
    assert np.max(np.abs(want)) < 2 ** 24
    assert np.array_equal(_np(y), want)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_lora_views_in_place_and_unused_places(dtype):
    """Strided x, base and y, y added in place, unused ranks and adapters holding NaN, columns beside y kept."""
    torch = torch_cuda()
    m, d, rows, na, r = 33, 200, 90, 3, 12
    x = _rand((m, d + 3), 1, dtype)[:, 3:]
    A, B = _rand((na, r, d), 2, dtype, 0.1), _rand((na, rows, r), 3, dtype)
    A[:, 7:], B[:, :, 7:] = float("nan"), float("nan")
    A[1], B[1] = float("inf"), float("nan")
    idx = np.where(np.arange(m) % 3 == 1, -1, np.arange(m) % 3)
    wide = _rand((m, rows + 5), 4, "f32")
    kept = wide.clone()
    y = wide[:, 2:2 + rows]
    base = y.clone()
    _g().gptq_lora_gemm(x, A, B, _ints(idx), ranks=_ints([7, 7, 7]), base=y, y=y)
    torch.cuda.synchronize()
    want, mag = attn_ref.lora(_np(x), np.nan_to_num(_np(A), posinf=0), np.nan_to_num(_np(B)), idx, None, [7, 7, 7],
                              _np(base))
    assert np.all(np.abs(_np(y) - want) <= (d + r + 8) * U * mag)
    assert torch.equal(wide[:, :2], kept[:, :2]) and torch.equal(wide[:, 2 + rows:], kept[:, 2 + rows:])


def test_lora_nan_stays_with_its_rows():
    """NaN in one row of x, or in one adapter, reaches the rows that name it and no others, in mixed tiles."""
    torch = torch_cuda()
    for m in (20, 600):
        x, A, B = _rand((m, 64), 1, "bf16"), _rand((3, 16, 64), 2, "bf16"), _rand((3, 40, 16), 3, "bf16")
        x[7], A[2] = float("nan"), float("nan")
        idx = np.arange(m) % 4 - 1
        idx[7] = 0
        y = _g().gptq_lora_gemm(x, A, B, _ints(idx))
        torch.cuda.synchronize()
        bad = torch.isnan(y).any(1).cpu().numpy()
        assert np.array_equal(bad, (idx == 2) | (np.arange(m) == 7))


def test_lora_more_rows_than_one_piece():
    """Rows beyond 2^19 go in pieces that share the workspace: they equal a small call's."""
    torch = torch_cuda()
    m, d, rows, na, r = (1 << 19) + 300, 16, 24, 3, 4
    rr = np.random.default_rng(1)
    to = lambda *s: torch.from_numpy(rr.integers(-2, 3, s).astype(np.float32)).half().cuda()   # noqa: E731
    x, A, B = to(m, d), to(na, r, d), to(na, rows, r)
    idx = _ints(rr.integers(-1, na, m))
    y = _g().gptq_lora_gemm(x, A, B, idx)
    for a in (0, (1 << 19) - 30, m - 60):
        p = _g().gptq_lora_gemm(x[a:a + 60], A, B, idx[a:a + 60].contiguous())
        torch.cuda.synchronize()
        assert torch.equal(y[a:a + 60], p)


def test_lora_without_adapters_copies_the_base():
    torch = torch_cuda()
    x, base = _rand((5, 16), 1, "f16"), _rand((5, 24), 2, "f32")
    y = _g().gptq_lora_gemm(x, x.new_empty(0, 4, 16), x.new_empty(0, 24, 4), _ints([0, 1, -1, 2, 3]), base=base)
    torch.cuda.synchronize()
    assert torch.equal(y, base)


# --------------------------------------------------------------------------------- streams, graphs

def _three(s):
    """norm + rotation, attention and an adapter on one stream, as a layer uses them."""
    g = _g()
    q, k = g.gptq_norm_rotate(s["q"], s["k"], s["pos"], s["f"], q_out=s["qo"], k_out=s["ko"], stream=s.get("stream"))
    o = g.gptq_attention(q, k, s["v"], q_start=s["start"], kv_start=s["start"], out=s["o"], work=s["aw"],
                         stream=s.get("stream"))
    g.gptq_lora_gemm(o.flatten(1), s["A"], s["B"], s["idx"], base=s["base"], y=s["y"], work=s["lw"],
                     stream=s.get("stream"))


def _state(dtype="f16", n=200, hq=4, hk=2, dh=64):
    torch = torch_cuda()
    g = _g()
    s = dict(q=_rand((n, hq, dh), 1, dtype), k=_rand((n, hk, dh), 2, dtype), v=_rand((n, hk, dh), 3, dtype),
             pos=_ints(np.arange(n)), f=torch.rand(dh // 2, device="cuda:0"), start=_ints([0, n // 3, n]),
             A=_rand((2, 8, hq * dh), 4, dtype, 0.1), B=_rand((2, 50, 8), 5, dtype), idx=_ints(np.arange(n) % 3 - 1),
             base=_rand((n, 50), 6, "f32"))
    s.update(qo=torch.empty_like(s["q"]), ko=torch.empty_like(s["k"]), o=torch.empty_like(s["q"]),
             y=torch.empty(n, 50, device="cuda:0"))
    s["aw"] = torch.empty(max(1, g.gptq_attention_workspace_bytes(s["q"], s["k"], 2)), dtype=torch.uint8,
                          device="cuda:0")
    s["lw"] = torch.empty(g.gptq_lora_workspace_bytes(n, hq * dh, 50, 2, 8), dtype=torch.uint8, device="cuda:0")
    return s


@pytest.mark.parametrize("n", [2, 200])
def test_captured_graph_replays(n):
    """The three calls captured once and replayed on new inputs, with eager work between the replays."""
    torch = torch_cuda()
    s = _state(n=n)
    _three(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        _three(s)
    for r in range(4):
        for name in ("q", "k", "v"):
            s[name].copy_(_rand(s[name].shape, 100 + 10 * r + ord(name), "f16"))
        s["y"].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got, o = s["y"].clone(), s["o"].clone()
        s["y"].fill_(float("nan"))
        _three(s)
        torch.cuda.synchronize()
        assert torch.equal(got, s["y"]) and torch.equal(o, s["o"])


def test_first_call_inside_a_capture():
    """A head width and type that no call has used yet, captured at once."""
    torch = torch_cuda()
    q, k, v = (_rand((300, 4, 176), s, "bf16") for s in (1, 2, 3))
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.05], device="cuda:0")
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _g().gptq_attention(q, k, v, slopes=slopes, softcap=4.0, out=out)
    for r in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, _g().gptq_attention(q, k, v, slopes=slopes, softcap=4.0))
        torch.cuda.synchronize()


def test_two_calls_at_once():
    """Calls on two streams with workspaces of their own give what each gives alone."""
    torch = torch_cuda()
    a, b = _state(n=300), _state("bf16", n=2)
    want = []
    for s in (a, b):
        _three(s)
        torch.cuda.synchronize()
        want.append((s["o"].clone(), s["y"].clone()))
        s["o"].zero_()
        s["y"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s, st in zip((a, b), streams):
            s["stream"] = st
            _three(s)
    torch.cuda.synchronize()
    for s, (o, y) in zip((a, b), want):
        assert torch.equal(s["o"], o) and torch.equal(s["y"], y)


def test_named_stream_matches_the_current_one():
    torch = torch_cuda()
    s = _state()
    _three(s)
    torch.cuda.synchronize()
    want = s["y"].clone()
    s["y"].fill_(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s["stream"] = side
    s["aw"] = s["lw"] = None          # made by the calls, on the named stream
    _three(s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(want, s["y"])


def test_results_do_not_change_between_runs():
    torch = torch_cuda()
    s = _state(n=500)
    _three(s)
    torch.cuda.synchronize()
    first = s["y"].clone()
    for _ in range(5):
        s["y"].fill_(0)
        _three(s)
        torch.cuda.synchronize()
        assert torch.equal(first, s["y"])
