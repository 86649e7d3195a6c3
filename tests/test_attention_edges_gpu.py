"""Edges of gptq_norm_rotate, gptq_attention and gptq_lora_gemm against their float64 oracle: inputs that are not
finite beside ranks that are not used, infinities in every range of a split key axis, values near the largest fp32
holds and heads whose squares leave fp32's range.

Tolerances are those of test_attention_gpu.py, which count roundings; what a case adds is written beside it.
"""

import numpy as np
import pytest

from gpu_util import torch_cuda
from oracle import attn_ref
from test_attention_gpu import DT, U, _check_attention, _check_rotate, _dtype, _g, _ints, _np, _rand, _starts

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------------------------------- lora

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rank,ranks", [(16, [0, 1, 16, 7]), (1, None), (20, [0, 1, 20, 7]), (20, None),
                                        (40, [0, 1, 40, 33]), (64, [0, 5, 64, 17])], ids=str)
@pytest.mark.parametrize("m", [1, 20, 300, 1100])
def test_lora_infinite_inputs_beside_unused_ranks(m, rank, ranks, dtype):
    """A row of x that holds an infinity or NaN gives what the definition gives at the ranks in use: +-inf where all
    of them agree, the base where there are none."""
    torch = torch_cuda()
    print(f"lora {(m, rank, ranks, dtype)}", flush=True)
    d, rows, na = 200, 90, 4
    x, A = _rand((m, d), 1, dtype), _rand((na, rank, d), 2, dtype, d ** -0.5)
    B = _rand((na, rows, rank), 3, dtype, 0.3).abs() + 0.01
    A[:, :, 9] = A[:, :, 9].abs() + 0.01                 # every rank gets an infinity's own sign
    for i in range(m):
        if i % 5 < 3:
            x[i, 9] = [float("inf"), -float("inf"), float("nan")][i % 5]
    base = _rand((m, rows), 5, "f32")
    idx = np.arange(m) // 5 % (na + 1)                    # each kind of row with each adapter, and with none
    y = _g().gptq_lora_gemm(x, A, B, _ints(idx), ranks=None if ranks is None else _ints(ranks), base=base)
    torch.cuda.synchronize()
    want, mag = attn_ref.lora(_np(x), _np(A), _np(B), idx, None, ranks, _np(base))
    got, fin = _np(y), np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin], equal_nan=True)
    assert np.all(np.abs(got[fin] - want[fin]) <= (d + rank + 8) * U * mag[fin])
    none = (idx >= na) if ranks is None else (idx >= na) | (idx == 0)
    assert np.array_equal(got[none], _np(base)[none])


# --------------------------------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [600, 2000, 4200, 6000])
def test_attention_infinity_in_each_split_range(n, dtype):
    """One infinite value anywhere in a long range shows in its column alone, whatever number of ranges the keys are
    split into (2, 7, 16 and 23 here)."""
    torch = torch_cuda()
    q, k, v = _rand((1, 2, 64), 1, dtype), _rand((n, 1, 64), 2, dtype), _rand((n, 1, 64), 3, dtype)
    for at in range(60, n, 125):
        w = v.clone()
        w[at, 0, 9] = -float("inf")
        o = _g().gptq_attention(q, k, w)
        torch.cuda.synchronize()
        bad = ~torch.isfinite(o)
        assert torch.all(o[:, :, 9] == -float("inf")) and bad.sum() == 2, at


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dh", [64, 128, 300])
@pytest.mark.parametrize("size", [1e33, 3e34, 1e36, 3e38])
def test_attention_values_near_the_largest(size, dh, dtype):
    """Weighted sums of finite values may pass fp32's range; their averages do not. Of one sign and of both, in one
    range of keys and in several. An average over n keys that is kept key by key errs by u of itself at each, which
    the keys after it dilute: n / 2 u for even weights, and n / 32 u for four roundings each 64 keys. 1200 keys make
    638 u; the bound's (2 (dh + 8) spread + 64) u is above 784 u, as the spread is above 5 here."""
    torch = torch_cuda()
    r = np.random.default_rng(8)
    for both in (False, True):
        for lens in ([(300, 300)], [(1, 1200)], [(2, 700), (3, 800)]):
            lq, lk = [a for a, _ in lens], [b for _, b in lens]
            q0, k0 = _starts(lq), _starts(lk)
            q, k = _rand((q0[-1], 2, dh), 1, dtype, 1.5), _rand((k0[-1], 1, dh), 2, dtype)
            val = r.uniform(0.3, 1.0, (k0[-1], 1, dh)) * (r.choice([-1.0, 1.0], (k0[-1], 1, dh)) if both else 1.0)
            v = torch.from_numpy(val * size).to(_dtype(dtype)).cuda()
            for work in (None, torch.empty(0, dtype=torch.uint8, device="cuda:0")):
                print(f"values {(size, dh, dtype, both, lens, work is None)}", flush=True)
                o = _g().gptq_attention(q, k, v, q_start=_ints(q0), kv_start=_ints(k0), work=work)
                torch.cuda.synchronize()
                assert torch.isfinite(o).all()
                # compared in units of the size: the bounds are relative
                _check_attention(dtype, q, k, v.double() / size, o.double() / size,
                                 list(zip(q0[:-1], q0[1:], k0[:-1], k0[1:])), dh ** -0.5)


# ------------------------------------------------------------------------------------- norm_rotate

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dh,rd,inter", [(2, 2, False), (7, 4, True), (64, 32, False), (128, 128, True),
                                         (1024, 1024, False)])
def test_norm_rotate_heads_of_any_size(dh, rd, inter, dtype):
    """Finite heads whose squares overflow or vanish in fp32 are normed like any other; heads of one huge element
    too. Scaling by a power of two is exact, so the bound is test_attention_gpu.py's. In 64 bits the oracle's squares
    stay in range (1e-80 .. 1e77)."""
    torch = torch_cuda()
    f = torch.rand(rd // 2, device="cuda:0")
    qw = _rand((dh,), 3, "f32")
    for eps, sizes in ((0.0, [1e-40, 1e-30, 1e-22, 1e-12, 1.0, 1e18, 1e19, 1e20, 1e30, 6e37]),
                       (1e-6, [1.0, 1e18, 1e20, 6e37]), (1e-30, [1e-24, 1e-15, 1e-10, 1e20]),
                       (1e-42, [1e-30, 1e-21, 1e-20])):
        n = len(sizes)
        r = np.random.default_rng(9)
        x = r.uniform(0.5, 5.0, (n, 3, dh)) * r.choice([-1.0, 1.0], (n, 3, dh)) * np.array(sizes)[:, None, None]
        x[:, 1, 1:] = x[:, 1, 1:] * 1e-3
        q = torch.from_numpy(x).to(_dtype(dtype)).cuda()
        assert torch.isfinite(q).all()
        pos = _ints(np.arange(n) * 37)
        print(f"norm_rotate {(dh, rd, inter, dtype, eps)}", flush=True)
        o, _ = _g().gptq_norm_rotate(q, None, pos, f, q_weight=qw, eps=eps, interleaved=inter)
        torch.cuda.synchronize()
        # eps as the fp32 number that the kernel takes
        _check_rotate(dtype, q, None, o, None, qw, None, pos, f, None, True, float(np.float32(eps)), inter)
