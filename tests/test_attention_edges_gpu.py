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
