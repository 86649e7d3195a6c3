"""Python binding of the attention half of a decoder block and of the adapters beside stored layers:
gptq_norm_rotate, gptq_attention and gptq_lora_gemm (include/gptq.h).

Argument marshalling only, as in solver.py. A call runs on the tensors' device, on `stream` or that
device's current stream; outputs and workspaces it makes itself are allocated on the same stream.
"""

from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import _lib
from .solver import _DTYPE, GPTQ_F32, _check


class _Here:
    """Nothing to enter: the call's device is current and so is its stream."""

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_HERE = _Here()


def _place(device, stream):
    """(hipStream_t of the call, a context that makes its device and stream current, so that allocations
    follow them). A call on the current stream of the current device pays for neither."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream must be on {device}")
        return stream.cuda_stream, torch.cuda.stream(stream)
    here = _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)
    return torch._C._cuda_getCurrentRawStream(device.index), here


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _device(first: torch.Tensor, *others) -> torch.device:
    """The device of the call: every tensor must be on it."""
    if not first.is_cuda:
        raise ValueError("tensors must be on the GPU")
    dev = first.device
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError(f"every tensor must be on {dev}")
    return dev


def _heads(t: torch.Tensor, name: str, dtype=None) -> Tuple[int, int, int, int, int]:
    """(tokens, heads, head_dim, token pitch, head pitch) of a [tokens, heads, head_dim] tensor."""
    if t.dim() != 3 or t.dtype not in _DTYPE or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name} must be [tokens, heads, head_dim], "
                         + ("fp32/fp16/bf16" if dtype is None else str(dtype)))
    n, h, d = t.shape
    ld, hp, unit = t.stride()
    if d > 1 and unit != 1:
        raise ValueError(f"{name} must have unit stride along head_dim")
    return n, h, d, (ld if n > 1 else h * d), (hp if h > 1 else d)


def _vector(t: Optional[torch.Tensor], shape: tuple, dtype, name: str) -> None:
    if t is not None and (tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")


def _scratch(work: Optional[torch.Tensor], nbytes: int, device) -> torch.Tensor:
    if work is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if work.dtype != torch.uint8 or not work.is_contiguous():
        raise ValueError("work must be a contiguous uint8 tensor")
    return work


def gptq_norm_rotate(q: torch.Tensor, k: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                     inv_freq: Optional[torch.Tensor] = None, pair_axis: Optional[torch.Tensor] = None,
                     q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                     norm: bool = True, eps: float = 1e-6, interleaved: bool = False,
                     q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                     stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(q_out, k_out): each head of q [n, heads, head_dim] and k [n, kv_heads, head_dim] divided by the
    root of its mean square (norm), times q_weight / k_weight [head_dim], and its first
    2 * len(inv_freq) columns rotated by positions * inv_freq. positions is int32 [n], or [axes, n] with
    pair_axis (int32, one entry per pair) naming each pair's row. Outputs may be the inputs (in place)."""
    dev = _device(q, k, positions, inv_freq, pair_axis, q_weight, k_weight, q_out, k_out)
    n, hq, dh, q_ld, q_hp = _heads(q, "q")
    hk = k_ld = k_hp = ko_ld = ko_hp = 0
    if k is not None:
        nk, hk, dk, k_ld, k_hp = _heads(k, "k", q.dtype)
        if nk != n or dk != dh:
            raise ValueError("k must have q's tokens and head_dim")
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need k")
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("weights need norm=True")
    w_dtype = GPTQ_F32
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            if w.dtype not in _DTYPE or tuple(w.shape) != (dh,) or not w.is_contiguous():
                raise ValueError(f"{name} must be contiguous [head_dim], fp32/fp16/bf16")
            w_dtype = _DTYPE[w.dtype]
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise ValueError("q_weight and k_weight must have one dtype")
    rd, axes = 0, 1
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be one-dimensional")
        rd = 2 * inv_freq.numel()
        if rd > dh:
            raise ValueError("inv_freq has more pairs than a head")
        _vector(inv_freq, (rd // 2,), torch.float32, "inv_freq")
        if positions is None or positions.dtype != torch.int32 or positions.dim() not in (1, 2) \
                or positions.shape[-1] != n or not positions.is_contiguous():
            raise ValueError("positions must be contiguous int32 [n] or [axes, n]")
        axes = positions.shape[0] if positions.dim() == 2 else 1
        _vector(pair_axis, (rd // 2,), torch.int32, "pair_axis")
    elif positions is not None or pair_axis is not None:
        raise ValueError("positions and pair_axis need inv_freq")
    s, here = _place(dev, stream)
    with here:
        if q_out is None:
            q_out = torch.empty((n, hq, dh), dtype=q.dtype, device=dev)
        if k is not None and k_out is None:
            k_out = torch.empty((n, hk, dh), dtype=q.dtype, device=dev)
        no, ho, do, qo_ld, qo_hp = _heads(q_out, "q_out", q.dtype)
        if (no, ho, do) != (n, hq, dh):
            raise ValueError("q_out must have q's shape")
        if k is not None:
            no, ho, do, ko_ld, ko_hp = _heads(k_out, "k_out", q.dtype)
            if (no, ho, do) != (n, hk, dh):
                raise ValueError("k_out must have k's shape")
        a = _lib.gptq_norm_rotate_t(n, q_ld, q_hp, k_ld, k_hp, qo_ld, qo_hp, ko_ld, ko_hp, float(eps),
                                    _DTYPE[q.dtype], w_dtype, hq, hk, dh, rd, int(bool(interleaved)), axes,
                                    int(bool(norm)))
        _check(_lib.lib().gptq_norm_rotate(ctypes.byref(a), _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight),
                                           _ptr(positions), _ptr(inv_freq), _ptr(pair_axis), _ptr(q_out), _ptr(k_out),
                                           s))
    return q_out, k_out


def _attention_args(q, k, v, seqs, scale, causal, softcap, out=None) -> _lib.gptq_attention_t:
    nq, hq, dh, q_ld, q_hp = _heads(q, "q")
    nk, hk, dk, k_ld, k_hp = _heads(k, "k", q.dtype)
    nv, hv, dv, v_ld, v_hp = (nk, hk, dk, k_ld, k_hp) if v is None else _heads(v, "v", q.dtype)
    if (nv, hv, dv) != (nk, hk, dk) or dk != dh:
        raise ValueError("k and v must have one shape and q's head_dim")
    if hk == 0 or hq % hk:
        raise ValueError("q's heads must be a multiple of k's")
    o_ld, o_hp = hq * dh, dh
    if out is not None:
        no, ho, do, o_ld, o_hp = _heads(out, "out", q.dtype)
        if (no, ho, do) != (nq, hq, dh):
            raise ValueError("out must have q's shape")
    if scale is None:
        scale = 1.0 / math.sqrt(dh) if dh else 0.0
    return _lib.gptq_attention_t(int(seqs), nq, nk, q_ld, q_hp, k_ld, k_hp, v_ld, v_hp, o_ld, o_hp, float(scale),
                                 float(softcap), _DTYPE[q.dtype], hq, hk, dh, int(bool(causal)))


def gptq_attention_workspace_bytes(q: torch.Tensor, k: torch.Tensor, seqs: int) -> int:
    """Workspace bytes of gptq_attention for tensors of these shapes and so many sequences."""
    return int(_lib.lib().gptq_attention_workspace_bytes(
        ctypes.byref(_attention_args(q, k, None, seqs, None, True, 0.0))))


def gptq_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: Optional[float] = None,
                   causal: bool = True, seqs: int = 1, q_start: Optional[torch.Tensor] = None,
                   kv_start: Optional[torch.Tensor] = None, softcap: float = 0.0,
                   slopes: Optional[torch.Tensor] = None, q_doc: Optional[torch.Tensor] = None,
                   kv_doc: Optional[torch.Tensor] = None, prefix: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, work: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Softmax attention of q [n_q, heads, head_dim] over k and v [n_kv, kv_heads, head_dim], packed
    sequence after sequence: rows q_start[s] .. q_start[s + 1] of q and kv_start[s] .. of k and v (int32
    [seqs + 1]; without them, `seqs` equal ranges). The queries are each sequence's last tokens. softcap,
    slopes (float32 [heads]), q_doc and kv_doc (int32 per token) and prefix (int32 per sequence) as in
    gptq.h; scale is 1 / sqrt(head_dim) unless given. work: uint8, gptq_attention_workspace_bytes. Rows of
    out that belong to no sequence are left as they were (undefined in an out made here)."""
    dev = _device(q, k, v, q_start, kv_start, slopes, q_doc, kv_doc, prefix, out, work)
    for name, t in (("q_start", q_start), ("kv_start", kv_start)):
        if t is not None:
            if t.dim() != 1 or t.numel() < 1:
                raise ValueError(f"{name} must be int32 [seqs + 1]")
            seqs = t.numel() - 1
    _vector(q_start, (seqs + 1,), torch.int32, "q_start")
    _vector(kv_start, (seqs + 1,), torch.int32, "kv_start")
    _vector(prefix, (seqs,), torch.int32, "prefix")
    if (q_doc is None) != (kv_doc is None):
        raise ValueError("q_doc and kv_doc go together")
    s, here = _place(dev, stream)
    with here:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        a = _attention_args(q, k, v, seqs, scale, causal, softcap, out)
        _vector(slopes, (a.q_heads,), torch.float32, "slopes")
        _vector(q_doc, (a.n_q,), torch.int32, "q_doc")
        _vector(kv_doc, (a.n_kv,), torch.int32, "kv_doc")
        L = _lib.lib()
        work = _scratch(work, 0 if work is not None else int(L.gptq_attention_workspace_bytes(ctypes.byref(a))), dev)
        _check(L.gptq_attention(ctypes.byref(a), _ptr(q), _ptr(k), _ptr(v), _ptr(q_start), _ptr(kv_start),
                                _ptr(slopes), _ptr(q_doc), _ptr(kv_doc), _ptr(prefix), _ptr(out), _ptr(work),
                                work.numel(), s))
    return out


def gptq_lora_workspace_bytes(m: int, d: int, rows: int, adapters: int, rank: int) -> int:
    return int(_lib.lib().gptq_lora_workspace_bytes(m, d, rows, adapters, rank))


def gptq_lora_gemm(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, index: torch.Tensor,
                   scales: Optional[torch.Tensor] = None, ranks: Optional[torch.Tensor] = None,
                   base: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                   work: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[i] = base[i] + scales[a] * (x[i] A[a]^T) B[a]^T with a = index[i] (outside [0, adapters): base[i]),
    for x [m, d], A [adapters, rank, d], B [adapters, rows, rank] of one dtype, and float32 base and y
    [m, rows]; base None is zeros, and y may be base (added in place, beside gptq_dequant_gemm's y)."""
    dev = _device(x, A, B, index, scales, ranks, base, y, work)
    if x.dim() != 2 or x.dtype not in _DTYPE or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be [m, d] with unit column stride, fp32/fp16/bf16")
    m, d = x.shape
    if A.dim() != 3 or A.shape[2] != d or A.dtype != x.dtype or not A.is_contiguous():
        raise ValueError("A must be contiguous [adapters, rank, d] of x's dtype")
    na, r, _ = A.shape
    if B.dim() != 3 or B.shape[0] != na or B.shape[2] != r or B.dtype != x.dtype or not B.is_contiguous():
        raise ValueError("B must be contiguous [adapters, rows, rank] of x's dtype")
    rows = B.shape[1]
    _vector(index, (m,), torch.int32, "index")
    _vector(scales, (na,), torch.float32, "scales")
    _vector(ranks, (na,), torch.int32, "ranks")
    s, here = _place(dev, stream)
    with here:
        if y is None:
            y = torch.empty((m, rows), dtype=torch.float32, device=dev)
        for name, t in (("base", base), ("y", y)):
            if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (m, rows)
                                  or (rows > 1 and t.stride(1) != 1)):
                raise ValueError(f"{name} must be float32 [m, rows] with unit column stride")
        L = _lib.lib()
        work = _scratch(work, 0 if work is not None else int(L.gptq_lora_workspace_bytes(m, d, rows, na, r)), dev)
        _check(L.gptq_lora_gemm(_ptr(x), _DTYPE[x.dtype], m, x.stride(0) if m > 1 else d, _ptr(A), _ptr(B), _ptr(ranks),
                                _ptr(scales), na, r, _ptr(index), rows, d, _ptr(base),
                                0 if base is None else base.stride(0) if m > 1 else rows, _ptr(y),
                                y.stride(0) if m > 1 else rows, _ptr(work), work.numel(),
                                s))
    return y
