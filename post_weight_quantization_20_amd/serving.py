"""Python binding of serving in 8 bits: gptq_norm_quant, gptq_byte_gemm, gptq_kv_append and gptq_kv_attention
(include/gptq.h).

Argument marshalling only, as in attention.py. A call runs on the tensors' device, on `stream` or that device's
current stream; outputs and workspaces it makes itself are allocated on the same stream.
"""

from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import _lib
from .attention import _device, _heads, _place, _ptr, _scratch, _vector
from .solver import _DTYPE, GPTQ_F32, _check


def _rows(t: torch.Tensor, shape: tuple, dtype, name: str) -> int:
    """Row pitch of a matrix with unit column stride."""
    if t.dim() != 2 or tuple(t.shape) != shape or t.dtype != dtype \
            or (shape[0] > 0 and shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be {dtype} {list(shape)} with unit column stride")
    return t.stride(0) if shape[0] > 1 else max(shape[1], 1)


def _tokens(t: torch.Tensor, name: str, dtype=None) -> Tuple[int, int, int, int, int]:
    """_heads, where a tensor without tokens may have any strides."""
    if t.dim() == 3 and t.shape[0] == 0:
        t = t.new_empty(t.shape)
    return _heads(t, name, dtype)


def gptq_norm_quant(x: torch.Tensor, residual: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                    eps: float = 1e-6, sum_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                    codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(codes, scales, sum): with h = x + residual (x [n, d], rounded to its type) and
    y = weight * h / sqrt(mean(h^2) + eps), int8 codes [n, d] and float32 scales [n] of y: scales = max |y| / 127 and
    codes = y / scales to the nearest. sum is h, in sum_out (which may be x or residual) or a new tensor, or None
    without a residual and sum_out. y, if given, receives the normed rows."""
    dev = _device(x, residual, weight, sum_out, y, codes, scales)
    if x.dim() != 2 or x.dtype not in _DTYPE:
        raise ValueError("x must be [n, d], fp32/fp16/bf16")
    n, d = x.shape
    x_ld = _rows(x, (n, d), x.dtype, "x")
    r_ld = 0 if residual is None else _rows(residual, (n, d), x.dtype, "residual")
    w_dtype = GPTQ_F32
    if weight is not None:
        if weight.dtype not in _DTYPE or tuple(weight.shape) != (d,) or not weight.is_contiguous():
            raise ValueError("weight must be contiguous [d], fp32/fp16/bf16")
        w_dtype = _DTYPE[weight.dtype]
    s, here = _place(dev, stream)
    with here:
        if sum_out is None and residual is not None:
            sum_out = torch.empty((n, d), dtype=x.dtype, device=dev)
        if codes is None:
            codes = torch.empty((n, d), dtype=torch.int8, device=dev)
        if scales is None:
            scales = torch.empty(n, dtype=torch.float32, device=dev)
        _vector(scales, (n,), torch.float32, "scales")
        a = _lib.gptq_norm_quant_t(n, d, x_ld, r_ld,
                                   0 if sum_out is None else _rows(sum_out, (n, d), x.dtype, "sum_out"),
                                   0 if y is None else _rows(y, (n, d), x.dtype, "y"),
                                   _rows(codes, (n, d), torch.int8, "codes"), float(eps), _DTYPE[x.dtype], w_dtype)
        _check(_lib.lib().gptq_norm_quant(ctypes.byref(a), _ptr(x), _ptr(residual), _ptr(weight), _ptr(sum_out),
                                          _ptr(y), _ptr(codes), _ptr(scales), s))
    return codes, scales, sum_out


def gptq_byte_gemm(x: torch.Tensor, x_scales: Optional[torch.Tensor], w: torch.Tensor,
                   w_scales: Optional[torch.Tensor], zeros: Optional[torch.Tensor] = None,
                   y: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """y[i, r] = x_scales[i] * w_scales[r] * sum_k x[i, k] * (w[r, k] - zeros[r]) for int8 x [m, d]. w is int8
    [rows, d] (zeros None), or a layer stored with bits = 8 and one group per row: its codes, uint8 [rows, d], or
    gptq_pack's words, int32 [rows, d / 4], with its int32 zeros [rows] ([rows, 1] too, as are w_scales). y is fp32,
    fp16 or bf16 [m, rows] (a new one: of `dtype`)."""
    dev = _device(x, x_scales, w, w_scales, zeros, y)
    if x.dim() != 2:
        raise ValueError("x must be int8 [m, d]")
    m, d = x.shape
    x_ld = _rows(x, (m, d), torch.int8, "x")
    if w.dim() != 2:
        raise ValueError("w must be two-dimensional")
    rows = w.shape[0]
    if zeros is None:
        w_ld = _rows(w, (rows, d), torch.int8, "w (without zeros)")
    elif w.dtype == torch.int32:
        if d % 4:
            raise ValueError("packed words hold a multiple of 4 columns")
        w_ld = 4 * _rows(w, (rows, d // 4), torch.int32, "w (packed, with zeros)")
    else:
        w_ld = _rows(w, (rows, d), torch.uint8, "w (codes, with zeros)")
    if w_scales is not None and w_scales.dim() == 2 and w_scales.shape[1] == 1:
        w_scales = w_scales[:, 0]
    if zeros is not None and zeros.dim() == 2 and zeros.shape[1] == 1:
        zeros = zeros[:, 0]
    _vector(x_scales, (m,), torch.float32, "x_scales")
    _vector(w_scales, (rows,), torch.float32, "w_scales")
    _vector(zeros, (rows,), torch.int32, "zeros")
    s, here = _place(dev, stream)
    with here:
        if y is None:
            y = torch.empty((m, rows), dtype=dtype, device=dev)
        if y.dtype not in _DTYPE:
            raise ValueError("y must be fp32/fp16/bf16")
        y_ld = _rows(y, (m, rows), y.dtype, "y")
        _check(_lib.lib().gptq_byte_gemm(_ptr(x), m, x_ld, _ptr(x_scales), _ptr(w), w_ld, _ptr(w_scales), _ptr(zeros),
                                         rows, d, _ptr(y), _DTYPE[y.dtype], y_ld, s))
    return y


def _cache(k_cache, v_cache, k_scales, v_scales, table) -> _lib.gptq_kv_cache_t:
    """The cache of [pages, page_size, kv_heads, head_dim] codes and [pages, kv_heads] scales."""
    pitch = []
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dim() != 4 or t.dtype != torch.int8 or t.shape != k_cache.shape or (t.shape[3] > 1 and t.stride(3) != 1):
            raise ValueError(f"{name} must be int8 [pages, page_size, kv_heads, head_dim] with unit stride along "
                             "head_dim")
        # a pitch that no element needs may be anything: what a contiguous array has
        dense = (t.shape[1] * t.shape[2] * t.shape[3], t.shape[2] * t.shape[3], t.shape[3])
        pitch.append([t.stride(i) if t.shape[i] > 1 else dense[i] for i in range(3)])
    pages, ps, hk, dh = k_cache.shape
    _vector(k_scales, (pages, hk), torch.float32, "k_scales")
    _vector(v_scales, (pages, hk), torch.float32, "v_scales")
    if table.dim() != 2 or table.dtype != torch.int32 or not table.is_contiguous():
        raise ValueError("table must be contiguous int32 [seqs, max_pages]")
    return _lib.gptq_kv_cache_t(_ptr(k_cache), _ptr(v_cache), _ptr(k_scales), _ptr(v_scales), pages, *pitch[0],
                                *pitch[1], ps, hk, dh, table.shape[1])


def gptq_kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   k_scales: torch.Tensor, v_scales: torch.Tensor, table: torch.Tensor, past: torch.Tensor,
                   start: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                   inv_freq: Optional[torch.Tensor] = None, pair_axis: Optional[torch.Tensor] = None,
                   interleaved: bool = False, stream=None) -> None:
    """Appends k (rotated by position) and v [n, kv_heads, head_dim] to an int8 cache [pages, page_size, kv_heads,
    head_dim] with float32 scales [pages, kv_heads], in place. Rows start[s] .. start[s + 1] (int32 [seqs + 1];
    without it, equal ranges) follow sequence s's past[s] tokens (int32 [seqs]) in the pages of table[s] (int32
    [seqs, max_pages]). Rotation with inv_freq, as in gptq_norm_rotate; positions (int32 [n] or [axes, n]) are the
    tokens' places unless given."""
    dev = _device(k, v, k_cache, v_cache, k_scales, v_scales, table, past, start, positions, inv_freq, pair_axis)
    c = _cache(k_cache, v_cache, k_scales, v_scales, table)
    n, hk, dh, k_ld, k_hp = _tokens(k, "k")
    nv, hv, dv, v_ld, v_hp = _tokens(v, "v", k.dtype)
    if (hk, dh) != (c.kv_heads, c.head_dim) or (nv, hv, dv) != (n, hk, dh):
        raise ValueError("k and v must be [n, kv_heads, head_dim] with the cache's heads")
    seqs = table.shape[0]
    _vector(past, (seqs,), torch.int32, "past")
    _vector(start, (seqs + 1,), torch.int32, "start")
    rd, axes = 0, 1
    if inv_freq is not None:
        if inv_freq.dim() != 1 or 2 * inv_freq.numel() > dh:
            raise ValueError("inv_freq must be one-dimensional, with no more pairs than a head")
        rd = 2 * inv_freq.numel()
        _vector(inv_freq, (rd // 2,), torch.float32, "inv_freq")
        if positions is not None:
            if positions.dtype != torch.int32 or positions.dim() not in (1, 2) or positions.shape[-1] != n \
                    or not positions.is_contiguous():
                raise ValueError("positions must be contiguous int32 [n] or [axes, n]")
            axes = positions.shape[0] if positions.dim() == 2 else 1
        _vector(pair_axis, (rd // 2,), torch.int32, "pair_axis")
    elif positions is not None or pair_axis is not None:
        raise ValueError("positions and pair_axis need inv_freq")
    s, here = _place(dev, stream)
    with here:
        a = _lib.gptq_kv_append_t(seqs, n, k_ld, k_hp, v_ld, v_hp, _DTYPE[k.dtype], rd, int(bool(interleaved)), axes)
        _check(_lib.lib().gptq_kv_append(ctypes.byref(a), ctypes.byref(c), _ptr(k), _ptr(v), _ptr(start), _ptr(past),
                                         _ptr(table), _ptr(positions), _ptr(inv_freq), _ptr(pair_axis), s))


def _kv_attention_args(q, seqs, c, scale, causal, window, softcap, out=None) -> _lib.gptq_kv_attention_t:
    nq, hq, dh, q_ld, q_hp = _tokens(q, "q")
    if dh != c.head_dim or hq == 0 or c.kv_heads == 0 or hq % c.kv_heads:
        raise ValueError("q must have the cache's head_dim and a multiple of its heads")
    o_ld, o_hp = hq * dh, dh
    if out is not None:
        no, ho, do, o_ld, o_hp = _tokens(out, "out", q.dtype)
        if (no, ho, do) != (nq, hq, dh):
            raise ValueError("out must have q's shape")
    if scale is None:
        scale = 1.0 / math.sqrt(dh)
    return _lib.gptq_kv_attention_t(seqs, nq, q_ld, q_hp, o_ld, o_hp, float(scale), float(softcap), _DTYPE[q.dtype],
                                    hq, int(bool(causal)), int(window))


def _shape_of(k_cache: torch.Tensor, table: torch.Tensor) -> _lib.gptq_kv_cache_t:
    if k_cache.dim() != 4 or table.dim() != 2:
        raise ValueError("k_cache must be [pages, page_size, kv_heads, head_dim] and table [seqs, max_pages]")
    pages, ps, hk, dh = k_cache.shape
    return _lib.gptq_kv_cache_t(16, 16, 16, 16, pages, ps * hk * dh, hk * dh, dh, ps * hk * dh, hk * dh, dh, ps, hk, dh,
                                table.shape[1])


def gptq_kv_attention_workspace_bytes(q: torch.Tensor, k_cache: torch.Tensor, table: torch.Tensor) -> int:
    """Workspace bytes of gptq_kv_attention for tensors of these shapes."""
    c = _shape_of(k_cache, table)
    a = _kv_attention_args(q, table.shape[0], c, None, True, 0, 0.0)
    return int(_lib.lib().gptq_kv_attention_workspace_bytes(ctypes.byref(a), ctypes.byref(c)))


def gptq_kv_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                      v_scales: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, scale: Optional[float] = None,
                      causal: bool = True, q_start: Optional[torch.Tensor] = None, window: int = 0,
                      softcap: float = 0.0, slopes: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      work: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Softmax attention of q [n_q, heads, head_dim] over the cache that gptq_kv_append fills: rows q_start[s] ..
    q_start[s + 1] of q (int32 [seqs + 1]; without it, equal ranges) are the last of sequence s's lens[s] tokens
    (int32 [seqs]), which stand in the pages of table[s]. causal, window (0: none), softcap and slopes (float32
    [heads]) as in gptq.h; scale is 1 / sqrt(head_dim) unless given. work: uint8,
    gptq_kv_attention_workspace_bytes. Rows of out that belong to no sequence are left as they were (undefined in
    an out made here)."""
    dev = _device(q, k_cache, v_cache, k_scales, v_scales, table, lens, q_start, slopes, out, work)
    c = _cache(k_cache, v_cache, k_scales, v_scales, table)
    seqs = table.shape[0]
    _vector(lens, (seqs,), torch.int32, "lens")
    _vector(q_start, (seqs + 1,), torch.int32, "q_start")
    s, here = _place(dev, stream)
    with here:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        a = _kv_attention_args(q, seqs, c, scale, causal, window, softcap, out)
        _vector(slopes, (a.q_heads,), torch.float32, "slopes")
        L = _lib.lib()
        if work is None:
            nb = int(L.gptq_kv_attention_workspace_bytes(ctypes.byref(a), ctypes.byref(c)))
            work = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
        else:
            work = _scratch(work, 0, dev)
        _check(L.gptq_kv_attention(ctypes.byref(a), ctypes.byref(c), _ptr(q), _ptr(q_start), _ptr(lens), _ptr(table),
                                   _ptr(slopes), _ptr(out), _ptr(work), 0 if work is None else work.numel(), s))
    return out
