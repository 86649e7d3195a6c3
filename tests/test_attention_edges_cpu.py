"""Refusals and workspace sizes of gptq_norm_rotate, gptq_attention, gptq_lora_gemm and the block driver that reads
them (CPU only: no call here launches a kernel)."""

import ctypes

import pytest

from test_attention_cpu import EINVAL, ENOMEM, FAKE, _attention, _lib, _lora

EUNSUPPORTED = -3


# ------------------------------------------------------------------------------ more than a launch

def test_attention_refuses_more_tiles_than_one_launch():
    """(n_q * group / 128 + seqs) * kv_heads from 2^24 on."""
    big = dict(n_kv=0, seqs=1, q_ld=128, out_ld=128, q_heads=8, head_dim=16, out_hp=16)
    at = dict(out=FAKE << 30)
    assert _attention(at, n_q=1 << 30, kv_heads=8, **big) == EUNSUPPORTED
    assert _attention(at, n_q=1 << 30, kv_heads=1, **big) == EUNSUPPORTED
    assert _attention(at, n_q=1 << 29, kv_heads=2, **big) == EUNSUPPORTED


def test_block_attention_refuses_more_tiles_than_one_launch():
    """The block driver refuses what its attention would, before anything is queued."""
    L = _lib()
    shape = L.gptq_block_shape_t(8, 8, 8, 1 << 8, 1 << 20, 1e-6)
    at = L.gptq_block_attn_t(kv_heads=8, norm_eps=1e-6, axes=1, causal=1)
    p = L.gptq_params_t(4, 8, 8, 0, 0, 0, 0, 0.01)
    assert L.lib().gptq_block_attn_workspace_bytes(ctypes.byref(shape), ctypes.byref(at), ctypes.byref(p)) == 0
    lay = (L.gptq_block_layer_t * 7)(*[L.gptq_block_layer_t(*[FAKE] * 7, 1) for _ in range(7)])
    info = (ctypes.c_int64 * 2)()
    P = ctypes.c_void_p(FAKE)
    assert L.lib().gptq_quantize_block_attn(ctypes.byref(shape), ctypes.byref(at), P, 1, ctypes.byref(p), 1, lay, P, None,
                                            P, 1 << 62, info, None) == EUNSUPPORTED


# -------------------------------------------------------------------------------------------- lora

@pytest.mark.parametrize("kw", [
    dict(base=5 * FAKE + 16, ld_y=1 << 31, ld_base=1 << 31),     # overlapping, at a byte count past 64 bits
    dict(ld_y=1 << 31), dict(ld_x=1 << 31), dict(base=1 << 60, ld_base=1 << 31),
], ids=str)
def test_lora_rejects_arrays_past_the_address_space(kw):
    assert _lora(m=1 << 31, work_bytes=0) == ENOMEM
    assert _lora(m=1 << 31, work_bytes=0, **kw) == EINVAL


# ------------------------------------------------------------------------------------ block driver

def test_block_shape_without_heads_is_refused_by_the_library():
    torch = pytest.importorskip("torch")                   # noqa: F841
    import post_weight_quantization_20_amd as g
    p = g.Params(bits=4, group_size=8, block_size=8)
    for attn in (None, g.BlockAttention(kv_heads=1)):
        for heads in (0, 3, -1):
            assert g.gptq_block_workspace_bytes(g.BlockShape(8, heads, 8, 1, 4), p, attn) == 0
    assert g.BlockShape(8, 0, 8, 1, 4).layer_dims(1, 1) == (8, 8)


# ------------------------------------------------------------------- adapters that no row names

@pytest.mark.parametrize("m,d", [(40, 4096), (333, 4096), (512, 11008), (1000, 11008), (1024, 4096), (2000, 11008)])
def test_lora_split_of_features_does_not_follow_the_loaded_adapters(m, d):
    """The workspace holds one T for each range of d: as many ranges with 64 or 1000 adapters as with four."""
    f = _lib().lib().gptq_lora_workspace_bytes
    need = f(m, d, 4096, 4, 16)
    assert need > 0 and f(m, d, 4096, 64, 16) == need and f(m, d, 4096, 1000, 16) == need
