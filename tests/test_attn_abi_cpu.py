"""Refusals of the paged attention entry points, on the host before any launch (CPU only: error paths and empty
problems, none of which reach the HIP runtime), and the binding's argument checks."""
import ctypes

import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from fp8_w8a8_quantized_quantize_amd import (FP8_ERR_INVALID_ARGUMENT, FP8_ERR_UNSUPPORTED, FP8_ERR_WORKSPACE,
                                             FP8_KV_BF16, FP8_OK, SIZE_MAX)

P, Q, MIS = 0x10000, 0x20000, 0x10008   # fake device addresses, never dereferenced on these paths
S0 = ctypes.c_void_p(0)

APPEND = dict(q=P, ldq=1024, q_out=Q, ldqo=1024, k=P, ldk=256, v=P, ldv=256, dtype=FP8_KV_BF16, T=4, Hq=8, Hkv=2, D=128,
              positions=P, cos_sin=P, P=100, rot=128, inter=0, scales=P, fmt=1, slot=P, cache=Q, num_slots=64, stream=S0)
DECODE = dict(q=P, ldq=1024, dtype=FP8_KV_BF16, cache=Q, num_blocks=10, block=16, scales=P, fmt=1, table=P, ld_table=8,
              max_blocks=8, lens=P, B=4, Hq=8, Hkv=2, D=128, max_len=100, scale=0.1, softcap=0.0, alibi=0, window=0,
              out=Q, ldo=1024, lse=0, ws=0, ws_bytes=0, stream=S0)
PREFILL = dict(q=P, ldq=1024, dtype=FP8_KV_BF16, cu=P, T=20, cache=Q, num_blocks=10, block=16, scales=P, fmt=1, table=P,
               ld_table=8, max_blocks=8, lens=P, B=4, Hq=8, Hkv=2, D=128, max_q=5, max_len=100, causal=1, prefix=0,
               scale=0.1, softcap=0.0, alibi=0, window=0, out=Q, ldo=1024, lse=0, ws=0, ws_bytes=0, stream=S0)


def call(base, fn, **kw):
    assert set(kw) <= set(base), kw
    return fn(*{**base, **kw}.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), FP8_ERR_INVALID_ARGUMENT), (dict(Hq=-1), FP8_ERR_INVALID_ARGUMENT),
    (dict(num_slots=-1), FP8_ERR_INVALID_ARGUMENT), (dict(P=-1), FP8_ERR_INVALID_ARGUMENT),
    (dict(D=120, rot=112), FP8_ERR_UNSUPPORTED), (dict(rot=8), FP8_ERR_UNSUPPORTED), (dict(rot=0), FP8_ERR_UNSUPPORTED),
    (dict(rot=144), FP8_ERR_INVALID_ARGUMENT), (dict(dtype=3), FP8_ERR_INVALID_ARGUMENT),
    (dict(fmt=2), FP8_ERR_INVALID_ARGUMENT), (dict(k=0), FP8_ERR_INVALID_ARGUMENT), (dict(v=0), FP8_ERR_INVALID_ARGUMENT),
    (dict(q=0), FP8_ERR_INVALID_ARGUMENT), (dict(q_out=0), FP8_ERR_INVALID_ARGUMENT),
    (dict(ldk=255), FP8_ERR_INVALID_ARGUMENT), (dict(ldk=260), FP8_ERR_UNSUPPORTED), (dict(ldq=1000), FP8_ERR_INVALID_ARGUMENT),
    (dict(q=MIS), FP8_ERR_UNSUPPORTED), (dict(cos_sin=MIS), FP8_ERR_UNSUPPORTED), (dict(cos_sin=0), FP8_ERR_INVALID_ARGUMENT),
    (dict(scales=0), FP8_ERR_INVALID_ARGUMENT), (dict(scales=MIS), FP8_ERR_UNSUPPORTED), (dict(cache=0), FP8_ERR_INVALID_ARGUMENT),
    (dict(cache=MIS), FP8_ERR_UNSUPPORTED), (dict(positions=0), FP8_ERR_INVALID_ARGUMENT), (dict(positions=P + 2), FP8_ERR_UNSUPPORTED),
    (dict(slot=0), FP8_ERR_INVALID_ARGUMENT), (dict(slot=P + 1), FP8_ERR_UNSUPPORTED),
    (dict(T=1 << 40), FP8_ERR_UNSUPPORTED), (dict(num_slots=1 << 40), FP8_ERR_UNSUPPORTED),
    (dict(Hkv=1 << 40), FP8_ERR_UNSUPPORTED), (dict(Hq=1 << 40), FP8_ERR_UNSUPPORTED),
    (dict(T=0, k=0, v=0, q=0, q_out=0, positions=0, slot=0, scales=0, cos_sin=0), FP8_OK),
    (dict(P=0, cos_sin=0), FP8_OK),                    # no position is inside the table: nothing to write
    (dict(Hq=0, q=0, q_out=0, Hkv=0, k=0, v=0, scales=0, slot=0, cache=0), FP8_OK),
], ids=str)
def test_append_refusals(kw, code):
    assert call(APPEND, fp8.lib().fp8_kv_append_rope_paged, **kw) == code


SHARED = [
    (dict(B=-1), FP8_ERR_INVALID_ARGUMENT), (dict(block=0), FP8_ERR_INVALID_ARGUMENT), (dict(Hkv=0), FP8_ERR_INVALID_ARGUMENT),
    (dict(Hq=7, ldq=1024), FP8_ERR_INVALID_ARGUMENT), (dict(D=96), FP8_ERR_UNSUPPORTED), (dict(D=512), FP8_ERR_UNSUPPORTED),
    (dict(dtype=5), FP8_ERR_INVALID_ARGUMENT), (dict(fmt=-1), FP8_ERR_INVALID_ARGUMENT), (dict(q=0), FP8_ERR_INVALID_ARGUMENT),
    (dict(out=0), FP8_ERR_INVALID_ARGUMENT), (dict(cache=0), FP8_ERR_INVALID_ARGUMENT), (dict(scales=0), FP8_ERR_INVALID_ARGUMENT),
    (dict(lens=0), FP8_ERR_INVALID_ARGUMENT), (dict(table=0), FP8_ERR_INVALID_ARGUMENT), (dict(ld_table=7), FP8_ERR_INVALID_ARGUMENT),
    (dict(num_blocks=-1), FP8_ERR_INVALID_ARGUMENT), (dict(num_blocks=1 << 28), FP8_ERR_UNSUPPORTED),
    (dict(max_blocks=1 << 27, ld_table=1 << 27), FP8_ERR_UNSUPPORTED), (dict(max_blocks=-1), FP8_ERR_INVALID_ARGUMENT),
    (dict(max_len=-1), FP8_ERR_INVALID_ARGUMENT), (dict(window=-1), FP8_ERR_INVALID_ARGUMENT),
    (dict(softcap=-1.0), FP8_ERR_INVALID_ARGUMENT), (dict(softcap=float("nan")), FP8_ERR_INVALID_ARGUMENT),
    (dict(softcap=float("inf")), FP8_ERR_INVALID_ARGUMENT), (dict(scale=float("inf")), FP8_ERR_INVALID_ARGUMENT),
    (dict(scale=float("nan")), FP8_ERR_INVALID_ARGUMENT), (dict(ldq=1023), FP8_ERR_INVALID_ARGUMENT),
    (dict(ldq=1028), FP8_ERR_UNSUPPORTED), (dict(ldo=1028), FP8_ERR_UNSUPPORTED), (dict(q=MIS), FP8_ERR_UNSUPPORTED),
    (dict(out=MIS), FP8_ERR_UNSUPPORTED), (dict(scales=MIS), FP8_ERR_UNSUPPORTED), (dict(lse=P + 2), FP8_ERR_UNSUPPORTED),
    (dict(lens=P + 1), FP8_ERR_UNSUPPORTED), (dict(table=P + 3), FP8_ERR_UNSUPPORTED), (dict(alibi=P + 2), FP8_ERR_UNSUPPORTED),
    (dict(Hq=1 << 40, ldq=1 << 50, ldo=1 << 50), FP8_ERR_UNSUPPORTED), (dict(B=1 << 40), FP8_ERR_UNSUPPORTED),
    (dict(Hq=0), FP8_OK),
]


@pytest.mark.parametrize("kw,code", SHARED + [(dict(B=0, q=0, out=0, lens=0, table=0, scales=0), FP8_OK)], ids=str)
def test_decode_refusals(kw, code):
    assert call(DECODE, fp8.lib().fp8_attn_decode_paged, **kw) == code


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(T=-1), FP8_ERR_INVALID_ARGUMENT), (dict(cu=0), FP8_ERR_INVALID_ARGUMENT), (dict(cu=P + 2), FP8_ERR_UNSUPPORTED),
    (dict(prefix=P + 2), FP8_ERR_UNSUPPORTED), (dict(max_q=-1), FP8_ERR_INVALID_ARGUMENT),
    (dict(T=1 << 40), FP8_ERR_UNSUPPORTED), (dict(T=0, q=0, out=0, cu=0, lens=0, table=0, scales=0), FP8_OK),
    (dict(B=0, cu=0, lens=0, table=0, scales=0), FP8_OK)], ids=str)
def test_prefill_refusals(kw, code):
    assert call(PREFILL, fp8.lib().fp8_attn_prefill_paged, **kw) == code


def test_workspace():
    L = fp8.lib()
    need = fp8.fp8_attn_decode_workspace_bytes(1, 8, 2, 128, 16, 4096, 0)
    assert 0 < need < 1 << 28 and need % 256 == 0
    long = dict(B=1, max_blocks=4096, ld_table=4096, max_len=0)
    assert call(DECODE, L.fp8_attn_decode_paged, **long) == FP8_ERR_WORKSPACE
    assert call(DECODE, L.fp8_attn_decode_paged, **long, ws=P, ws_bytes=need - 1) == FP8_ERR_WORKSPACE
    assert call(DECODE, L.fp8_attn_decode_paged, **long, ws=0, ws_bytes=need) == FP8_ERR_INVALID_ARGUMENT
    assert call(DECODE, L.fp8_attn_decode_paged, **long, ws=MIS, ws_bytes=need) == FP8_ERR_UNSUPPORTED
    # a short batch needs none; refused sizes say so
    assert fp8.fp8_attn_decode_workspace_bytes(64, 64, 8, 128, 16, 8, 100) == 0
    assert fp8.fp8_attn_decode_workspace_bytes(0, 8, 2, 128, 16, 8) == 0
    for bad in [(-1, 8, 2, 128, 16, 8), (1, 8, 3, 128, 16, 8), (1, 8, 2, 96, 16, 8), (1, 8, 2, 128, 0, 8)]:
        assert fp8.fp8_attn_decode_workspace_bytes(*bad) == SIZE_MAX
    need = fp8.fp8_attn_prefill_workspace_bytes(4, 1, 8, 2, 128, 16, 4096, 4, 0)
    assert 0 < need < 1 << 28
    assert call(PREFILL, L.fp8_attn_prefill_paged, T=4, B=1, max_q=4, max_blocks=4096, ld_table=4096, max_len=0,
                ws=P, ws_bytes=need - 1) == FP8_ERR_WORKSPACE
    assert fp8.fp8_attn_prefill_workspace_bytes(-4, 1, 8, 2, 128, 16, 4096) == SIZE_MAX


def test_binding_takes_device_tensors_only():
    t = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros((32, 256), dtype=torch.uint8)
    with pytest.raises(TypeError):
        fp8.fp8_kv_append_rope_paged(t, t, i, torch.zeros(4, 64), torch.ones(256), i, c)
    with pytest.raises(TypeError):
        fp8.fp8_attn_decode_paged(t, c, i.view(2, 1), i, torch.ones(256), 16)
    with pytest.raises(TypeError):
        fp8.fp8_attn_prefill_paged(t, i, c, i.view(2, 1), i, torch.ones(256), 16)
