"""Refusals of the expert-row, epilogue and activation-quantizer entry points, on the host before any launch (CPU only:
error paths and empty problems, none of which reach the HIP runtime), and the binding's argument checks."""
import ctypes

import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from fp8_w8a8_quantized_quantize_amd import (FP8_ERR_INVALID_ARGUMENT, FP8_ERR_UNSUPPORTED, FP8_ERR_WORKSPACE,
                                             FP8_KV_BF16, FP8_KV_F16, FP8_KV_F32, FP8_OK, SIZE_MAX)

P, Q, MIS = 0x10000, 0x20000, 0x10008   # fake device addresses, never dereferenced on these paths
S0 = ctypes.c_void_p(0)
BAD, NO = FP8_ERR_INVALID_ARGUMENT, FP8_ERR_UNSUPPORTED

SORT = dict(ids=P, ids_64=0, T=8, topk=2, E=4, offsets=P, row_token=P, row_of=P, ws=0, ws_bytes=0, stream=S0)
PERMUTE = dict(x=P, ldx=100, s_tok=0, row_of=P, T=8, topk=2, R=16, H=100, elem=2, out=Q, ldo=100, s_out=0, stream=S0)
COMBINE = dict(y=P, ldy=100, yt=FP8_KV_BF16, row_of=P, weights=P, residual=0, ldr=0, out=Q, ot=FP8_KV_F32, ldo=100, T=8,
               topk=2, R=16, H=100, stream=S0)
GRAD = dict(dout=P, ldd=100, dt=FP8_KV_F32, y=P, ldy=100, yt=FP8_KV_BF16, row_of=P, weights=P, dy=Q, lddy=100, dw=Q, T=8,
            topk=2, R=16, H=100, stream=S0)
GEMM = dict(qa=P, lda=64, s_tok=P, qw=P, ldw=64, s_ch=P, bias=P, act=3, residual=P, ldr=10, y=Q, yt=FP8_KV_BF16, ldy=10,
            M=5, N=10, K=64, ws=0, ws_bytes=0, stream=S0)
GROUPED = dict(qa=P, s_tok=P, row_token=P, offsets=P, qw=P, s_ch=P, bias=P, act=2, y=Q, yt=FP8_KV_F16, ldy=10, T=5, R=9,
               E=3, N=10, K=64, ws=0, ws_bytes=0, stream=S0)
QUANT = dict(h=P, ldh=64, dtype=FP8_KV_BF16, rows=5, F=32, act=2, gated=1, q=Q, ldq=32, scales=P, live=0, stream=S0)


def call(base, fn, **kw):
    assert set(kw) <= set(base), kw
    return fn(*{**base, **kw}.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(topk=-1), BAD), (dict(E=-1), BAD), (dict(E=1025), NO), (dict(T=1 << 31), NO),
    (dict(T=1 << 20, topk=1 << 12), NO), (dict(ids=0), BAD), (dict(offsets=0), BAD), (dict(row_token=0), BAD),
    (dict(row_of=0), BAD), (dict(ids=MIS), NO), (dict(offsets=MIS), NO), (dict(row_token=MIS), NO), (dict(row_of=MIS), NO),
    (dict(T=1 << 20), FP8_ERR_WORKSPACE), (dict(T=1 << 20, ws_bytes=1 << 30), BAD),
    (dict(T=1 << 20, ws=MIS, ws_bytes=1 << 30), NO), (dict(T=0, offsets=0), BAD),
], ids=str)
def test_sort_refusals(kw, code):
    assert call(SORT, fp8.lib().fp8_moe_sort, **kw) == code


def test_sort_workspace():
    assert fp8.fp8_moe_sort_workspace_bytes(8, 8, 64) == 0
    need = fp8.fp8_moe_sort_workspace_bytes(1 << 20, 8, 1024)
    assert 0 < need < 1 << 24 and need % 256 == 0
    assert call(SORT, fp8.lib().fp8_moe_sort, T=1 << 20, topk=8, E=1024, ws=P, ws_bytes=need - 1) == FP8_ERR_WORKSPACE
    for bad in [(-1, 8, 64), (8, -1, 64), (8, 8, -1), (8, 8, 1025), (1 << 31, 1, 4), (1 << 20, 1 << 20, 4)]:
        assert fp8.fp8_moe_sort_workspace_bytes(*bad) == SIZE_MAX


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(topk=-2), BAD), (dict(R=-1), BAD), (dict(H=-1), BAD), (dict(R=1 << 31), NO),
    (dict(H=1 << 31, ldx=1 << 31, ldo=1 << 31), NO), (dict(elem=3), BAD), (dict(elem=8), BAD), (dict(elem=0), BAD),
    (dict(x=0), BAD), (dict(out=0), BAD), (dict(row_of=0), BAD), (dict(ldx=99), BAD), (dict(ldo=99), BAD),
    (dict(x=MIS), NO), (dict(out=MIS), NO), (dict(row_of=MIS), NO), (dict(s_tok=P), BAD), (dict(s_out=P), BAD),
    (dict(s_tok=MIS, s_out=P), NO), (dict(s_tok=P, s_out=MIS), NO),
    (dict(T=0, x=0, row_of=0), FP8_OK), (dict(topk=0, row_of=0), FP8_OK), (dict(R=0, out=0), FP8_OK),
    (dict(H=0, x=0, out=0, ldx=0, ldo=0), FP8_OK),
], ids=str)
def test_permute_refusals(kw, code):
    assert call(PERMUTE, fp8.lib().fp8_moe_permute, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(R=-1), BAD), (dict(H=-1), BAD), (dict(topk=1 << 31), NO), (dict(yt=3), BAD), (dict(ot=-1), BAD),
    (dict(y=0), BAD), (dict(out=0), BAD), (dict(row_of=0), BAD), (dict(ldy=99), BAD), (dict(ldo=99), BAD),
    (dict(residual=P, ldr=99), BAD), (dict(residual=MIS, ldr=100), NO), (dict(weights=MIS), NO), (dict(y=MIS), NO),
    (dict(out=MIS), NO), (dict(row_of=MIS), NO),
    (dict(T=0, out=0, row_of=0, weights=0), FP8_OK), (dict(H=0, y=0, out=0, ldy=0, ldo=0), FP8_OK),
], ids=str)
def test_combine_refusals(kw, code):
    assert call(COMBINE, fp8.lib().fp8_moe_combine, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(R=-1), BAD), (dict(H=-1), BAD), (dict(T=1 << 31), NO), (dict(dt=9), BAD), (dict(yt=9), BAD),
    (dict(dout=0), BAD), (dict(y=0), BAD), (dict(row_of=0), BAD), (dict(ldd=99), BAD), (dict(ldy=99), BAD),
    (dict(lddy=99), BAD), (dict(dout=MIS), NO), (dict(y=MIS), NO), (dict(dy=MIS), NO), (dict(dw=MIS), NO),
    (dict(weights=MIS), NO), (dict(T=0, dout=0, row_of=0, weights=0, dw=0), FP8_OK), (dict(dy=0, dw=0, y=0), FP8_OK),
    (dict(topk=0, row_of=0, weights=0), FP8_OK),
], ids=str)
def test_grad_refusals(kw, code):
    assert call(GRAD, fp8.lib().fp8_moe_combine_grad, **kw) == code


EPILOGUE = [
    (dict(N=-1), BAD), (dict(K=-1), BAD), (dict(K=40), NO), (dict(act=5), BAD), (dict(act=-1), BAD), (dict(yt=3), BAD),
    (dict(y=0), BAD), (dict(ldy=9), BAD), (dict(y=MIS), NO), (dict(bias=MIS), NO), (dict(s_ch=0), BAD), (dict(s_ch=MIS), NO),
    (dict(s_tok=0), BAD), (dict(qa=0), BAD), (dict(qw=0), BAD), (dict(qw=MIS), NO),
    (dict(N=0, y=0, qw=0, s_ch=0, bias=0), FP8_OK),
]


@pytest.mark.parametrize("kw,code", EPILOGUE + [
    (dict(M=-1), BAD), (dict(lda=63), BAD), (dict(lda=72), NO), (dict(ldw=72), NO), (dict(ldr=9), BAD),
    (dict(residual=MIS), NO), (dict(M=(1 << 31) - 1), NO), (dict(M=1 << 40), NO), (dict(N=1 << 40, ldy=1 << 40), NO),
    (dict(M=0, qa=0, s_tok=0, residual=0, y=0), FP8_OK),
], ids=str)
def test_gemm_act_refusals(kw, code):
    assert call(GEMM, fp8.lib().fp8_gemm_scaled_act, **kw) == code


@pytest.mark.parametrize("kw,code", EPILOGUE + [
    (dict(T=-1), BAD), (dict(R=-1), BAD), (dict(E=-1), BAD), (dict(E=1025), NO), (dict(E=0), BAD), (dict(T=0), BAD),
    (dict(R=1 << 31), NO), (dict(R=(1 << 31) - 1), NO), (dict(row_token=0), BAD), (dict(offsets=0), BAD),
    (dict(offsets=MIS), NO), (dict(R=0, row_token=0, offsets=0, y=0), FP8_OK),
], ids=str)
def test_grouped_act_refusals(kw, code):
    assert call(GROUPED, fp8.lib().fp8_gemm_grouped_scaled_act, **kw) == code


def test_gemm_act_workspace():
    L = fp8.lib()
    need = fp8.fp8_gemm_act_workspace_bytes(64, 8192, 28672)
    assert need >= 64 * 8192 * 4
    big = dict(M=64, N=8192, K=28672, lda=28672, ldw=28672, ldy=8192, ldr=8192)
    assert call(GEMM, L.fp8_gemm_scaled_act, **big) == FP8_ERR_WORKSPACE
    assert call(GEMM, L.fp8_gemm_scaled_act, **big, ws=P, ws_bytes=need - 1) == FP8_ERR_WORKSPACE
    assert call(GEMM, L.fp8_gemm_scaled_act, **big, ws_bytes=need) == BAD
    assert call(GEMM, L.fp8_gemm_scaled_act, **big, ws=MIS, ws_bytes=need) == NO
    assert fp8.fp8_gemm_act_workspace_bytes(0, 8, 16) == 0
    for bad in [(-1, 8, 16), (8, -1, 16), (8, 8, 24), ((1 << 31) - 1, 8, 16)]:
        assert fp8.fp8_gemm_act_workspace_bytes(*bad) == SIZE_MAX


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), BAD), (dict(F=-16), BAD), (dict(F=24), NO), (dict(rows=1 << 31), NO), (dict(act=5), BAD),
    (dict(dtype=3), BAD), (dict(h=0), BAD), (dict(q=0), BAD), (dict(scales=0), BAD), (dict(ldh=63), BAD), (dict(ldh=68), NO),
    (dict(ldq=31), BAD), (dict(ldq=40), NO), (dict(h=MIS), NO), (dict(q=MIS), NO), (dict(scales=MIS), NO),
    (dict(live=P + 2), NO), (dict(gated=0, ldh=31), BAD), (dict(rows=0, h=0, q=0, scales=0), FP8_OK),
], ids=str)
def test_act_quantize_refusals(kw, code):
    assert call(QUANT, fp8.lib().fp8_act_quantize, **kw) == code


@pytest.mark.parametrize("base,fn,kw", [
    (PERMUTE, "fp8_moe_permute", dict(out=P)), (PERMUTE, "fp8_moe_permute", dict(s_tok=P, s_out=P)),
    (COMBINE, "fp8_moe_combine", dict(out=P)), (COMBINE, "fp8_moe_combine", dict(residual=Q, ldr=101)),
    (GRAD, "fp8_moe_combine_grad", dict(dy=P, dout=P, y=Q)), (GRAD, "fp8_moe_combine_grad", dict(y=Q, ldy=101)),
    (GEMM, "fp8_gemm_scaled_act", dict(residual=Q, ldr=16)), (QUANT, "fp8_act_quantize", dict(q=P, ldq=64)),
], ids=str)
def test_outputs_at_an_inputs_address_are_refused(base, fn, kw):
    assert call(base, getattr(fp8.lib(), fn), **kw) == BAD


def test_binding_takes_device_tensors_only():
    x, i = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((4, 2), dtype=torch.int32)
    c, s = torch.zeros((4, 64), dtype=torch.uint8), torch.ones(4)
    for f in (lambda: fp8.fp8_moe_sort(i, 3), lambda: fp8.fp8_moe_permute(x, i), lambda: fp8.fp8_moe_combine(x, i),
              lambda: fp8.fp8_moe_combine_grad(x, x, i), lambda: fp8.fp8_gemm_scaled_act(c, s, c, s),
              lambda: fp8.fp8_gemm_grouped_scaled_act(c, s, i[0], i[0], c[None], s[None]),
              lambda: fp8.fp8_act_quantize(x)):
        with pytest.raises(TypeError):
            f()
