"""A type named beside an output that is given has to be that output's."""
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._experts import codes, randn
from tests._gpu import DEV

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def product(**kw):
    return fp8.fp8_gemm_scaled_act(codes(1, 8, 64), torch.ones(8, device=DEV), codes(2, 24, 64), torch.ones(24, device=DEV), **kw)


def grouped(**kw):
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return fp8.fp8_gemm_grouped_scaled_act(codes(1, 8, 64), torch.ones(8, device=DEV), i(*range(8)), i(0, 3, 8),
                                           codes(2, 48, 64).view(2, 24, 64), torch.ones((2, 24), device=DEV), **kw)


def combine(y=None, y_dtype=None, **kw):
    row_of = torch.arange(16, dtype=torch.int32, device=DEV).view(8, 2)
    return fp8.fp8_moe_combine(randn(3, 16, 24, dtype=BF), row_of, out=y, out_dtype=y_dtype, **kw)


@pytest.mark.parametrize("call", [product, grouped, combine])
def test_types(call):
    for given in (BF, HF, F32):
        y = torch.empty((8, 24), dtype=given, device=DEV)
        assert call(y=y) is y and call(y=y, y_dtype=given) is y and call(y_dtype=given).dtype is given
        for named in {BF, HF, F32} - {given}:
            with pytest.raises(TypeError):
                call(y=y, y_dtype=named)
    assert call().dtype is BF
    with pytest.raises(TypeError):
        call(y=[1.0])


@pytest.mark.parametrize("call", [product, combine])
def test_types_beside_a_residual(call):
    res = randn(1, 8, 24)
    assert call(residual=res).dtype is F32 and call(residual=res, y_dtype=F32).dtype is F32
    for kw in (dict(y_dtype=BF), dict(y=torch.empty((8, 24), dtype=BF, device=DEV)), dict(y_dtype=BF, y=torch.empty_like(res))):
        with pytest.raises(TypeError):
            call(residual=res, **kw)
    with pytest.raises(TypeError):
        call(residual=[[1.0]])
