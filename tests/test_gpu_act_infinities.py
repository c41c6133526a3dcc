"""The epilogues' activations of infinite and of the largest values, in every output type: as the formulas have it."""
import math

import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._gpu import DEV, log

pytestmark = pytest.mark.gpu
INF, NAN, MOST = math.inf, math.nan, torch.finfo(torch.float32).max
# value of x: none, relu, silu, gelu, gelu_tanh
EXPECT = {INF: (INF, INF, INF, INF, INF), -INF: (-INF, 0.0, NAN, NAN, NAN), NAN: (NAN,) * 5, MOST: (MOST,) * 5,
          -MOST: (-MOST, 0.0, 0.0, 0.0, 0.0), 1e19: (1e19,) * 5, -1e19: (-1e19, 0.0, 0.0, 0.0, 0.0)}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [1, 70, 300])
def test_infinite_and_largest(rows, dtype):
    """K = 0: y = act(bias), by the decode kernel, by tiles and by larger tiles."""
    x = torch.tensor(list(EXPECT) * 3, device=DEV)
    qa, qw = torch.zeros((rows, 0), dtype=torch.uint8, device=DEV), torch.zeros((x.numel(), 0), dtype=torch.uint8, device=DEV)
    one = torch.ones(rows, device=DEV)
    for i, act in enumerate(("none", "relu", "silu", "gelu", "gelu_tanh")):
        log(f"{act} {rows} {dtype}")
        y = fp8.fp8_gemm_scaled_act(qa, one, qw, torch.ones_like(x), bias=x, act=act, y_dtype=dtype)
        want = torch.tensor([v[i] for v in EXPECT.values()] * 3, device=DEV).to(dtype).expand(rows, -1)
        torch.testing.assert_close(y, want, rtol=0, atol=0, equal_nan=True, msg=act)


def test_a_grouped_bias_of_infinity():
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV)
    tok = torch.arange(5, dtype=torch.int32, device=DEV)
    qa, qw = torch.zeros((5, 16), dtype=torch.uint8, device=DEV), torch.zeros((2, 9, 16), dtype=torch.uint8, device=DEV)
    bias = torch.zeros((2, 9), device=DEV)
    bias[0, 3] = bias[1, 8] = INF
    y = fp8.fp8_gemm_grouped_scaled_act(qa, torch.ones(5, device=DEV), tok, off, qw, torch.ones((2, 9), device=DEV),
                                        bias=bias, act="gelu", y_dtype=torch.bfloat16)
    want = torch.where(torch.tensor([0, 0, 1, 1, 1], device=DEV)[:, None] == 0, bias[0], bias[1]).to(torch.bfloat16)
    assert torch.equal(y, want)
