"""Products of up to 16 rows with an epilogue keep fp32's sums whatever their output's type: a 16-bit output is the exact
value rounded, but for values next to a border."""
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._experts import U, act64, act_bound, codes, product64, randn
from tests._gpu import DEV, log
from tests.test_gpu_gemm_act import scales

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 4000, 4096), (8, 3333, 2064), (16, 4096, 14336)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_outputs_off_by_a_step(M, N, K, dtype, act):
    """An fp32 sum is off by at most (K / 32) 2 u of its running value in K / 32 steps that add up like a walk, well below
    2^-20 of the output's norm; a value changes its rounding only when it is as near to a border: of uniformly placed
    values two such errors in a step, 2 2^-20 norm / (eps |value|), summed here over the outputs, with a factor of 2 and
    10 outputs for chance."""
    log(f"decode {M} {N} {K} {dtype} {act}")
    qa, qw, st, sc = codes(1, M, K), codes(2, N, K), scales(3, M), scales(4, N, K)
    y = fp8.fp8_gemm_scaled_act(qa, st, qw, sc, act=act, y_dtype=dtype)
    v, _ = product64(qa, st, qw, sc)
    norm = (qa.view(torch.float8_e4m3fn).double() ** 2) @ (qw.view(torch.float8_e4m3fn).double() ** 2).t()
    norm = norm.sqrt() * st.double()[:, None] * sc.double()
    ref = act64(v, act)
    err = norm * 2.0 ** -20 * 1.13 + act_bound(v, act, True) + ref.abs() * 3 * U
    off = y != ref.to(dtype)
    step = torch.finfo(dtype).eps * torch.exp2(torch.floor(torch.log2(ref.abs().clamp_min(torch.finfo(dtype).tiny))))
    likely = (2 * err / step).clamp_max(1.0).sum()
    assert off.sum() <= 2 * likely + 10, f"{int(off.sum())} of {off.numel()} off, {float(likely):.1f} expected at most"
