"""The FP8-output product of no K at rows that the tiled kernels take: zeros, whatever the LDS held before."""
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._gpu import DEV, log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N", [(65, 16), (300, 528), (2048, 4096)])
def test_no_k(M, N):
    log(f"fp8out {M} x {N} of no k")
    qa, qw = (torch.zeros((n, 0), dtype=torch.uint8, device=DEV) for n in (M, N))
    st, sc = torch.full((M,), 2.0, device=DEV), torch.full((N,), 3.0, device=DEV)
    # a product whose operands, left over in LDS, would read as NaN and infinite scales
    bad = torch.full((512, 1024), 0x7F, dtype=torch.uint8, device=DEV)
    fp8.fp8_gemm_scaled(bad, torch.full((512,), float("inf"), device=DEV), bad, torch.full((512,), float("nan"), device=DEV))
    q, s = fp8.fp8_gemm_scaled_fp8out(qa, st, qw, sc)
    assert (q.view(torch.float8_e4m3fn).float() == 0).all()
    assert torch.equal(s, torch.full_like(s, 1e-12))
