"""The grouped product's 2-norm error: fp32 outputs keep fp32's sums, which the elementwise bounds, made for sums that
cancel, would not tell from the FP8 instructions'."""
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._experts import choices, codes, randn, sorted_rows
from tests._gpu import DEV, log
from tests.test_gpu_gemm_act import grouped_expect, near, scales

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("T,topk,E,N,K", [
    (40, 3, 6, 257, 256), (200, 2, 4, 300, 1040), (600, 4, 40, 96, 2064),   # tiles of 64, rings of 4 and 2
    (4000, 1, 3, 3500, 2064), (4000, 1, 3, 3500, 2048), (9000, 1, 8, 2049, 1024)])  # the larger tiles
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_norm(T, topk, E, N, K, dtype):
    log(f"grouped {T} {topk} {E} {N} {K} {dtype}")
    off, tok, _ = sorted_rows(choices(T + N, T, topk, E, 0.02, 7), E)
    qa, qw, st = codes(1, T, K), codes(2, E * N, K).view(E, N, K), scales(3, T)
    sc, bias = scales(4, E * N, K).view(E, N), randn(5, E, N) * 0.5
    live = int(off[-1])
    for act in ("none", "silu", "gelu"):
        y = torch.zeros((tok.size, N), dtype=dtype, device=DEV)
        fp8.fp8_gemm_grouped_scaled_act(qa, st, torch.from_numpy(tok).to(DEV), torch.from_numpy(off).to(DEV), qw, sc,
                                        bias=bias, act=act, y=y)
        ref, _ = grouped_expect(qa, st, tok, off, qw, sc, bias, act, torch.zeros_like(y), dtype)
        near(y[:live], ref[:live], dtype, K, act)


def test_two_streams_of_two_products():
    """A split k on two streams at once, other operands on each: sums of one in the other's workspace would show."""
    M, N, K = 40, 600, 8192
    assert fp8.fp8_gemm_act_workspace_bytes(M, N, K) > 0
    qw, sc = codes(2, N, K), scales(4, N, K)
    sides = [(torch.cuda.Stream(), codes(10 + i, M, K), scales(20 + i, M)) for i in range(2)]
    call = lambda qa, st, **kw: fp8.fp8_gemm_scaled_act(qa, st, qw, sc, act="silu", y_dtype=F32, **kw)  # noqa: E731
    want = [call(qa, st) for _, qa, st in sides]
    assert not torch.equal(*want)
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (s, qa, st) in enumerate(sides):
            got[i].append(call(qa, st, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i]), f"stream {i}"
