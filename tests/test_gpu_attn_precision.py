"""GPU precision of paged attention beyond what worst-case elementwise bounds can see."""
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._attn import F8, make
from tests._gpu import DEV, log

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def call(s, decode=False, **kw):
    q, cu, cache, table, lens, scales = [s[k].to(DEV) for k in ("q", "cu", "cache", "table", "lens", "scales")]
    if decode:
        out = fp8.fp8_attn_decode_paged(q, cache, table, lens, scales, s["block"], fmt=s["fmt"], **kw)
    else:
        out = fp8.fp8_attn_prefill_paged(q, cu, cache, table, lens, scales, s["block"], fmt=s["fmt"], **kw)
    torch.cuda.synchronize()
    return out.double().cpu()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("D,new", [(64, 1), (128, 1), (256, 1), (64, 80), (128, 80), (256, 80)])
def test_equal_values_come_out_as_they_are(D, new, dtype, fmt):
    """Where all keys carry the same value v, sum p v / sum p is v whatever p is, so both sums have to see the same p.

    Sequences of n <= 8 keys: each sum is off by n 2^-24 at the most, the quotient, its product with the scale and the
    fp32 scale itself by 2^-24 each: v comes out within (2 n + 4) 2^-24 < 2^-19 before it is rounded to the type.  The
    channels' values are bf16 midpoints moved by 2^-16 of themselves either way, so a bf16 output that is off by more
    than that (a p rounded for one sum alone is off by 2^-12) rounds to the wrong neighbour."""
    lens = [2, 3, 5, 8] if new > 1 else [2, 3, 5, 8] * 8
    log(f"  equal values D={D} {dtype} {fmt} {new}")
    s = make(lens, 8, 4, D, 16, fmt, dtype, seed=D + new, new=None if new == 1 else [new] * 4)
    C = 4 * D
    one = torch.tensor([1.0]).to(F8[fmt][0]).view(torch.uint8)[0]
    s["cache"][:, C:] = one
    g = torch.Generator().manual_seed(3)
    m = torch.randint(128, 256, (C,), generator=g).double()
    sign = torch.where(torch.rand(C, generator=g) < 0.5, -1.0, 1.0).double()
    v = (m + 0.5) / 128 * (1 + sign * 2.0 ** -16)
    s["scales"][C:] = v.float()
    v = s["scales"][C:].double().view(4, 1, D).expand(4, 2, D).reshape(8, D)
    out = call(s, decode=new == 1, **({} if new == 1 else dict(causal=False, max_q=new)))
    want = v.expand(out.shape[0], 8, D)
    if dtype == BF16:
        assert torch.equal(out, want.to(BF16).double()), float(((out - want) / want).abs().max())
    else:
        half = {FP16: 2.0 ** -11, FP32: 2.0 ** -24}[dtype]
        assert float(((out - want) / want).abs().max()) <= half + 2.0 ** -19
