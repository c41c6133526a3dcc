"""GPU precision of paged attention beyond what worst-case elementwise bounds can see."""
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._attn import F8, make
from tests._attn_rms import assert_rms, lse_excess, model
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


SHAPES = [
    # lens, new, Hq, Hkv, D: both kernels, whole sequences and shares of keys
    ([33, 90, 64, 7, 12], None, 16, 4, 64), ([577], None, 32, 8, 128), ([300, 1000], None, 6, 3, 256), ([2500], None, 10, 5, 64),
    ([4000, 9, 2222], None, 16, 4, 128), ([9000], None, 4, 2, 128), ([2000, 130], None, 40, 1, 128),
    ([500, 140], [130, 40], 4, 2, 128), ([900], [900], 4, 2, 64), ([150, 700], [150, 129], 4, 2, 256), ([4000], [70], 8, 4, 128),
    ([200, 3000], [4, 3], 8, 2, 128)]


@pytest.mark.parametrize("kw", [{}, dict(softcap=20.0), dict(window=100), dict(alibi=True)], ids=str)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"L{s[0][0]}x{len(s[0])}h{s[2]}d{s[4]}" + (f"n{s[1][0]}" if s[1] else ""))
def test_mean_square_error(shape, fmt, kw):
    """No larger than the operands' terms and fp32 explain: one term for bf16 alone, two for the other types and beside
    log-sum-exp (whose outputs are held to two)."""
    lens, new, Hq, Hkv, D = shape
    kw = dict(kw)
    launch = dict(kw)
    if kw.get("alibi"):
        kw["alibi"] = torch.linspace(0.001, 0.3, Hq)
        del launch["alibi"]
        launch["alibi_slopes"] = kw["alibi"].to(DEV)
    if new:
        launch["max_q"] = max(new)
    for dtype, terms, want_lse in ((BF16, 1, False), (BF16, 2, True), (FP16, 2, True), (FP32, 2, True), (FP32, 2, False)):
        s = make(lens, Hq, Hkv, D, 16, fmt, dtype, seed=len(lens) + D, new=new)
        what = f"{shape} {fmt} {dtype} {kw.keys()} lse={want_lse}"
        log(f"  {what}")
        lse = torch.full(s["q"].shape[:2], 7.0, dtype=torch.float32, device=DEV) if want_lse else None
        out = call(s, decode=new is None, max_len=max(lens), lse=lse, **launch)
        want, var, ref, lvar = model(s, terms, **kw)
        assert_rms(out, want, var, dtype, what)
        if want_lse:
            x = lse_excess(lse, ref, lvar)
            assert x <= 1, f"{what}: lse {x:.3g}"
