"""The mean-square bounds of paged attention tell its own roundings from coarser ones: emulated on the CPU, the terms
that the kernels feed pass, operands of few bits and a lost second term fail, at short and at long sequences."""
import pytest
import torch

from tests._attn import make
from tests._attn_rms import excess, lse_excess, model

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
SHAPES = [([33, 90, 64, 7, 12], None, 16, 4, 64), ([577], None, 32, 8, 128), ([300, 1000], None, 6, 3, 256), ([2500], None, 10, 5, 64),
          ([500, 140], [130, 40], 4, 2, 128)]


@pytest.mark.parametrize("kw", [{}, dict(softcap=20.0), dict(window=100)], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"L{s[0][0]}d{s[4]}")
def test_coarser_operands_are_seen(shape, kw):
    lens, new, Hq, Hkv, D = shape
    for dtype, terms, lost in ((BF16, 1, [(1, 6), (1, 8)]), (FP16, 2, [(1, 11)]), (FP32, 2, [(1, 11)])):
        s = make(lens, Hq, Hkv, D, 16, "e5m2", dtype, seed=len(lens) + D, new=new)
        want, var, lse, lvar = model(s, terms, **kw)
        own, _, own_lse, _ = model(s, terms, emulate=(terms, 11), **kw)
        assert excess(own.to(dtype), want, var, dtype) <= 1
        if terms == 2:
            assert lse_excess(own_lse.float(), lse, lvar) <= 1
        for mistake in lost:
            out, _, bad_lse, _ = model(s, terms, emulate=mistake, **kw)
            assert excess(out.to(dtype), want, var, dtype) > 2, (dtype, mistake)
            if terms == 2:
                assert lse_excess(bad_lse.float(), lse, lvar) > 2, (dtype, mistake)
