"""The activation quantizer's fp32 evaluation: scales, which are fp32 outputs, to a few units of 2^-24 of their value."""
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._experts import U, act64, act_bound
from tests._gpu import DEV, log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
def test_scales(act, kind, gated):
    """Rows of one value each, whose scale is |act(x) u| / 448: the activation's bound, the product's and the division's
    roundings."""
    log(f"{act} {kind} gated={gated}")
    x = torch.cat([torch.linspace(-11, 11, 4001, device=DEV), torch.logspace(-3, 1, 500, device=DEV)]).to(kind)
    h = x[:, None].expand(-1, 32).clone()
    if gated:
        h[:, 16:] = torch.linspace(0.5, 3.0, x.numel(), device=DEV).to(kind)[:, None]
    q, s = fp8.fp8_act_quantize(h, act=act, gated=gated)
    v, err = act64(x.double(), act), act_bound(x.double(), act, True)
    if gated:
        u = h[:, 16].double()
        v, err = v * u, err * u + (v * u).abs() * U
    want = v.abs() / 448
    over = (s.double() - want).abs() - (err / 448 + want * U)
    # below 1e-11 the floor of scales is near; gelu(-6) / 448 is 1.3e-11, so all x from -6 on stay, 3591 rows
    keep = want > 1e-11
    assert keep.sum() > 3500
    assert over[keep].max() <= 0, f"{(over[keep] / (want[keep] * U)).max():.3g} units of 2^-24 outside"
