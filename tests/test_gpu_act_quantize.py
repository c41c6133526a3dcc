"""The (gated) activation with per-token quantization, against a 64-bit form and against the plain quantizer."""
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._experts import F8, U, act64, act_bound, randn
from tests._gpu import DEV, log

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def round_e4m3(x):
    """The nearest E4M3 value to each of x (float64), ties to even, held at +-448."""
    x = x.clamp(-448, 448)
    step = torch.exp2((torch.frexp(x)[1].double() - 1).clamp_min(-6) - 3)
    return torch.round(x / step) * step


def quantize_ok(h, act, gated, q, s, what):
    """Scales and codes within the fp32 evaluation's error of the 64-bit values."""
    F = q.shape[1]
    x = h[:, :F].double()
    v, err = act64(x, act), act_bound(x, act, False)
    if gated:
        u = h[:, F:].double()
        v, err = v * u, err * u.abs() + (v * u).abs() * U
    # the scale: no value's error moves the maximum by more than itself; the quotient's rounding
    want = (v.abs().amax(1) / 448).clamp_min(1e-12)
    assert ((s.double() - want).abs() <= err.amax(1) / 448 + want * 2 * U).all(), f"{what}: scales"
    # the code: that of some quotient within the value's error and the division's two roundings
    scale = s.double()[:, None]
    z, slack = v / scale, err / scale + (v / scale).abs() * 2 * U
    got = q.view(F8).double()
    bad = (got < round_e4m3(z - slack)) | (got > round_e4m3(z + slack)) | got.isnan()
    assert not bad.any(), f"{what}: {int(bad.sum())} codes"


@pytest.mark.parametrize("rows,F", [(1, 16), (3, 48), (5, 512), (64, 1040), (2, 4096), (7, 8208), (3, 16384), (2, 32768),
                                    (2, 65552), (1, 131088), (511, 528), (512, 512), (513, 1024), (700, 2048), (600, 4096),
                                    (520, 4112), (512, 16384), (515, 16400)])
@pytest.mark.parametrize("kind", [BF, HF, F32])
def test_quantize(rows, F, kind):
    log(f"quantize {rows} x {F} {kind}")
    for i, act in enumerate(ACTS):
        gated = (i + rows) % 2 == 0
        h = randn(rows + i, rows, 2 * F if gated else F, dtype=F32).mul(2.0).to(kind)
        q, s = fp8.fp8_act_quantize(h, act=act, gated=gated)
        quantize_ok(h, act, gated, q, s, f"{act} gated={gated}")


@pytest.mark.parametrize("rows,F", [(3, 48), (64, 4096), (600, 1040), (700, 5120)])
@pytest.mark.parametrize("kind", [BF, HF, F32])
def test_the_same_bits_as_the_quantizer(rows, F, kind):
    """none and relu have no error of their own, nor has one product: the codes are those of the fp32 quantizer."""
    h = randn(rows, rows, 2 * F, dtype=kind)
    for act, gated in (("none", False), ("relu", False), ("none", True), ("relu", True)):
        x = h if gated else h[:, :F]
        v = x[:, :F].float() if act == "none" else x[:, :F].float().clamp_min(0)
        v = (v * x[:, F:].float() if gated else v).contiguous()
        q, s = fp8.fp8_act_quantize(x, act=act, gated=gated)
        wq, ws = fp8.fp8_quantize_per_token(v)
        assert torch.equal(s, ws) and torch.equal(q.view(F8).float(), wq.view(F8).float()), (act, gated)


def test_zero_rows_and_far_values():
    h = torch.zeros((4, 64), dtype=F32, device=DEV)
    h[1] = -200.0
    h[2, :32], h[2, 32:] = -1e4, 1e4
    h[3, :32] = 3e3
    for act in ACTS:
        q, s = fp8.fp8_act_quantize(h, act=act, gated=False)
        want = act64(h.double(), act).abs().amax(1) / 448
        assert (s[0] == 1e-12) and (q[0].view(F8).float() == 0).all()
        assert torch.allclose(s.double(), want.clamp_min(1e-12), rtol=1e-6, atol=0), act
        assert not q.view(F8).float().isnan().any()


@pytest.mark.parametrize("rows", [40, 800])
def test_live_rows(rows):
    h = randn(1, rows, 256, dtype=BF)
    whole = fp8.fp8_act_quantize(h)
    for live in (0, 1, rows // 3, rows, rows + 5, -4):
        q, s = torch.full((rows, 128), 0x33, dtype=torch.uint8, device=DEV), torch.full((rows,), -1.0, device=DEV)
        fp8.fp8_act_quantize(h, q=q, scales=s, live_rows=torch.tensor([live], dtype=torch.int32, device=DEV))
        n = min(max(live, 0), rows)
        assert torch.equal(q[:n], whole[0][:n]) and torch.equal(s[:n], whole[1][:n])
        assert (q[n:] == 0x33).all() and (s[n:] == -1).all()


def test_strides_and_refusals():
    h = randn(1, 20, 300, dtype=BF)
    x, q = h[:, :256], torch.full((20, 160), 0x33, dtype=torch.uint8, device=DEV)
    with pytest.raises(fp8.Fp8Error):  # rows of 300 elements are not 16-byte aligned
        fp8.fp8_act_quantize(x)
    h = randn(1, 20, 304, dtype=BF)
    got, s = fp8.fp8_act_quantize(h[:, :256], act="gelu", q=q[:, :128])
    want = fp8.fp8_act_quantize(h[:, :256].contiguous(), act="gelu")
    assert torch.equal(got, want[0]) and torch.equal(s, want[1]) and (q[:, 128:] == 0x33).all()
    assert fp8.fp8_act_quantize(h[:0, :256])[0].shape == (0, 128)
    q0, s0 = fp8.fp8_act_quantize(h[:, :0], gated=False)
    assert q0.shape == (20, 0) and torch.equal(s0, torch.full_like(s0, 1e-12))
    for f in (lambda: fp8.fp8_act_quantize(h, act="swish"), lambda: fp8.fp8_act_quantize(h[:, :255]),
              lambda: fp8.fp8_act_quantize(h, q=q), lambda: fp8.fp8_act_quantize(h.t())):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        fp8.fp8_act_quantize(h.double())


def test_rows_past_four_gigabytes():
    rows, F, ld = 3, 1040, (1 << 31) + 48
    for kind in (BF, F32):
        log(f"rows 2^31 elements apart, {kind}")
        h = torch.empty(2 * ld + 2 * F, dtype=kind, device=DEV).as_strided((rows, 2 * F), (ld, 1))
        h.copy_(randn(1, rows, 2 * F, dtype=kind))
        q = torch.empty(2 * ld + F, dtype=torch.uint8, device=DEV).as_strided((rows, F), (ld, 1))
        _, s = fp8.fp8_act_quantize(h, "silu", True, q=q)
        want_q, want_s = fp8.fp8_act_quantize(h.contiguous(), "silu", True)
        quantize_ok(h.contiguous(), "silu", True, want_q, want_s, str(kind))
        assert torch.equal(q, want_q) and torch.equal(s, want_s)
