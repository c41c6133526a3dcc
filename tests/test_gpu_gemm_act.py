"""The scaled product with bias, activation and residual in its epilogue, dense and per expert, against 64 bits."""
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._experts import (U, act64, act_bound, check, choices, codes, product64, product_bound, randn, round_bound,
                            sorted_rows)
from tests._gpu import DEV, log

pytestmark = pytest.mark.gpu
BF, HF, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def scales(seed, n, k=1):
    return (randn(seed, n) * 0.3).exp() * (0.01 / max(1, k) ** 0.5)


def expect(qa, st, qw, sc, bias, act, residual, dtype):
    """(values, bound) in 64 bits: the product's error and the bias addition's go through the activation, whose slope is
    at most 1.13."""
    K = qa.shape[1]
    v, size = product64(qa, st, qw, sc)
    err = product_bound(size, K, dtype)
    if bias is not None:
        v = v + bias.double()
    err = err + v.abs() * U
    ref, err = act64(v, act), err * 1.13 + act_bound(v, act, dtype is F32)
    if residual is not None:
        ref = ref + residual.double()
        err = err + (ref.abs() + err) * U
    return ref, err + round_bound(ref, dtype) * (1 + 2.0 ** -8)


def near(got, ref, dtype, K, what):
    """The 2-norm: an fp32 output keeps fp32 sums, 16-bit ones are their rounding (and the FP8 instructions' 3e-5)."""
    norm = ref.norm().item()
    if norm:
        most = {F32: 2e-6, BF: 2.2e-3, HF: 3e-4}[dtype]
        off = ((got.double() - ref).norm() / norm).item()
        assert off <= most, f"{what}: 2-norm {off:.3g}"


CASES = [  # M, N, K: waves' and tiles' ends, K splits, K that is no multiple of 128, one row or column
    (1, 1, 16), (1, 100, 128), (3, 17, 4096), (8, 4096, 1040), (16, 257, 2064), (17, 130, 256), (33, 1000, 144),
    (48, 513, 4112), (64, 300, 1024), (64, 2048, 8192), (64, 28672, 256), (20, 1027, 6160), (65, 64, 256), (65, 1, 128),
    (100, 255, 112), (127, 129, 384), (128, 128, 16), (129, 257, 128), (191, 500, 2064), (193, 256, 640), (256, 256, 256),
    (257, 513, 272), (300, 1001, 1024), (400, 5000, 528), (777, 1203, 2064), (1025, 640, 4096), (2048, 2048, 512),
    (70, 8192, 3968), (2500, 90, 96), (1, 3, 0), (80, 70, 0)]


@pytest.mark.parametrize("M,N,K", CASES)
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_gemm(M, N, K, dtype):
    log(f"gemm {M} {N} {K} {dtype}")
    qa, qw = codes(1, M, K), codes(2, N, K)
    st, sc, bias, res = scales(3, M), scales(4, N, K), randn(5, N) * 0.5, randn(6, M, N, dtype=dtype)
    for i, act in enumerate(ACTS):
        b, r = (bias, None)[(i + M) % 2], (None, res)[(i + N // 2) % 2]
        y = fp8.fp8_gemm_scaled_act(qa, st, qw, sc, bias=b, act=act, residual=r, y_dtype=dtype)
        assert y.dtype is dtype
        ref, bound = expect(qa, st, qw, sc, b, act, r, dtype)
        check(y, ref, bound, f"{act} {b is not None} {r is not None}")
        if M * N >= 4096:
            near(y, ref, dtype, K, act)


@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (16, 4096, 2048), (40, 520, 1040), (64, 8192, 4096), (100, 300, 256),
                                   (260, 700, 384), (1000, 1024, 1024)])
def test_plain_epilogue_is_the_plain_product(M, N, K):
    """Nothing in the epilogue: bf16 values of the same sums, rounded once."""
    qa, qw, st, sc = codes(1, M, K), codes(2, N, K), scales(3, M), scales(4, N, K)
    y = fp8.fp8_gemm_scaled_act(qa, st, qw, sc)
    plain = fp8.fp8_gemm_scaled(qa, st, qw, sc)
    ref, bound = expect(qa, st, qw, sc, None, "none", None, BF)
    check(y, ref, bound, "act")
    check(plain, ref, bound, "plain")


@pytest.mark.parametrize("M", [4, 40, 100, 300])
def test_strides_in_place_and_padding_codes(M):
    N, K = 203, 336
    qa, qw = codes(1, M, 480, nan_from=K)[:, :K], codes(2, N, 480, nan_from=K)[:, :K]  # NaN codes past K
    st, sc, bias = scales(3, M), scales(4, N, K), randn(5, N)
    for dtype in (BF, HF, F32):
        for pad in (0, 1, 5, 53):
            y = torch.full((M, N + pad), 3.0, dtype=dtype, device=DEV)
            res = randn(6, M, N + 9, dtype=dtype)[:, :N]
            got = fp8.fp8_gemm_scaled_act(qa, st, qw, sc, bias=bias, act="silu", residual=res, y=y[:, :N])
            ref, bound = expect(qa, st, qw, sc, bias, "silu", res, dtype)
            check(got, ref, bound, f"{dtype} pad {pad}")
            assert (y[:, N:] == 3).all()
            own = torch.full((M, N + pad), 3.0, dtype=dtype, device=DEV)
            own[:, :N] = res
            fp8.fp8_gemm_scaled_act(qa, st, qw, sc, bias=bias, act="silu", residual=own[:, :N], y=own[:, :N])
            assert torch.equal(own[:, :N], y[:, :N]) and (own[:, N:] == 3).all()


def test_activations_of_any_value():
    """K = 0: y = act(bias)."""
    one = torch.ones(1, device=DEV)
    x = torch.cat([torch.linspace(-30, 30, 20001, device=DEV), randn(1, 20000) * 3, torch.logspace(-40, 38, 500, device=DEV),
                   -torch.logspace(-40, 38, 500, device=DEV), torch.tensor([0.0, -0.0, 5.0, -5.0, -87.5, -104.0, -1e30], device=DEV)])
    q0, w0 = torch.zeros((1, 0), dtype=U8, device=DEV), torch.zeros((x.numel(), 0), dtype=U8, device=DEV)
    for rows in (1, 70):
        for act in ACTS:
            y = fp8.fp8_gemm_scaled_act(q0.expand(rows, 0).contiguous(), one.repeat(rows), w0, torch.ones_like(x), bias=x,
                                        act=act, y_dtype=F32)
            ref = act64(x.double(), act)
            check(y, ref.expand(rows, -1), (act_bound(x.double(), act, True) + ref.abs() * U + 2.0 ** -126).expand(rows, -1), act)
    for act in ACTS:  # NaN stays NaN
        y = fp8.fp8_gemm_scaled_act(q0, one, w0[:3], torch.ones(3, device=DEV), act=act, y_dtype=BF,
                                    bias=torch.tensor([float("nan"), 1.0, float("nan")], device=DEV))
        assert y.isnan().tolist() == [[True, False, True]], act


def grouped_expect(qa, st, tok, off, qw, sc, bias, act, y, dtype):
    ref, bound = y.double(), torch.zeros_like(y, dtype=torch.float64)
    for e in range(qw.shape[0]):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            t = torch.from_numpy(tok[a:b]).to(DEV).long()
            ref[a:b], bound[a:b] = expect(qa[t], st[t], qw[e], sc[e], None if bias is None else bias[e], act, None, dtype)
    return ref, bound


@pytest.mark.parametrize("T,topk,E,N,K,dropped", [
    (1, 1, 1, 1, 16, 0), (1, 4, 16, 130, 128, 0), (5, 2, 3, 64, 144, 0.3), (40, 3, 6, 257, 256, 0.1), (200, 2, 4, 300, 1040, 0),
    (700, 1, 2, 513, 384, 0.05), (600, 4, 40, 96, 2064, 0), (3, 2, 200, 40, 512, 0.2), (260, 2, 2, 1024, 1024, 0)])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_grouped(T, topk, E, N, K, dropped, dtype):
    log(f"grouped {T} {topk} {E} {N} {K} {dtype}")
    off, tok, _ = sorted_rows(choices(T + N, T, topk, E, dropped, T // 9), E)
    R = T * topk
    qa, qw, st = codes(1, T, K), codes(2, E * N, K).view(E, N, K), scales(3, T)
    sc, bias = scales(4, E * N, K).view(E, N), randn(5, E, N) * 0.5
    offd, tokd = torch.from_numpy(off).to(DEV), torch.from_numpy(tok).to(DEV)
    for i, act in enumerate(ACTS):
        b = bias if i % 2 == 0 else None
        pad = (0, 8, 3)[i % 3]
        whole = torch.full((R, N + pad), 7.0, dtype=dtype, device=DEV)
        y = whole[:, :N]
        before = y.clone()
        assert fp8.fp8_gemm_grouped_scaled_act(qa, st, tokd, offd, qw, sc, bias=b, act=act, y=y) is y
        ref, bound = grouped_expect(qa, st, tok, off, qw, sc, b, act, before, dtype)
        check(y, ref, bound, f"{act} {b is not None}")
        assert (whole[:, N:] == 7).all() and (y[int(off[-1]):] == 7).all()


@pytest.mark.parametrize("M,N,K", [(4000, 4090, 4112), (4090, 4001, 4096), (5000, 7000, 528), (4097, 4096, 512),
                                   (1100, 2000, 2064), (300, 300, 8192), (20, 300, 16384), (17, 64, 32768)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gemm_of_each_division(M, N, K, dtype):
    """Sizes that take the larger tiles and the longer splits, ragged on every side."""
    log(f"gemm {M} {N} {K} {dtype}")
    qa, qw, st, sc = codes(1, M, K), codes(2, N, K), scales(3, M), scales(4, N, K)
    bias, res = randn(5, N) * 0.5, randn(6, M, N, dtype=dtype)
    for act, r in (("gelu", res), ("none", None)):
        y = fp8.fp8_gemm_scaled_act(qa, st, qw, sc, bias=bias, act=act, residual=r, y_dtype=dtype)
        ref, bound = expect(qa, st, qw, sc, bias, act, r, dtype)
        check(y, ref, bound, act)
        near(y, ref, dtype, K, act)
        if r is not None:
            own = r.clone()
            fp8.fp8_gemm_scaled_act(qa, st, qw, sc, bias=bias, act=act, residual=own, y=own)
            assert torch.equal(own, y)


@pytest.mark.parametrize("T,topk,E,N,K", [(4000, 1, 3, 3500, 2064), (4000, 1, 3, 3500, 2048), (3000, 3, 2, 3000, 528),
                                          (9000, 1, 8, 2049, 1024)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_grouped_of_each_division(T, topk, E, N, K, dtype):
    log(f"grouped {T} {topk} {E} {N} {K} {dtype}")
    off, tok, _ = sorted_rows(choices(T + N, T, min(topk, E), E, 0.02, 50), E)
    qa, qw, st = codes(1, T, K), codes(2, E * N, K).view(E, N, K), scales(3, T)
    sc, bias = scales(4, E * N, K).view(E, N), randn(5, E, N) * 0.5
    y = torch.full((tok.size, N), 7.0, dtype=dtype, device=DEV)
    before = y.clone()
    fp8.fp8_gemm_grouped_scaled_act(qa, st, torch.from_numpy(tok).to(DEV), torch.from_numpy(off).to(DEV), qw, sc, bias=bias,
                                    act="silu", y=y)
    ref, bound = grouped_expect(qa, st, tok, off, qw, sc, bias, "silu", before, dtype)
    check(y, ref, bound, "grouped")
    assert (y[int(off[-1]):] == 7).all()


def test_replays_match_eager():
    """Captured products, one of them with its sums in a workspace of its own, replayed with eager work in between."""
    made = []
    for M, N, K, dtype in ((5, 300, 512, BF), (20, 300, 16384, F32), (100, 700, 528, HF), (300, 1300, 1024, BF)):
        qa, qw, st, sc = codes(1, M, K), codes(2, N, K), scales(3, M), scales(4, N, K)
        res, y = randn(6, M, N, dtype=dtype), torch.empty((M, N), dtype=dtype, device=DEV)
        ws = torch.empty(max(1, fp8.fp8_gemm_act_workspace_bytes(M, N, K)), dtype=U8, device=DEV)
        made.append((qa, st, qw, sc, res, y, ws))
    assert made[1][6].numel() > 1

    def run():
        for qa, st, qw, sc, res, y, ws in made:
            fp8.fp8_gemm_scaled_act(qa, st, qw, sc, act="gelu", residual=res, y=y, ws=ws)

    run()
    torch.cuda.synchronize()
    eager = [m[5].clone() for m in made]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for r in range(3):
        for m in made:
            m[5].zero_()
            m[6].fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for m, e in zip(made, eager):
            assert torch.equal(m[5], e), f"replay {r}: {tuple(m[5].shape)}"
        run()


def test_two_streams_at_once():
    M, N, K = 40, 600, 8192  # a split k: each call has a workspace of its own
    qa, qw, st, sc = codes(1, M, K), codes(2, N, K), scales(3, M), scales(4, N, K)
    want = fp8.fp8_gemm_scaled_act(qa, st, qw, sc, act="silu", y_dtype=F32)
    assert fp8.fp8_gemm_act_workspace_bytes(M, N, K) > 0
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s in streams:
            got.append(fp8.fp8_gemm_scaled_act(qa, st, qw, sc, act="silu", y_dtype=F32, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


def test_refused_arguments():
    qa, qw, st, sc = codes(1, 8, 64), codes(2, 24, 64), scales(3, 8), scales(4, 24)
    for f in (lambda: fp8.fp8_gemm_scaled_act(qa, st, qw, sc, act="tanh"), lambda: fp8.fp8_gemm_scaled_act(qa, st, qw[:, :48], sc),
              lambda: fp8.fp8_gemm_scaled_act(qa, st, qw, sc, bias=torch.ones(8, device=DEV)),
              lambda: fp8.fp8_gemm_scaled_act(qa, st, qw, sc, residual=torch.ones((8, 23), device=DEV)),
              lambda: fp8.fp8_gemm_scaled_act(qa.t(), st, qw, sc)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: fp8.fp8_gemm_scaled_act(qa, st, qw, sc, y_dtype=torch.float64),
              lambda: fp8.fp8_gemm_scaled_act(qa, st, qw, sc, residual=torch.ones((8, 24), device=DEV), y_dtype=BF),
              lambda: fp8.fp8_gemm_scaled_act(qa, st, qw.float(), sc)):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: fp8.fp8_gemm_scaled_act(codes(1, 8, 72), st, codes(2, 24, 72), sc),
              lambda: fp8.fp8_gemm_scaled_act(qa[:, :48], st, qw[:, :48], sc, y=torch.empty((8, 26), device=DEV)[:, 1:25])):
        with pytest.raises(fp8.Fp8Error):
            f()


def far(t):
    """t's rows, 2^31 elements and some apart."""
    ld = (1 << 31) + 48
    out = torch.empty((t.shape[0] - 1) * ld + t.shape[1], dtype=t.dtype, device=DEV).as_strided(tuple(t.shape), (ld, 1))
    return out.copy_(t)


@pytest.mark.parametrize("M,N", [(3, 100), (20, 3), (300, 3)])
def test_rows_past_four_gigabytes(M, N):
    """Of the weights, and with few rows of the codes, the residual and the output too (which decode, tiles and a split k write)."""
    K = 4112
    qa, qw, st, sc, bias = codes(1, M, K), codes(2, N, K), scales(3, M), scales(4, N, K), randn(5, N)
    for dtype in (BF, F32):
        log(f"far rows {M} {N} {dtype}")
        res = randn(6, M, N, dtype=dtype)
        want = fp8.fp8_gemm_scaled_act(qa, st, qw, sc, bias=bias, act="gelu", residual=res)
        if M == 3:
            got = fp8.fp8_gemm_scaled_act(far(qa), st, qw, sc, bias=bias, act="gelu", residual=far(res), y=far(torch.zeros_like(res)))
        else:
            got = fp8.fp8_gemm_scaled_act(qa, st, far(qw), sc, bias=bias, act="gelu", residual=res)
        assert torch.equal(got, want)


@pytest.mark.parametrize("M", [17, 30])
def test_outputs_past_four_gigabytes(M):
    N, K, ld = 40, 1040, (1 << 28) + 16
    qa, qw, st, sc = codes(1, M, K), codes(2, N, K), scales(3, M), scales(4, N, K)
    res = randn(6, M, N, dtype=BF)
    log(f"rows 2^28 elements apart, {M}")
    want = fp8.fp8_gemm_scaled_act(qa, st, qw, sc, act="silu", residual=res)
    y = torch.empty((M - 1) * ld + N, dtype=BF, device=DEV).as_strided((M, N), (ld, 1))
    y.copy_(res)
    assert torch.equal(fp8.fp8_gemm_scaled_act(qa, st, qw, sc, act="silu", residual=y, y=y), want)
