"""GPU parity of the rotating append (fp8_kv_append_rope_paged): rotated queries and cache codes equal, bit for bit,
the rotation evaluated step by step in fp32 followed by the codec's oracle; and a prompt, its attention, an appended
token and its attention run together."""
import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
import oracle
from tests._attn import assert_close, reference
from tests._gpu import DEV, assert_codes_equal, log, to_host

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
FID = {"e4m3": oracle.E4M3, "e5m2": oracle.E5M2}


def table(P, rot):
    i = np.arange(rot // 2, dtype=np.float64)
    a = np.arange(P, dtype=np.float64)[:, None] * 10000.0 ** (-2 * i / rot)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))


def turn(x, cs, rot, interleaved):
    """x [T, H, D] fp32 numpy, cs [T, rot]: every product and sum rounded to fp32."""
    y = x.copy()
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def expect(q, k, v, pos, cs, rot, interleaved, scales, slot, fmt, prior):
    rows = cs.numpy()[pos.numpy()]
    T = k.shape[0]
    kk = turn(k.float().numpy(), rows, rot, interleaved).reshape(T, -1)
    kv = np.concatenate([kk, v.float().numpy().reshape(T, -1)], 1)
    cache = oracle.kv_quantize(kv, scales.numpy(), FID[fmt], slot.numpy(), prior.shape[0], cache=prior.numpy())
    qq = None if q is None else torch.from_numpy(turn(q.float().numpy(), rows, rot, interleaved)).to(q.dtype)
    return qq, cache


def problem(T, Hq, Hkv, D, rot, dtype, seed, P=500, slots=None):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g).to(dtype)
    slots = slots or T + 7
    slot = torch.randperm(slots, generator=g)[:T].int()
    pos = torch.randint(0, P, (T,), generator=g).int()
    C = 2 * Hkv * D
    scales = (torch.randn(C, generator=g) * 0.5).exp() / 20000
    prior = torch.randint(0, 120, (slots, C), generator=g).to(torch.uint8)
    return qkv, slot, pos, table(P, rot), scales, prior


def split(qkv, Hq, Hkv, D):
    T = qkv.shape[0]
    return (qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),
            qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D))


def same(got, want, what):
    g, w = got.cpu(), want
    kind = torch.int32 if g.dtype == FP32 else torch.int16
    off = int((g.contiguous().view(kind) != w.contiguous().view(kind)).sum())
    assert off == 0, f"{what}: {off} of {g.numel()} differ"


SHAPES = [(1, 32, 8, 128, 128), (3, 1, 1, 16, 16), (64, 64, 8, 128, 128), (37, 5, 5, 64, 32), (300, 6, 3, 256, 128),
          (5000, 2, 1, 64, 64), (11, 3, 1, 48, 16)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_append(shape, dtype, interleaved, fmt):
    T, Hq, Hkv, D, rot = shape
    log(f"  append {shape} {dtype} interleaved={interleaved} {fmt}")
    qkv, slot, pos, cs, scales, prior = problem(T, Hq, Hkv, D, rot, dtype, seed=T + D)
    if T > 2:
        slot[1] = -1                        # padding
        slot[T // 2] = prior.shape[0] + 5   # outside the cache
        scales[0] = 0.0                     # below the floor: saturates
    qd, kd, vd = split(qkv.to(DEV), Hq, Hkv, D)   # slices of one projection output
    cache = prior.to(DEV)
    out = fp8.fp8_kv_append_rope_paged(kd, vd, pos.to(DEV), cs.to(DEV), scales.to(DEV), slot.to(DEV), cache, fmt=fmt,
                                       q=qd, interleaved=interleaved)
    want_q, want_cache = expect(*split(qkv, Hq, Hkv, D), pos, cs, rot, interleaved, scales, slot, fmt, prior)
    assert_codes_equal(to_host(cache), want_cache, "cache")
    same(out, want_q, "q_out")


def test_in_place_queries_and_no_queries():
    T, Hq, Hkv, D = 200, 8, 2, 128
    qkv, slot, pos, cs, scales, prior = problem(T, Hq, Hkv, D, D, BF16, seed=2)
    want_q, want_cache = expect(*split(qkv, Hq, Hkv, D), pos, cs, D, False, scales, slot, "e5m2", prior)
    dev = qkv.to(DEV)
    q, k, v = split(dev, Hq, Hkv, D)
    cache = prior.to(DEV)
    assert fp8.fp8_kv_append_rope_paged(k, v, pos.to(DEV), cs.to(DEV), scales.to(DEV), slot.to(DEV), cache, q=q, q_out=q) is q
    same(q, want_q, "in place")
    assert_codes_equal(to_host(cache), want_cache, "cache")
    assert torch.equal(dev[:, Hq * D:].cpu(), qkv[:, Hq * D:])   # k and v stay
    cache = prior.to(DEV)
    assert fp8.fp8_kv_append_rope_paged(k, v, pos.to(DEV), cs.to(DEV), scales.to(DEV), slot.to(DEV), cache) is None
    assert_codes_equal(to_host(cache), want_cache, "cache without q")


def test_positions_outside_the_table_write_nothing():
    T, Hq, Hkv, D = 50, 4, 2, 64
    qkv, slot, pos, cs, scales, prior = problem(T, Hq, Hkv, D, D, FP16, seed=3)
    bad = torch.tensor([0, 7, 49])
    want_q, want_cache = expect(*split(qkv, Hq, Hkv, D), pos, cs, D, False, scales,
                                torch.where(torch.isin(torch.arange(T), bad), -1, slot).int(), "e4m3", prior)
    pos[bad] = torch.tensor([-1, 500, 2147483647], dtype=torch.int32)
    q, k, v = split(qkv.to(DEV), Hq, Hkv, D)
    cache, out = prior.to(DEV), torch.full((T, Hq, D), 9.0, dtype=FP16, device=DEV)
    fp8.fp8_kv_append_rope_paged(k, v, pos.to(DEV), cs.to(DEV), scales.to(DEV), slot.to(DEV), cache, fmt="e4m3", q=q,
                                 q_out=out)
    want_q[bad] = 9.0
    same(out, want_q, "q_out")
    assert_codes_equal(to_host(cache), want_cache, "cache")


def test_more_tokens_than_a_grid_has_rows():
    T = 140001
    qkv, slot, pos, cs, scales, prior = problem(T, 1, 1, 16, 16, BF16, seed=5)
    want_q, want_cache = expect(*split(qkv, 1, 1, 16), pos, cs, 16, False, scales, slot, "e5m2", prior)
    q, k, v = split(qkv.to(DEV), 1, 1, 16)
    cache = prior.to(DEV)
    out = fp8.fp8_kv_append_rope_paged(k, v, pos.to(DEV), cs.to(DEV), scales.to(DEV), slot.to(DEV), cache, q=q)
    same(out, want_q, "q_out")
    assert_codes_equal(to_host(cache), want_cache, "cache")


def test_far_positions_and_rows_past_32_bits():
    T, Hkv, D = 20, 8, 128
    P = 300000
    qkv, _, _, _, scales, _ = problem(T, 0, Hkv, D, D, BF16, seed=4)
    pos = torch.arange(P - T, P, dtype=torch.int32)
    cs = table(P, D)
    C = 2 * Hkv * D
    slots = (1 << 32) // C + 100
    slot = torch.arange(slots - T, slots, dtype=torch.int32)
    cache = torch.empty((slots, C), dtype=torch.uint8, device=DEV)
    _, k, v = split(qkv.to(DEV), 0, Hkv, D)
    fp8.fp8_kv_append_rope_paged(k, v, pos.to(DEV), cs.to(DEV), scales.to(DEV), slot.to(DEV), cache)
    _, kc, vc = split(qkv, 0, Hkv, D)
    _, want = expect(None, kc, vc, pos, cs, D, False, scales, torch.arange(T, dtype=torch.int32), "e5m2",
                     torch.zeros((T, C), dtype=torch.uint8))
    assert_codes_equal(to_host(cache[-T:]), want, "far rows")


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
def test_prompt_then_decode_steps(fmt):
    """As a serving step uses them: a ragged batch of prompts is appended and attended, then each sequence decodes
    three tokens, every step captured once and replayed; cache, rotated queries and outputs checked at every step."""
    Hq, Hkv, D, block, P = 8, 2, 128, 16, 400
    C = 2 * Hkv * D
    prompts = [70, 1, 133]
    B, n = len(prompts), sum(prompts)
    g = torch.Generator().manual_seed(31)
    cs = table(P, D)
    scales = (torch.randn(C, generator=g) * 0.3).exp() * (5 / (57344 if fmt == "e5m2" else 448))
    nb = 40
    tab = torch.randperm(nb, generator=g)[:36].view(B, 12).int()
    cache = torch.zeros((nb * block, C), dtype=torch.uint8)
    cache_d, cs_d, scales_d, tab_d = cache.to(DEV), cs.to(DEV), scales.to(DEV), tab.to(DEV)

    def slots_of(b, at):
        at = torch.tensor(at)
        return tab[b, at // block] * block + at % block

    qkv = torch.randn((n, (Hq + 2 * Hkv) * D), generator=g).to(BF16)
    pos = torch.cat([torch.arange(m) for m in prompts]).int()
    slot = torch.cat([slots_of(b, list(range(m))) for b, m in enumerate(prompts)]).int()
    cu = torch.tensor([0] + list(np.cumsum(prompts)), dtype=torch.int32)
    lens = torch.tensor(prompts, dtype=torch.int32)
    q, k, v = split(qkv.to(DEV), Hq, Hkv, D)
    qr = fp8.fp8_kv_append_rope_paged(k, v, pos.to(DEV), cs_d, scales_d, slot.to(DEV), cache_d, fmt=fmt, q=q)
    out = fp8.fp8_attn_prefill_paged(qr, cu.to(DEV), cache_d, tab_d, lens.to(DEV), scales_d, block, fmt=fmt)
    want_q, want_cache = expect(*split(qkv, Hq, Hkv, D), pos, cs, D, False, scales, slot, fmt, cache)
    assert_codes_equal(to_host(cache_d), want_cache, "prompt cache")
    same(qr, want_q, "prompt queries")
    s = dict(q=want_q, cache=torch.from_numpy(want_cache), table=tab, lens=lens, scales=scales, cu=cu, block=block,
             fmt=fmt, Hq=Hq, Hkv=Hkv, D=D)
    want, _, tol = reference(s, lse=False)
    assert_close(out, want, tol, "prompt attention")

    # the decode step, captured once: its inputs are refilled for every replay
    step_qkv = torch.zeros((B, (Hq + 2 * Hkv) * D), dtype=BF16, device=DEV)
    step_pos, step_slot = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(2))
    step_lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    q, k, v = split(step_qkv, Hq, Hkv, D)

    def step():
        qr = fp8.fp8_kv_append_rope_paged(k, v, step_pos, cs_d, scales_d, step_slot, cache_d, fmt=fmt, q=q)
        return qr, fp8.fp8_attn_decode_paged(qr, cache_d, tab_d, step_lens, scales_d, block, fmt=fmt)

    step_slot.fill_(-1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr, out = step()
    for i in range(3):
        x = torch.randn((B, (Hq + 2 * Hkv) * D), generator=g).to(BF16)
        at = [m + i for m in prompts]
        slot = torch.stack([slots_of(b, [at[b]])[0] for b in range(B)]).int()
        step_qkv.copy_(x)
        step_pos.copy_(torch.tensor(at, dtype=torch.int32))
        step_slot.copy_(slot)
        step_lens.copy_(torch.tensor(at, dtype=torch.int32) + 1)
        graph.replay()
        torch.cuda.synchronize()
        want_q, want_cache = expect(*split(x, Hq, Hkv, D), torch.tensor(at, dtype=torch.int32), cs, D, False, scales,
                                    slot, fmt, torch.from_numpy(want_cache))
        assert_codes_equal(to_host(cache_d), want_cache, f"cache after step {i}")
        same(qr, want_q, f"queries of step {i}")
        s = dict(q=want_q, cache=torch.from_numpy(want_cache), table=tab,
                 lens=torch.tensor(at, dtype=torch.int32) + 1, scales=scales,
                 cu=torch.arange(B + 1, dtype=torch.int32), block=block, fmt=fmt, Hq=Hq, Hkv=Hkv, D=D)
        want, _, tol = reference(s, lse=False)
        assert_close(out, want, tol, f"decode step {i}")


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T", [1, 7, 4000])
def test_queries_alone(T, dtype):
    """Without KV heads nothing of the cache's side is there: k, v, scales, slot_mapping and cache are null."""
    Hq, D, P = 12, 128, 500
    log(f"  queries alone T={T} {dtype}")
    g = torch.Generator().manual_seed(T)
    q = torch.randn((T, Hq, D), generator=g).to(dtype)
    pos = torch.randint(0, P, (T,), generator=g).int()
    cs = table(P, D)
    qd, pd, cd = q.to(DEV), pos.to(DEV), cs.to(DEV)
    out = torch.full((T, Hq, D), 9.0, dtype=dtype, device=DEV)
    kind = {FP32: fp8.FP8_KV_F32, BF16: fp8.FP8_KV_BF16, FP16: fp8.FP8_KV_F16}[dtype]
    code = fp8.lib().fp8_kv_append_rope_paged(qd.data_ptr(), Hq * D, out.data_ptr(), Hq * D, 0, 0, 0, 0, kind, T, Hq, 0, D,
                                              pd.data_ptr(), cd.data_ptr(), P, D, 0, 0, 1, 0, 0, 0,
                                              torch.cuda.current_stream().cuda_stream)
    assert code == fp8.FP8_OK
    want = torch.from_numpy(turn(q.float().numpy(), cs.numpy()[pos.numpy()], D, False)).to(dtype)
    same(out, want, "q_out")
