"""GPU parity of paged prefill attention (fp8_attn_prefill_paged): ragged batches, causal, prefix, window, cap and
bias against the plain 64-bit attention."""
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._attn import assert_close, assert_lse, make, reference
from tests._gpu import DEV, log

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def run(s, out=None, want_lse=True, **kw):
    q = s["q"].to(DEV)
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV) if want_lse else None
    kw = dict(kw)
    if kw.get("alibi") is not None:
        kw["alibi_slopes"] = kw.pop("alibi").to(DEV)
    if kw.get("prefix") is not None:
        kw["prefix_lens"] = kw.pop("prefix").to(DEV)
    out = fp8.fp8_attn_prefill_paged(q, s["cu"].to(DEV), s["cache"].to(DEV), s["table"].to(DEV), s["lens"].to(DEV),
                                     s["scales"].to(DEV), s["block"], fmt=s["fmt"], out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def check(s, what, launch=(), **kw):
    log(f"  {what}")
    out, lse = run(s, **dict(launch), **kw)
    want, want_lse, tol = reference(s, **kw)
    assert_close(out, want, tol, what)
    assert_lse(lse, want_lse, s, what)
    if out.dtype == BF16:  # without lse, by the one-term products
        want, _, tol = reference(s, lse=False, **kw)
        assert_close(run(s, want_lse=False, **dict(launch), **kw)[0], want, tol, what + ", no lse")


SHAPES = [
    # lens, new, Hq, Hkv, D, block
    ([1], [1], 1, 1, 64, 16),
    ([200, 33, 5], [4, 4, 4], 8, 2, 128, 16),             # drafted tokens
    ([0, 1, 70, 300], [0, 1, 64, 17], 4, 4, 64, 8),
    ([300], [300], 8, 1, 128, 16),                        # a whole prompt
    ([150, 700, 129], [150, 129, 1], 6, 2, 256, 24),
    ([513, 257], [300, 257], 3, 3, 128, 1),
    ([900], [900], 10, 2, 64, 100),
    ([400, 140], [190, 130], 24, 1, 64, 32),
]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"L{s[0][0]}n{s[1][0]}x{len(s[0])}h{s[2]}-{s[3]}d{s[4]}p{s[5]}")
def test_prefill(shape, dtype, fmt):
    lens, new, Hq, Hkv, D, block = shape
    s = make(lens, Hq, Hkv, D, block, fmt, dtype, seed=sum(lens) + D, new=new)
    check(s, f"prefill {shape} {dtype} {fmt}", launch=dict(max_q=max(new), max_len=max(lens)))


@pytest.mark.parametrize("kw", [
    dict(causal=False), dict(prefix=[50, 0, 400, -3, 9]), dict(window=20), dict(prefix=[50, 0, 400, 7, 9], window=100),
    dict(causal=False, window=30), dict(softcap=4.0), dict(alibi=True, prefix=[10, 1, 2000, 100, 0], softcap=30.0),
    dict(sm_scale=0.3, window=1)], ids=str)
@pytest.mark.parametrize("D,fmt,dtype", [(64, "e4m3", FP32), (128, "e5m2", BF16), (256, "e4m3", FP16)])
def test_prefill_masks(D, fmt, dtype, kw):
    s = make([290, 3, 500, 180, 40], 8, 4, D, 16, fmt, dtype, seed=D + 1, new=[290, 2, 133, 8, 40])
    kw = dict(kw)
    if kw.get("alibi"):
        kw["alibi"] = torch.linspace(0.001, 1.0, 8)
    if kw.get("prefix"):
        kw["prefix"] = torch.tensor(kw["prefix"], dtype=torch.int32)
    check(s, f"masks D={D} {fmt} {dtype} {kw}", **kw)


@pytest.mark.parametrize("max_q,max_len", [(0, 0), (1, 1), (40, 100), (5000, 100000)])
def test_hints_change_no_result(max_q, max_len):
    s = make([700, 90, 300], 8, 2, 128, 16, "e5m2", BF16, seed=3, new=[500, 90, 2])
    check(s, f"hints {max_q} {max_len}", launch=dict(max_q=max_q, max_len=max_len))


@pytest.mark.parametrize("nq", [3, 200])
def test_more_new_tokens_than_keys(nq):
    """Rows whose causal mask leaves nothing: zeros and -inf."""
    s = make([nq // 2, 0], 4, 2, 64, 16, "e5m2", FP32, seed=4, new=[nq, 2])
    check(s, f"{nq} new over {nq // 2}")


@pytest.mark.parametrize("new", [[5, 3], [150, 140]])
def test_rows_behind_the_last_sequence_stay(new):
    s = make([300, 200], 4, 2, 128, 16, "e4m3", BF16, seed=6, new=new)
    n = sum(new)
    s["q"] = torch.cat([s["q"], torch.zeros((9, 4, 128), dtype=BF16)])
    out = torch.full((n + 9, 4, 128), -5.0, dtype=BF16, device=DEV)
    out, lse = run(s, out=out)
    want, want_lse, tol = reference(s)
    assert_close(out[:n], want[:n], tol[:n], "owned rows")
    assert bool((out[n:] == -5).all()) and bool((lse[n:] == 7).all())


def test_offsets_outside_the_rows_are_held_inside():
    s = make([300, 200, 100], 4, 2, 64, 16, "e5m2", FP32, seed=8, new=[140, 130, 7])
    good = reference(s)
    s["cu"][3] = 100000                    # taken as the last row
    out, _ = run(s)
    assert_close(out[:270], good[0][:270], good[2][:270], "the other sequences")


def test_cache_rows_past_32_bits():
    Hkv, D, block = 8, 128, 16
    s = make([260], 8, Hkv, D, block, "e5m2", BF16, seed=13, new=[200])
    nb = ((1 << 32) // (2 * Hkv * D) + 4096) // block
    cache = torch.empty((nb * block, 2 * Hkv * D), dtype=torch.uint8, device=DEV)
    n_small = s["cache"].shape[0] // block
    cache[-n_small * block:] = s["cache"].to(DEV)
    table = torch.where(s["table"] >= 0, s["table"] + nb - n_small, s["table"])
    out = fp8.fp8_attn_prefill_paged(s["q"].to(DEV), s["cu"].to(DEV), cache, table.to(DEV), s["lens"].to(DEV),
                                     s["scales"].to(DEV), block)
    torch.cuda.synchronize()
    want, _, tol = reference(s, lse=False)
    assert_close(out, want, tol, "past 32 bits")


@pytest.mark.parametrize("new", [[4, 4], [260, 150]])
def test_graph_replay(new):
    s = make([2000, 900], 8, 2, 128, 16, "e5m2", BF16, seed=21, new=new)
    args = [t.to(DEV) for t in (s["q"], s["cu"], s["cache"], s["table"], s["lens"], s["scales"])]
    eager = fp8.fp8_attn_prefill_paged(*args, 16, max_q=max(new))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fp8.fp8_attn_prefill_paged(*args, 16, max_q=max(new))
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        fp8.fp8_attn_prefill_paged(*args, 16, max_q=max(new))
    want, _, tol = reference(s, lse=False)
    assert_close(out, want, tol, "replay")
