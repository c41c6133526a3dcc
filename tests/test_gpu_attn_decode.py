"""GPU parity of paged decode attention (fp8_attn_decode_paged) against the plain 64-bit attention, every element
within a tolerance derived from the arithmetic; every byte of the cache that no query sees is a NaN code."""
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._attn import assert_close, assert_lse, make, reference
from tests._gpu import DEV, log

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def run(s, want_lse=True, q=None, **kw):
    q = s["q"].to(DEV) if q is None else q
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV) if want_lse else None
    if kw.get("alibi") is not None:
        kw["alibi_slopes"] = kw.pop("alibi").to(DEV)
    out = fp8.fp8_attn_decode_paged(q, s["cache"].to(DEV), s["table"].to(DEV), s["lens"].to(DEV), s["scales"].to(DEV),
                                    s["block"], fmt=s["fmt"], lse=lse, **kw)
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
    return out


SHAPES = [
    # lens, Hq, Hkv, D, block
    ([1], 1, 1, 64, 16),
    ([0, 1, 2, 31, 32, 33], 4, 2, 64, 8),
    ([577], 32, 8, 128, 16),
    ([127, 128, 129, 0, 640, 1, 255], 8, 1, 128, 1),
    ([500, 3], 17, 1, 128, 100),          # 17 query heads: a second column tile with one column
    ([300, 1000], 6, 3, 256, 24),
    ([63, 64, 65], 40, 2, 256, 7),        # 20 heads per KV head
    ([2500], 5, 5, 64, 128),
]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"L{s[0][0]}x{len(s[0])}h{s[1]}-{s[2]}d{s[3]}p{s[4]}")
def test_decode(shape, dtype, fmt):
    lens, Hq, Hkv, D, block = shape
    s = make(lens, Hq, Hkv, D, block, fmt, dtype, seed=len(lens) + D + Hq)
    check(s, f"decode {shape} {dtype} {fmt}")


@pytest.mark.parametrize("kw", [
    dict(softcap=5.0), dict(softcap=50.0, window=100), dict(window=1), dict(window=33), dict(window=100000),
    dict(alibi=True), dict(alibi=True, softcap=20.0, window=64), dict(sm_scale=0.5), dict(sm_scale=0.0),
    dict(sm_scale=-0.05)], ids=str)
@pytest.mark.parametrize("D,fmt", [(64, "e5m2"), (128, "e4m3"), (256, "e5m2")])
def test_decode_scores(D, fmt, kw):
    s = make([0, 1, 40, 700, 3001], 12, 4, D, 16, fmt, FP32, seed=D)
    kw = dict(kw)
    if kw.get("alibi"):
        kw["alibi"] = torch.linspace(0.001, 1.0, 12)
    check(s, f"scores D={D} {fmt} {kw}", **kw)


@pytest.mark.parametrize("max_len", [0, 1, 300, 100000])
def test_hint_changes_no_result(max_len):
    """The length hint plans the launch: too small, unknown or too large, sequences are computed whole."""
    s = make([3000, 10, 0, 700], 8, 2, 128, 16, "e5m2", FP32, seed=5)
    check(s, f"hint {max_len}", launch=dict(max_len=max_len))


def test_lengths_past_the_table_and_bad_pages():
    s = make([100, 200, 64, 70], 4, 1, 64, 16, "e4m3", FP32, seed=9, width_extra=0)
    s["lens"][1] = 5000                   # past the table: taken as its width
    s["lens"][2] = -7                     # taken as empty
    last = s["table"][1].clone()
    s["table"][0, 2] = -1                 # pages outside the pool hide their keys
    s["table"][0, 4] = 1 << 30
    s["table"][3, :] = s["cache"].shape[0] // 16
    s["table"][1] = last
    # sequence 1 now covers its table's whole width: make the tail of its last page finite
    page = int(s["table"][1, -1])
    s["cache"][page * 16:(page + 1) * 16] &= 0x3F
    check(s, "clamped lengths, bad pages")


def test_strided_queries_and_outputs():
    s = make([77, 1300, 5], 6, 2, 128, 16, "e5m2", BF16, seed=11)
    big = torch.zeros((3, 6 * 128 + 1024), dtype=BF16, device=DEV)
    big[:, 512:512 + 768] = s["q"].view(3, -1).to(DEV)
    q = big[:, 512:512 + 768].view(3, 6, 128)
    outb = torch.full((3, 904), -3.0, dtype=BF16, device=DEV)
    out = outb[:, 64:64 + 768].view(3, 6, 128)
    wide = torch.full((3, s["table"].shape[1] + 5), -1, dtype=torch.int32)
    wide[:, :s["table"].shape[1]] = s["table"]
    table = wide.to(DEV)[:, :s["table"].shape[1]]
    got = fp8.fp8_attn_decode_paged(q, s["cache"].to(DEV), table, s["lens"].to(DEV), s["scales"].to(DEV), 16, out=out)
    torch.cuda.synchronize()
    assert got is out
    want, _, tol = reference(s, lse=False)
    assert_close(out, want, tol, "strided")
    assert bool((outb[:, :64] == -3).all()) and bool((outb[:, 64 + 768:] == -3).all())


def test_cache_rows_past_32_bits():
    """Rows whose byte offset passes 2^32."""
    Hkv, D, block = 8, 128, 16
    s = make([200], 8, Hkv, D, block, "e5m2", FP32, seed=13)
    slots = (1 << 32) // (2 * Hkv * D) + 4096
    nb = slots // block
    cache = torch.empty((nb * block, 2 * Hkv * D), dtype=torch.uint8, device=DEV)
    n_small = s["cache"].shape[0] // block
    cache[-n_small * block:] = s["cache"].to(DEV)
    table = torch.where(s["table"] >= 0, s["table"] + nb - n_small, s["table"])
    out = fp8.fp8_attn_decode_paged(s["q"].to(DEV), cache, table.to(DEV), s["lens"].to(DEV), s["scales"].to(DEV), block)
    torch.cuda.synchronize()
    want, _, tol = reference(s, lse=False)
    assert_close(out, want, tol, "past 32 bits")


def test_scales_below_the_floor_and_tiny_scales():
    s = make([90, 300], 4, 2, 64, 16, "e5m2", FP32, seed=15)
    s["scales"][:] = 1e-9
    s["scales"][3] = 0.0
    s["scales"][200] = 1e-20
    check(s, "tiny scales")
    s["scales"][:] = 1e-3
    s["q"] *= 1e6                          # one key takes all the weight
    out, _ = run(s)
    assert bool(torch.isfinite(out).all())


def test_same_bits_twice_and_on_another_stream():
    s = make([4000, 9, 2222], 16, 4, 128, 16, "e5m2", BF16, seed=17)
    args = [t.to(DEV) for t in (s["q"], s["cache"], s["table"], s["lens"], s["scales"])]
    a = fp8.fp8_attn_decode_paged(*args, 16, max_len=4000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = fp8.fp8_attn_decode_paged(*args, 16, max_len=4000, stream=side)
    c = fp8.fp8_attn_decode_paged(*args, 16, max_len=4000)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


def test_graph_replay_follows_its_inputs():
    """A captured step replayed with other queries, lengths and pages (a padded batch: an empty sequence fills up)."""
    first = make([3000, 0, 700], 16, 4, 128, 16, "e5m2", BF16, seed=19, width_extra=60)
    second = make([1, 2900, 0], 16, 4, 128, 16, "e5m2", BF16, seed=20, width_extra=60)
    W = max(first["table"].shape[1], second["table"].shape[1])
    slots = max(first["cache"].shape[0], second["cache"].shape[0])

    def padded(s):
        t = torch.full((3, W), -1, dtype=torch.int32)
        t[:, :s["table"].shape[1]] = s["table"]
        c = torch.zeros((slots, s["cache"].shape[1]), dtype=torch.uint8)
        c[:s["cache"].shape[0]] = s["cache"]
        return [x.to(DEV) for x in (s["q"], c, t, s["lens"], s["scales"])]

    static = padded(first)
    ws = torch.empty(fp8.fp8_attn_decode_workspace_bytes(3, 16, 4, 128, 16, W, 3000), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0
    fp8.fp8_attn_decode_paged(*static, 16, max_len=3000, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fp8.fp8_attn_decode_paged(*static, 16, max_len=3000, ws=ws)
    for s in (first, second, first, second):
        for dst, src in zip(static, padded(s)):
            dst.copy_(src)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        want, _, tol = reference(s, lse=False)
        assert_close(out, want, tol, "replay")


@pytest.mark.parametrize("cap", [1e3, 1e5, 1e8, 1e30])
@pytest.mark.parametrize("D,dtype,new", [(64, BF16, 1), (128, BF16, 1), (256, BF16, 1), (128, FP32, 1), (128, BF16, 90), (64, FP16, 90)])
def test_a_cap_far_above_the_scores(D, dtype, new, cap):
    """cap tanh(x / cap) is x less x^3 / (3 cap^2), under 2^-11 for the scores here (|x| < 10) and a cap of 1000 or more:
    the uncapped result, with that and the cap's own roundings (4 of 2^-24 of the score) added to every score's error."""
    s = make([700, 5, 0, 130], 8, 4, D, 16, "e5m2", dtype, seed=D + 3, new=None if new == 1 else [new, 2, 0, 30])
    want, _, tol = reference(s, lse=False)
    # both sums of p: at most exp(2 ds) - 1 < 3 ds of the largest value
    q, cache, table, lens, scales = [s[k].to(DEV) for k in ("q", "cache", "table", "lens", "scales")]
    kw = dict(softcap=cap)
    if new == 1:
        out = fp8.fp8_attn_decode_paged(q, cache, table, lens, scales, 16, **kw)
    else:
        out = fp8.fp8_attn_prefill_paged(q, s["cu"].to(DEV), cache, table, lens, scales, 16, max_q=new, **kw)
    torch.cuda.synchronize()
    v = s["cache"].view(torch.float8_e5m2).float().nan_to_num(0.0).abs().amax() * s["scales"].max()
    ds = 10.0 ** 3 / (3 * cap * cap) + 10 * 4 * 2.0 ** -24
    assert largest_score(s, D ** -0.5) < 10.0
    assert_close(out, want, tol + 3 * ds * float(v), f"cap {cap} D={D} {dtype} {new}")


def largest_score(s, scale):
    """Of all queries and keys, masked ones too."""
    top, block = 0.0, s["block"]
    for b in range(s["lens"].numel()):
        n = int(s["lens"][b])
        rows = s["q"][int(s["cu"][b]):int(s["cu"][b + 1])].double()
        if not n or not rows.numel():
            continue
        j = torch.arange(n)
        k = s["cache"][s["table"][b, (j // block).long()].long() * block + j % block].view(torch.float8_e5m2).double()
        k = (k * s["scales"].double()).view(n, 2, s["Hkv"], s["D"])[:, 0]
        for h in range(s["Hq"]):
            top = max(top, float((rows[:, h] @ k[:, h // (s["Hq"] // s["Hkv"])].T).abs().max()) * scale)
    return top


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cap", [1e-38, 1e-39, 1e-45])
def test_the_smallest_caps_and_zero_queries(cap, dtype):
    """Scores of 0 and of +-cap, which is nothing: every key weighs the same."""
    s = make([300, 1, 0, 40], 4, 2, 64, 16, "e5m2", dtype, seed=5)
    s["q"][0] = 0
    want, _, tol = reference(s, lse=False, sm_scale=0.0)
    out = fp8.fp8_attn_decode_paged(*[s[k].to(DEV) for k in ("q", "cache", "table", "lens", "scales")], 16, softcap=cap)
    torch.cuda.synchronize()
    assert_close(out, want, tol, f"cap {cap} {dtype}")
