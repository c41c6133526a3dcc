"""GPU parity of paged attention over the ways a call is divided among workgroups: whole sequences or equal shares of
the keys, one to four KV heads a workgroup, the search for a share's sequence in small and large batches, key shares
of the tiled kernel.  The rules look at sizes and hints alone, so small caches with wide tables reach them all."""
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._attn import assert_close, assert_lse, make, reference
from tests._gpu import DEV, log

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def spread(B, longest, seed):
    """Lengths with many empty and one-token sequences, empty ones first and last."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, 60, (B,), generator=g)
    lens[torch.rand(B, generator=g) < 0.3] = 0
    lens[torch.rand(B, generator=g) < 0.1] = 1
    lens[B // 3], lens[B // 2] = longest, longest // 2
    lens[0] = lens[-1] = 0
    return [int(n) for n in lens]


def arguments(s):
    return [s[k].to(DEV) for k in ("q", "cache", "table", "lens", "scales")]


def decode(s, what, max_len, **kw):
    log(f"  {what}")
    q, cache, table, lens, scales = arguments(s)
    width = table.shape[1]
    need = fp8.fp8_attn_decode_workspace_bytes(q.shape[0], s["Hq"], s["Hkv"], s["D"], s["block"], width, max_len)
    ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV)
    for lse in [lse, None] if q.dtype == BF16 else [lse]:  # bf16 without lse: the one-term products
        ws.fill_(0xFF)
        out = fp8.fp8_attn_decode_paged(q, cache, table, lens, scales, s["block"], fmt=s["fmt"], lse=lse,
                                        max_len=max_len, ws=ws, **kw)
        torch.cuda.synchronize()
        want, want_lse, tol = reference(s, lse=lse is not None, **kw)
        assert_close(out, want, tol, what)
        if lse is not None:
            assert_lse(lse, want_lse, s, what)
    return need


def prefill(s, what, max_q, max_len, **kw):
    log(f"  {what}")
    q, cache, table, lens, scales = arguments(s)
    need = fp8.fp8_attn_prefill_workspace_bytes(q.shape[0], table.shape[0], s["Hq"], s["Hkv"], s["D"], s["block"],
                                                table.shape[1], max_q, max_len)
    ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV)
    call = dict(kw)
    if call.get("prefix") is not None:
        call["prefix_lens"] = call.pop("prefix").to(DEV)
    if call.get("alibi") is not None:
        call["alibi_slopes"] = call.pop("alibi").to(DEV)
    for lse in [lse, None] if q.dtype == BF16 else [lse]:
        ws.fill_(0xFF)
        out = fp8.fp8_attn_prefill_paged(q, s["cu"].to(DEV), cache, table, lens, scales, s["block"], fmt=s["fmt"],
                                         lse=lse, max_q=max_q, max_len=max_len, ws=ws, **call)
        torch.cuda.synchronize()
        want, want_lse, tol = reference(s, lse=lse is not None, **kw)
        assert_close(out, want, tol, what)
        if lse is not None:
            assert_lse(lse, want_lse, s, what)
    return need


@pytest.mark.parametrize("B", [3, 63, 64, 65, 255, 256, 257, 600])
@pytest.mark.parametrize("D,Hkv", [(64, 2), (128, 1)])
def test_shares_over_batches(B, D, Hkv):
    """A share's sequence is looked up by a lane, a wave or a workgroup per sequence, in one pass or several."""
    s = make(spread(B, 2500, B), 2 * Hkv, Hkv, D, 16, "e5m2", BF16, seed=B)
    assert decode(s, f"shares B={B} D={D}", 2500) > 0


@pytest.mark.parametrize("B", [3, 70, 300])
def test_a_batch_of_empty_sequences(B):
    s = make([0] * B, 4, 2, 64, 16, "e4m3", BF16, seed=B, width_extra=200)
    decode(s, f"empty B={B}", 3000)
    s = make([0] * (B - 1) + [1], 4, 2, 64, 16, "e4m3", BF16, seed=B, width_extra=200)
    decode(s, f"all but one empty B={B}", 3000)


@pytest.mark.parametrize("Hkv", [2, 4, 6, 8, 12, 5])
@pytest.mark.parametrize("D,fmt,dtype", [(64, "e4m3", FP32), (128, "e5m2", BF16), (256, "e4m3", BF16)])
def test_shares_of_several_heads(Hkv, D, fmt, dtype):
    """Wide tables and a large bound of the length: as many KV heads a workgroup as divide their number."""
    s = make(spread(66, 700, Hkv), Hkv, Hkv, D, 16, fmt, dtype, seed=Hkv, width_extra=1900)
    assert decode(s, f"heads {Hkv} D={D} {fmt} {dtype}", 30000) > 0


@pytest.mark.parametrize("max_len", [600, 1000])
@pytest.mark.parametrize("B,Hkv,D,dtype", [(130, 8, 64, BF16), (132, 16, 64, FP16), (66, 16, 128, BF16), (70, 12, 256, BF16)])
def test_whole_sequences_of_several_heads(B, Hkv, D, dtype, max_len):
    s = make(spread(B, 500, B), Hkv, Hkv, D, 16, "e5m2", dtype, seed=B)
    decode(s, f"whole B={B} heads {Hkv} D={D} {max_len}", max_len)


@pytest.mark.parametrize("kw", [{}, dict(window=90), dict(causal=False), dict(softcap=6.0)], ids=str)
@pytest.mark.parametrize("Hq,Hkv,D,new,dtype", [
    (24, 3, 128, [3, 2, 0, 3], BF16), (16, 2, 64, [8, 1, 0, 7], FP32), (10, 2, 256, [12, 5, 0, 9], BF16),
    (8, 4, 128, [4, 4, 0, 4], FP16)])
def test_shares_over_several_column_tiles(Hq, Hkv, D, new, dtype, kw):
    s = make([3000, 40, 10, 1500], Hq, Hkv, D, 16, "e5m2", dtype, seed=Hq, new=new)
    assert prefill(s, f"column tiles {Hq}/{Hkv} D={D} {kw}", max(new), 3000, **kw) > 0


@pytest.mark.parametrize("kw", [{}, dict(window=300), dict(causal=False), dict(softcap=6.0, alibi=True), dict(prefix=True)],
                         ids=str)
@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (256, BF16), (128, FP32)])
def test_key_shares_of_the_tiled_kernel(D, dtype, kw):
    new = [70, 1, 0, 40, 5]
    s = make([2500, 300, 0, 35, 900], 8, 4, D, 16, "e5m2", dtype, seed=D, new=new)
    kw = dict(kw)
    if kw.get("alibi"):
        kw["alibi"] = torch.linspace(0.001, 1.0, 8)
    if kw.get("prefix"):
        kw["prefix"] = torch.tensor([2480, 400, 3, 30, 0], dtype=torch.int32)
    assert prefill(s, f"key shares D={D} {dtype} {kw}", 70, 2500, **kw) > 0


@pytest.mark.parametrize("max_q,max_len", [(17, 2500), (70, 300), (70, 0), (33, 100000), (5000, 2500)])
def test_key_shares_with_wrong_hints(max_q, max_len):
    new = [170, 1, 0, 40, 5]
    s = make([2500, 300, 0, 35, 900], 8, 4, 128, 16, "e4m3", BF16, seed=4, new=new, width_extra=300)
    prefill(s, f"hints {max_q} {max_len}", max_q, max_len)


@pytest.mark.parametrize("group", [31, 32, 40, 128, 130])
@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, FP16), (256, BF16)])
def test_decode_with_many_heads_on_a_kv_head(group, D, dtype):
    """From 32 (64) query rows a KV head on, decode takes the tiled kernel, with lse and empty sequences."""
    s = make([2000, 0, 1, 130], group, 1, D, 16, "e5m2", dtype, seed=group)
    decode(s, f"group {group} D={D} {dtype}", 2000)
    decode(s, f"group {group} D={D} {dtype} window", 2000, window=200)
    decode(s, f"group {group} D={D} {dtype} short", 100)


def test_arguments_by_name():
    s = make([50, 7], 4, 2, 64, 16, "e5m2", BF16, seed=1)
    q, cache, table, lens, scales = arguments(s)
    a = fp8.fp8_attn_decode_paged(q, cache, table, lens, scales, 16)
    b = fp8.fp8_attn_decode_paged(q=q, cache=cache, block_table=table, seq_lens=lens, scales=scales, block_size=16)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("new", [[3, 2], [90, 60]])
def test_two_streams_with_their_own_workspaces(new):
    """Two calls at once: each with its own workspace, results as alone."""
    s = make([9000, 5000], 8, 4, 128, 16, "e5m2", BF16, seed=2, new=new)
    args = [t.to(DEV) for t in (s["q"], s["cu"], s["cache"], s["table"], s["lens"], s["scales"])]
    call = dict(max_q=max(new), max_len=9000)
    alone = fp8.fp8_attn_prefill_paged(*args, 16, **call)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(fp8.fp8_attn_prefill_paged(*args, 16, **call))
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, alone)


@pytest.mark.parametrize("max_q", [16384, 600])
def test_many_sequences_and_a_long_one(max_q):
    """Column tiles of a batch of mostly empty sequences, as many sequences as rows: the launch goes by the rows, where
    tiles for max_q rows of every sequence would be 2^24 workgroups and more; rows behind the last sequence stay."""
    B, rows = 16384, 16384
    new = [0] * B
    new[0], new[63], new[64], new[4095], new[4096], new[9000], new[B - 1] = 3, 130, 1, 64, 600, 129, 200
    lens = [0] * B
    for b, n in enumerate(new):
        lens[b] = n + n // 3
    s = make(lens, 8, 8, 64, 16, "e5m2", BF16, seed=22, new=new)
    owned = sum(new)
    q, cache, table, lens_d, scales = arguments(s)
    q = torch.cat([q, torch.zeros((rows - owned, 8, 64), dtype=BF16, device=DEV)])
    for max_len in (800, 8000):  # without and with shares of the keys
        log(f"  many sequences, max_q {max_q}, max_len {max_len}")
        out = torch.full((rows, 8, 64), -5.0, dtype=BF16, device=DEV)
        lse = torch.full((rows, 8), 7.0, dtype=torch.float32, device=DEV)
        fp8.fp8_attn_prefill_paged(q, s["cu"].to(DEV), cache, table, lens_d, scales, 16, max_q=max_q, max_len=max_len,
                                   out=out, lse=lse)
        torch.cuda.synchronize()
        want, want_lse, tol = reference(s)
        assert_close(out[:owned], want, tol, "owned rows")
        assert_lse(lse[:owned], want_lse, s, "owned rows")
        assert bool((out[owned:] == -5).all()) and bool((lse[owned:] == 7).all())


def test_more_sequences_than_a_grid_has_workgroups():
    """2^24 + 37 sequences of one key or none: the last ones are taken in turn."""
    B, D = (1 << 24) + 37, 64
    s = make([1], 1, 1, D, 1, "e4m3", BF16, seed=23)
    q = torch.ones((B, 1, D), dtype=BF16, device=DEV)
    table = torch.full((B, 1), int(s["table"][0, 0]), dtype=torch.int32, device=DEV)
    lens = torch.ones(B, dtype=torch.int32, device=DEV)
    lens[torch.arange(3, B, 7, device=DEV)] = 0
    out = torch.full((B, 1, D), 7.0, dtype=BF16, device=DEV)
    fp8.fp8_attn_decode_paged(q, s["cache"].to(DEV), table, lens, s["scales"].to(DEV), 1, fmt="e4m3", max_len=1, out=out)
    torch.cuda.synchronize()
    want, _, tol = reference(s, lse=False)
    row, some = out[0].clone(), (lens > 0)[:, None, None]
    assert_close(row[None], want, tol, "one key")
    assert bool((out == torch.where(some, row, torch.zeros_like(row))).all())


@pytest.mark.parametrize("max_len", [0, 600, 1000, 3000])
@pytest.mark.parametrize("D,Hq,Hkv,dtype", [(128, 16, 4, BF16), (64, 6, 3, FP32), (256, 8, 2, BF16)])
def test_uneven_new_tokens_without_a_hint(D, Hq, Hkv, dtype, max_len):
    """Mostly one new token a sequence, some with none, one with many, and no bound told: by their mean they take the
    streaming form, and the long one is computed whole."""
    new = [1] * 70
    new[3], new[40], new[41], new[69] = 0, 45, 0, 7
    lens = [(37 * b) % 300 + n for b, n in enumerate(new)]
    lens[5], lens[40], lens[60] = 2700, 900, 0
    s = make(lens, Hq, Hkv, D, 16, "e5m2", dtype, seed=D, new=new)
    prefill(s, f"uneven D={D} {dtype} max_len {max_len}", 0, max_len)
    prefill(s, f"uneven D={D} {dtype} max_len {max_len} window", 0, max_len, window=100)


def test_even_drafted_tokens_without_a_hint():
    s = make([(61 * b) % 900 + 4 for b in range(32)], 32, 8, 128, 16, "e5m2", BF16, seed=33, new=[4] * 32)
    prefill(s, "32 x 4, no hints", 0, 0)


def test_none_turns_a_score_option_off():
    s = make([50, 7], 4, 2, 64, 16, "e5m2", BF16, seed=1, new=[2, 1])
    q, cache, table, lens, scales = arguments(s)
    off = dict(softcap=None, alibi_slopes=None, window=None, sm_scale=None, max_len=None)
    a = fp8.fp8_attn_decode_paged(q[:2], cache, table, lens, scales, 16)
    b = fp8.fp8_attn_decode_paged(q[:2], cache, table, lens, scales, 16, **off)
    c = fp8.fp8_attn_prefill_paged(q, s["cu"].to(DEV), cache, table, lens, scales, 16)
    d = fp8.fp8_attn_prefill_paged(q, s["cu"].to(DEV), cache, table, lens, scales, 16, prefix_lens=None, max_q=None, **off)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(c, d)


@pytest.mark.parametrize("max_len", [400, 8000])
@pytest.mark.parametrize("B", [2, 64, 65, 130, 1024, 1025])
def test_column_tiles_over_batches(B, max_len):
    """A workgroup finds its column tile by adding up the sequences' tiles, 64 at a time, or, for more than 1024 of them,
    by their first columns: sequences of none, one and many tiles, empty ones first and last, rows before and behind."""
    new = [0] * B
    for b, n in ((B // 3, 70), (B // 2, 300), (B - 2, 1), (B // 2 + 1, 64)):
        new[min(b, B - 1)] = n
    for b in range(7, B, 61):
        new[b] = b % 9
    lens = [n + (b % 5) * 20 if n else 0 for b, n in enumerate(new)]
    s = make(lens, 6, 3, 64, 16, "e5m2", BF16, seed=B, new=new)
    first, owned = 5, sum(new)
    s["q"] = torch.cat([torch.ones((first, 6, 64), dtype=BF16), s["q"], torch.ones((7, 6, 64), dtype=BF16)])
    s["cu"] = s["cu"] + first
    q, cache, table, lens_d, scales = arguments(s)
    log(f"  tiles of {B} sequences, max_len {max_len}")
    out = torch.full(q.shape, -5.0, dtype=BF16, device=DEV)
    fp8.fp8_attn_prefill_paged(q, s["cu"].to(DEV), cache, table, lens_d, scales, 16, max_q=300, max_len=max_len, out=out)
    torch.cuda.synchronize()
    want, _, tol = reference(s, lse=False)
    rows = slice(first, first + owned)
    assert_close(out[rows], want[rows], tol[rows], "owned rows")
    assert bool((out[:first] == -5).all()) and bool((out[first + owned:] == -5).all())
