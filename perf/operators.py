"""Cases of the paged FP8 attention operators: what a serving step does between the QKV projection and
the output projection of one layer, against the FP8 KV cache.

  append   rotate the queries and keys by their positions, quantize keys and values into cache pages
  decode   attention of one new token per sequence over its pages
  prefill  attention of several new tokens per sequence (a prompt, a chunk of one, drafted tokens)

`own` false: the operators in elementary torch operations, in fp32 whatever the inputs' type, rounded
once at the end.  `own` true: the calls of this package.  The cache is the package's: uint8
[num_blocks * block, 2 * kv_heads * dim], a row's K heads first and its V heads after them, one fp32
scale per channel.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
DEVICE = "cuda"


# ---------------------------------------------------------------- cases ----


def _append(name, tokens, q_heads, kv_heads, dim, rot, interleaved, kind, fmt, padded):
    return {"name": name, "op": "append", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "interleaved": interleaved, "type": kind, "format": fmt, "padded": padded}


def _decode(name, batch, shortest, longest, q_heads, kv_heads, dim, block, kind, fmt, softcap=0.0, alibi=False,
            window=0, lse=False):
    return {"name": name, "op": "decode", "batch": batch, "shortest": shortest, "longest": longest,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "block": block, "type": kind, "format": fmt,
            "softcap": softcap, "alibi": alibi, "window": window, "lse": lse}


def _prefill(name, batch, new_min, new_max, past_max, q_heads, kv_heads, dim, block, kind, fmt, causal=True,
             prefix=False, softcap=0.0, alibi=False, window=0):
    return {"name": name, "op": "prefill", "batch": batch, "new_min": new_min, "new_max": new_max,
            "past_max": past_max, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "block": block, "type": kind,
            "format": fmt, "causal": causal, "prefix": prefix, "softcap": softcap, "alibi": alibi, "window": window}


def listed():
    return [
        # one sequence decoding: a single token's heads, launch latency is all there is
        _append("append-one", 1, 32, 8, 128, 128, False, "bf16", "e5m2", 0),
        # a decode step of a full batch, its last slots padding as a captured graph has them
        _append("append-batch-256", 256, 64, 8, 128, 128, False, "bf16", "e5m2", 16),
        # a ragged prompt of a model with wide heads, of which half are rotated in neighbouring pairs
        _append("append-fp16-1777", 1777, 24, 3, 256, 128, True, "fp16", "e4m3", 5),
        # the benchmark's 32768-token prefill of one layer with 8 KV heads of 128
        _append("append-prefill-32k", 32768, 64, 8, 128, 128, False, "bf16", "e5m2", 0),
        # one short conversation: latency
        _decode("decode-one-577", 1, 577, 577, 32, 8, 128, 16, "bf16", "e5m2"),
        # a serving batch, lengths spread from empty to a few thousand
        _decode("decode-batch-64", 64, 0, 4096, 64, 8, 128, 16, "bf16", "e5m2"),
        # one long document: the cache's length is all the parallelism there is
        _decode("decode-long-128k", 1, 131072, 131072, 64, 8, 128, 64, "bf16", "e5m2", lse=True),
        # a large batch of long contexts: the cache's bytes
        _decode("decode-large-48x32k", 48, 4096, 32768, 64, 8, 128, 32, "bf16", "e4m3"),
        # capped scores over a sliding window, wide heads, pages of an odd size
        _decode("decode-fp16-capped", 19, 1, 9001, 16, 2, 256, 24, "fp16", "e4m3", softcap=50.0, window=4096,
                lse=True),
        # drafted tokens being verified: four new ones per sequence over a long cache
        _prefill("verify-32x4", 32, 4, 4, 8192, 32, 8, 128, 16, "bf16", "e5m2"),
        # a whole prompt of one layer with 64 query heads
        _prefill("prefill-8192", 1, 8192, 8192, 0, 64, 8, 128, 16, "bf16", "e5m2"),
        # ragged chunks over earlier pages, a prefix seen by every token, a bias falling with distance
        _prefill("chunks-fp16-biased", 6, 100, 3000, 4000, 12, 12, 64, 32, "fp16", "e4m3", prefix=True, alibi=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill"])
    kind, fmt = rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.choice(["e5m2", "e4m3"])
    dim, kv_heads, group = rng.choice([64, 128, 128, 256]), rng.randint(1, 8), rng.randint(1, 16)
    q_heads = kv_heads * group
    block = rng.choice([1, 8, 16, 24, 32, 64, 100, 128])
    bias = {"softcap": rng.choice([0.0, 0.0, 30.0, 50.0]), "alibi": rng.random() < 0.25}
    if op == "append":
        tokens = _log_int(rng, 1, 16000)
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        return _append("", tokens, q_heads, kv_heads, dim, rot, rng.random() < 0.4, kind, fmt,
                       rng.randint(0, tokens // 4))
    if op == "decode":
        batch = _log_int(rng, 1, 128)
        longest = _log_int(rng, 1, max(64, min(65536, (800 << 20) // (batch * 2 * kv_heads * dim))))
        return _decode("", batch, rng.choice([0, min(1, longest), longest // 4 + 1]), longest, q_heads, kv_heads, dim,
                       block, kind, fmt, window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), lse=rng.random() < 0.5,
                       **bias)
    batch = _log_int(rng, 1, 32)
    new = _log_int(rng, 1, max(2, 8192 // batch))
    past = rng.choice([0, _log_int(rng, 1, 8192)])
    while batch * new * (new + past) * q_heads * dim > 8192 * 8192 * 64 * 128 // 8 and past + new > 64:
        new, past = max(1, new * 3 // 4), past * 3 // 4
    causal = rng.random() < 0.8
    return _prefill("", batch, rng.randint(0, new), new, past, q_heads, kv_heads, dim, block, kind, fmt, causal=causal,
                    prefix=causal and rng.random() < 0.3, window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), **bias)


# ---------------------------------------------------------------- inputs ----


def _spread(rng, lo, hi, n):
    """n lengths between lo and hi, over their logarithm, the first of them hi; lo = 0: the last one is empty."""
    got = [hi] + [min(hi, _log_int(rng, max(1, lo), max(1, hi))) for _ in range(n - 1)]
    if lo == 0 and n > 1:
        got[-1] = 0
    return got


def _lengths(case):
    """(new tokens, cache length) of every sequence; the same for every seed."""
    rng = random.Random(case["batch"] * 1000003 + case.get("longest", case.get("new_max")))
    if case["op"] == "decode":
        return None, _spread(rng, case["shortest"], case["longest"], case["batch"])
    new = _spread(rng, case["new_min"], case["new_max"], case["batch"])
    past = [rng.randint(0, case["past_max"]) for _ in new]
    return new, [n + p for n, p in zip(new, past)]


def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _codes(g, rows, cols, fmt):
    """FP8 codes as per-channel absmax scales leave them: the largest of many normal values is the format's."""
    f8, top = FORMATS[fmt]
    out = torch.empty((rows, cols), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 28) // max(1, cols))
    for r in range(0, rows, step):
        x = torch.randn((min(step, rows - r), cols), generator=g, device=DEVICE).mul_(top / 5.5).clamp_(-top, top)
        out[r:r + step] = x.to(f8).view(torch.uint8)
    return out


def _channel_scales(g, cols, fmt):
    """The scales of such codes, for channels whose spread differs as keys' do."""
    return torch.randn(cols, generator=g, device=DEVICE).mul(0.4).exp().mul(5.5 / FORMATS[fmt][1])


def _cos_sin(positions, rot):
    """fp32 [positions, rot]: the cosines, then the sines, of position * 10000^(-2 i / rot)."""
    i = torch.arange(rot // 2, device=DEVICE, dtype=torch.float64)
    a = torch.arange(positions, device=DEVICE, dtype=torch.float64)[:, None] * 10000.0 ** (-2 * i / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _prepare_append(case, seed):
    g, n, dim = _gen(seed), case["tokens"], case["dim"]
    hq, hk = case["q_heads"], case["kv_heads"]
    kind = TYPES[case["type"]]
    qkv = torch.randn((n, (hq + 2 * hk) * dim), generator=g, device=DEVICE).to(kind)  # the projection's output
    block = 16
    slots = (n + block - 1) // block * block + 4 * block
    order = torch.randperm(slots // block, generator=g, device=DEVICE)
    at = torch.arange(n, device=DEVICE)
    slot = (order[at // block] * block + at % block).int()
    if case["padded"]:
        slot[n - case["padded"]:] = -1
    cols = 2 * hk * dim
    rows = _codes(g, slots + 1, cols, case["format"])  # one row past the cache: the plain form drops padding there
    limit = 40000
    return {"case": case, "q": qkv[:, :hq * dim].view(n, hq, dim),
            "k": qkv[:, hq * dim:(hq + hk) * dim].view(n, hk, dim), "v": qkv[:, (hq + hk) * dim:].view(n, hk, dim),
            "positions": torch.randint(0, limit - n, (1,), generator=g, device=DEVICE).add(at).int(),
            "cos_sin": _cos_sin(limit, case["rot"]), "scales": _channel_scales(g, cols, case["format"]),
            "slot_mapping": slot, "rows": rows, "cache": rows[:slots], "q_out": torch.empty((n, hq, dim), dtype=kind, device=DEVICE)}


def _prepare_attention(case, seed):
    g, block = _gen(seed), case["block"]
    hq, hk, dim = case["q_heads"], case["kv_heads"], case["dim"]
    new, lens = _lengths(case)
    pages = [(n + block - 1) // block for n in lens]
    width = max(1, max(pages))
    blocks = sum(pages) + 3
    order = torch.randperm(blocks, generator=g, device=DEVICE)[:sum(pages)].int()
    table = torch.zeros((case["batch"], width), dtype=torch.int32, device=DEVICE)
    live = torch.arange(width, device=DEVICE)[None, :] < torch.tensor(pages, device=DEVICE)[:, None]
    table[live] = order
    rows = case["batch"] if new is None else sum(new)
    s = {"case": case, "cache": _codes(g, blocks * block, 2 * hk * dim, case["format"]),
         "scales": _channel_scales(g, 2 * hk * dim, case["format"]), "block_table": table,
         "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEVICE), "max_len": max(lens),
         "q": torch.randn((rows, hq, dim), generator=g, device=DEVICE).mul(1.4).to(TYPES[case["type"]]),
         "alibi": None, "prefix": None}
    if case["alibi"]:
        s["alibi"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device=DEVICE) / hq)
    if new is not None:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu_q"], s["max_q"] = torch.tensor(cu, dtype=torch.int32, device=DEVICE), max(new)
        if case["prefix"]:
            s["prefix"] = torch.tensor([n * 2 // 3 for n in lens], dtype=torch.int32, device=DEVICE)
    return s


def prepare(case, seed):
    return _prepare_append(case, seed) if case["op"] == "append" else _prepare_attention(case, seed)


# ---------------------------------------------------------------- the operators ----


def _rotate(x, cos, sin, rot, interleaved):
    """x [tokens, heads, dim] in fp32, its first `rot` elements turned by their pair's angle."""
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    c, s = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([c, s], -1).flatten(-2) if interleaved else torch.cat([c, s], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _append_plain(s):
    case, rot = s["case"], s["case"]["rot"]
    f8, top = FORMATS[case["format"]]
    cs = s["cos_sin"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    q = _rotate(s["q"].float(), cos, sin, rot, case["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"].float(), cos, sin, rot, case["interleaved"])
    kv = torch.cat([k.flatten(1), s["v"].float().flatten(1)], 1)
    codes = (kv / s["scales"].clamp_min(1e-12)).clamp(-top, top).to(f8).view(torch.uint8)
    slot = s["slot_mapping"].long()
    s["rows"][torch.where(slot < 0, s["cache"].shape[0], slot)] = codes
    return q, s["cache"].view(f8)


def _append_own(s):
    import fp8_w8a8_quantized_quantize_amd as fp8

    case = s["case"]
    fp8.fp8_kv_append_rope_paged(s["k"], s["v"], s["positions"], s["cos_sin"], s["scales"], s["slot_mapping"],
                                 s["cache"], fmt=case["format"], q=s["q"], q_out=s["q_out"],
                                 interleaved=case["interleaved"])
    return s["q_out"], s["cache"].view(FORMATS[case["format"]][0])


def _keys_values(s):
    """fp32 [batch, kv_heads, length, dim] keys and values of every sequence, as long as the longest."""
    case, block = s["case"], s["case"]["block"]
    at = torch.arange(max(1, s["max_len"]), device=DEVICE)
    slots = s["block_table"].long()[:, at // block] * block + at % block
    kv = s["cache"][slots].view(FORMATS[case["format"]][0]).float() * s["scales"].clamp_min(1e-12)
    kv = kv.view(case["batch"], at.numel(), 2, case["kv_heads"], case["dim"]).permute(2, 0, 3, 1, 4).contiguous()
    return kv[0], kv[1]


def _attend(s, q, position, new):
    """q fp32 [batch, rows, q_heads, dim] at `position` [batch, rows] (rows from `new` on are padding) ->
    (outputs, log-sum-exp); a row that sees no key gives zeros and -inf."""
    case = s["case"]
    b, rows, hq, dim = q.shape
    hk = case["kv_heads"]
    k, v = _keys_values(s)
    n = k.shape[2]
    x = q.view(b, rows, hk, hq // hk, dim).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, dim)
    x = torch.matmul(x, k.transpose(2, 3)).mul_(1.0 / math.sqrt(dim)).view(b, hk, hq // hk, rows, n)
    if case["softcap"]:
        x = torch.tanh(x / case["softcap"]) * case["softcap"]
    at = torch.arange(n, device=DEVICE)
    if s["alibi"] is not None:
        x = x + s["alibi"].view(1, hk, -1, 1, 1) * (at - position[:, None, None, :, None])
    live = (at < s["seq_lens"][:, None, None]) & (torch.arange(rows, device=DEVICE)[None, :, None] < new[:, None, None])
    if case.get("causal", True):
        past = at <= position[..., None]
        live &= past if s["prefix"] is None else past | (at < s["prefix"][:, None, None])
    if case["window"]:
        live &= position[..., None] - at < case["window"]
    x = x.masked_fill_(~live[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(b, hk, -1, n), v).view(b, hk, hq // hk, rows, dim)
    out = out / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).view(b, hq, rows)
    return out.permute(0, 3, 1, 2, 4).reshape(b, rows, hq, dim), lse


def _decode_plain(s):
    position = (s["seq_lens"].long() - 1)[:, None]
    out, lse = _attend(s, s["q"].float()[:, None], position, torch.ones_like(s["seq_lens"]))
    out = out[:, 0].to(s["q"].dtype)
    return (out, lse[:, :, 0]) if s["case"]["lse"] else out


def _decode_own(s):
    import fp8_w8a8_quantized_quantize_amd as fp8

    case, q = s["case"], s["q"]
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if case["lse"] else None
    out = fp8.fp8_attn_decode_paged(q, s["cache"], s["block_table"], s["seq_lens"], s["scales"], case["block"],
                                    fmt=case["format"], max_len=s["max_len"], softcap=case["softcap"],
                                    alibi_slopes=s["alibi"], window=case["window"], lse=lse)
    return (out, lse) if case["lse"] else out


def _prefill_plain(s):
    cu = s["cu_q"].long()
    new = cu[1:] - cu[:-1]
    row = torch.arange(max(1, s["max_q"]), device=DEVICE)
    if not s["q"].shape[0]:
        return s["q"].clone()
    q = s["q"].float()[(cu[:-1, None] + row).clamp_max(s["q"].shape[0] - 1)]
    out, _ = _attend(s, q, s["seq_lens"].long()[:, None] - new[:, None] + row, new)
    t = torch.arange(s["q"].shape[0], device=DEVICE)
    of = (t[:, None] >= cu[None, 1:]).sum(1)
    return out[of, t - cu[of]].to(s["q"].dtype)


def _prefill_own(s):
    import fp8_w8a8_quantized_quantize_amd as fp8

    case = s["case"]
    return fp8.fp8_attn_prefill_paged(s["q"], s["cu_q"], s["cache"], s["block_table"], s["seq_lens"], s["scales"],
                                      case["block"], fmt=case["format"], max_q=s["max_q"], max_len=s["max_len"],
                                      causal=case["causal"], prefix_lens=s["prefix"], softcap=case["softcap"],
                                      alibi_slopes=s["alibi"], window=case["window"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _append_own, "decode": _decode_own, "prefill": _prefill_own}[op](state)
    return {"append": _append_plain, "decode": _decode_plain, "prefill": _prefill_plain}[op](state)


# ---------------------------------------------------------------- what a pass needs ----


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
    hq, hk, dim = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        n = case["tokens"]
        live = n - case["padded"]
        return {"bytes": n * (2 * hq * dim * size + 4 * case["rot"] + 8) + live * 2 * hk * dim * (size + 1) + 8 * hk * dim,
                "flops": n * hq * case["rot"] * 3 + live * hk * (case["rot"] * 3 + 2 * dim)}
    new, lens = _lengths(case)
    window = case["window"] or 1 << 40
    if case["op"] == "decode":
        seen = sum(min(n, window) for n in lens)
        pairs, rows = seen, case["batch"]
    else:
        seen = pairs = 0
        rows = sum(new)
        for n, total in zip(new, lens):
            if not n:
                continue
            past = total - n
            ahead = total * 2 // 3 if case["prefix"] else 0
            first = max(0, past - window + 1)
            seen += total - first
            for i in range(past, total):
                last = max(i + 1, min(ahead, total)) if case["causal"] else total
                pairs += max(0, last - max(0, i - window + 1))
    return {"bytes": seen * 2 * hk * dim + 2 * rows * hq * dim * size + 8 * hk * dim + 4 * (seen // case["block"] + 2 * case["batch"]),
            "flops": 4 * pairs * hq * dim}


# ---------------------------------------------------------------- the definition, in 64 bits ----


def _round_fp8(x, fmt):
    """The nearest value of the format to each of x (float64), ties to even, held at the largest finite one."""
    low, bits, top = (-6, 3, 448.0) if fmt == "e4m3" else (-14, 2, 57344.0)
    x = x.clamp(-top, top)
    e = torch.frexp(x)[1].double() - 1
    step = torch.exp2(e.clamp_min(low) - bits)
    return torch.round(x / step) * step


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    half, dim = case["rot"] // 2, case["dim"]
    at = torch.arange(half, device=DEVICE)
    first, second = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + half)
    angle = s["cos_sin"].double()[s["positions"].long()].unsqueeze(1)
    turned = []
    for x in (s["q"].double(), s["k"].double()):
        y = x.clone()
        y[..., first] = x[..., first] * angle[..., :half] - x[..., second] * angle[..., half:]
        y[..., second] = x[..., first] * angle[..., half:] + x[..., second] * angle[..., :half]
        turned.append(y)
    n = case["tokens"] - case["padded"]
    cache = s["cache"].view(FORMATS[case["format"]][0]).double()
    slot = s["slot_mapping"].long()[:n]
    width = case["kv_heads"] * dim
    scale = s["scales"].double()
    cache[slot, :width] = _round_fp8(turned[1][:n].reshape(n, width) / scale[:width], case["format"])
    cache[slot, width:] = _round_fp8(s["v"][:n].double().reshape(n, width) / scale[width:], case["format"])
    return turned[0], cache


def _exact_attention(case, seed):
    s = _prepare_attention(case, seed)
    new, lens = _lengths(case)
    hq, hk, dim, block = case["q_heads"], case["kv_heads"], case["dim"], case["block"]
    group = hq // hk
    new = [1] * case["batch"] if new is None else new
    out = torch.zeros((sum(new), hq, dim), dtype=torch.float64, device=DEVICE)
    lse = torch.full((sum(new), hq), -math.inf, dtype=torch.float64, device=DEVICE)
    scale = s["scales"].double().view(2, hk, dim)
    row = 0
    for b, (n, total) in enumerate(zip(new, lens)):
        if n and total:
            j = torch.arange(total, device=DEVICE)
            codes = s["cache"][s["block_table"][b].long()[j // block] * block + j % block]
            codes = codes.view(FORMATS[case["format"]][0]).view(total, 2, hk, dim)
            i = torch.arange(total - n, total, device=DEVICE)[:, None]
            seen = j[None, :] <= i if case.get("causal", True) else torch.ones((n, total), dtype=torch.bool, device=DEVICE)
            if s["prefix"] is not None:
                seen = seen | (j < s["prefix"][b])[None, :]
            if case["window"]:
                seen = seen & (i - j[None, :] < case["window"])
            for h in range(hk):
                k = codes[:, 0, h].double() * scale[0, h]
                v = codes[:, 1, h].double() * scale[1, h]
                for g in range(h * group, h * group + group):
                    w = s["q"][row:row + n, g].double() @ k.t() / math.sqrt(dim)
                    if case["softcap"]:
                        w = case["softcap"] * torch.tanh(w / case["softcap"])
                    if s["alibi"] is not None:
                        w = w + s["alibi"][g].double() * (j[None, :] - i)
                    w = torch.where(seen, w, -math.inf)
                    lse[row:row + n, g] = torch.logsumexp(w, 1)
                    w = torch.where(seen.any(1, keepdim=True), torch.softmax(w, 1), 0.0)
                    out[row:row + n, g] = w @ v
        row += n
    return (out, lse) if case["op"] == "decode" and case["lse"] else out


def exact(case, seed):
    return _exact_append(case, seed) if case["op"] == "append" else _exact_attention(case, seed)
