"""Cases of the operators around the experts' and the feed-forward products: from a router's choice to the layer's output.

  sort      the tokens' chosen experts in the order of the experts: offsets, rows and the way back
  permute   tokens (or their FP8 codes and scales) moved into that order
  combine   the experts' rows back to their tokens, weighted, summed, on top of a residual
  grad      the gradient of combine: of the experts' rows and of the weights
  gemm      scaled FP8 product with bias, activation and residual in its epilogue
  grouped   the same per expert over sorted rows
  quantize  (gated) activation of a product's rows, quantized per token for the next product

`own` false: the operators in elementary torch operations, in fp32 whatever the inputs' type, rounded once at the end.
`own` true: the calls of this package.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
E4M3, TOP = torch.float8_e4m3fn, 448.0
DEVICE = "cuda"


# ---------------------------------------------------------------- cases ----


def _sort(name, tokens, topk, experts, padded, dropped, wide):
    return {"name": name, "op": "sort", "tokens": tokens, "topk": topk, "experts": experts, "padded": padded,
            "dropped": dropped, "wide": wide}


def _move(name, op, tokens, topk, experts, width, kind, to, padded=0, dropped=0.0, weights=True, residual=False):
    return {"name": name, "op": op, "tokens": tokens, "topk": topk, "experts": experts, "width": width, "type": kind,
            "to": to, "padded": padded, "dropped": dropped, "weights": weights, "residual": residual}


def _gemm(name, m, n, k, bias, act, residual, to):
    return {"name": name, "op": "gemm", "m": m, "n": n, "k": k, "bias": bias, "act": act, "residual": residual, "to": to}


def _grouped(name, tokens, topk, experts, n, k, bias, act, to, padded=0):
    return {"name": name, "op": "grouped", "tokens": tokens, "topk": topk, "experts": experts, "n": n, "k": k,
            "bias": bias, "act": act, "to": to, "padded": padded, "dropped": 0.0}


def _quantize(name, rows, width, act, gated, kind, live):
    return {"name": name, "op": "quantize", "rows": rows, "width": width, "act": act, "gated": gated, "type": kind,
            "live": live}


def listed():
    return [
        # a decode step of eight sequences: latency is all there is
        _sort("sort-decode-8x8", 8, 8, 64, 0, 0.0, False),
        # the benchmark's expert layer: 4096 tokens, 8 of 64 experts each, ids as a top-k call leaves them
        _sort("sort-4096x8", 4096, 8, 64, 0, 0.0, True),
        # a long prefill over many experts, its buffer's last tokens padding, some choices dropped over capacity
        _sort("sort-32768x8-padded", 32768, 8, 256, 1500, 0.02, False),
        # FP8 codes and scales of the benchmark's tokens laid out by expert, as a send buffer has them
        _move("permute-codes-4096x8", "permute", 4096, 8, 64, 7168, "e4m3", "e4m3"),
        # the benchmark's experts' outputs back to 4096 tokens, beside the residual stream
        _move("combine-4096x8", "combine", 4096, 8, 64, 7168, "bf16", "bf16", residual=True),
        # a training step's gradients at an odd width with dropped choices
        _move("grad-fp16-1777x6", "grad", 1777, 6, 40, 4999, "fp16", "fp16", padded=30, dropped=0.05),
        # decode of the 8B up-projection with a bias and an exact gelu
        _gemm("gemm-decode-8", 8, 14336, 4096, True, "gelu", False, "bf16"),
        # a chunk of a prompt at odd sizes into an fp32 residual stream
        _gemm("gemm-777-fp32", 777, 5003, 2064, True, "none", True, "fp32"),
        # the benchmark's prefill, everything in the epilogue
        _gemm("gemm-8192", 8192, 8192, 8192, True, "gelu_tanh", True, "bf16"),
        # the benchmark's experts with a bias each and a silu
        _grouped("grouped-4096x8", 4096, 8, 64, 2048, 7168, True, "silu", "bf16"),
        # decode of the 70B feed-forward: gate and up side by side, for the down-projection
        _quantize("quantize-decode-64", 64, 28672, "silu", True, "bf16", 64),
        # the experts' hidden rows between their two products, the last ones of no expert
        _quantize("quantize-32768", 32768, 2048, "silu", True, "bf16", 32003),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "permute", "combine", "grad", "gemm", "gemm", "gemm", "grouped", "quantize", "quantize"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
    if op == "gemm":
        m, n, k = _log_int(rng, 1, 8192), _log_int(rng, 16, 16384), 16 * _log_int(rng, 4, 1024)
        while m * n * k > 8192 ** 3 // 4:
            m, n = max(1, m * 3 // 4), max(1, n * 3 // 4)
        return _gemm("", m, n, k, rng.random() < 0.7, act, rng.random() < 0.5, kind)
    if op == "quantize":
        width = 16 * _log_int(rng, 1, 2048)
        rows = _log_int(rng, 1, max(2, min(32768, 32768 * 2048 // width)))
        return _quantize("", rows, width, act, rng.random() < 0.6, kind, rng.choice([rows, rng.randint(0, rows)]))
    tokens, experts = _log_int(rng, 1, 16384), _log_int(rng, 1, 256)
    topk = rng.randint(1, min(experts, 10))
    padded, dropped = rng.choice([0, rng.randint(0, tokens // 2)]), rng.choice([0.0, 0.0, 0.1])
    if op == "sort":
        return _sort("", tokens, topk, experts, padded, dropped, rng.random() < 0.5)
    if op == "grouped":
        experts = min(experts, 64)
        topk = min(topk, experts)
        n, k = _log_int(rng, 16, 4096), 16 * _log_int(rng, 8, 448)
        while tokens * topk * n * k > 32768 * 2048 * 7168 // 4:
            tokens, n = max(1, tokens * 3 // 4), max(16, n * 3 // 4)
        return _grouped("", tokens, topk, experts, n, k, rng.random() < 0.7, act, kind, min(padded, tokens // 2))
    width = _log_int(rng, 8, 8192)
    if op == "permute":
        kind = rng.choice(["e4m3", "e4m3", kind])
    while tokens * topk * width * SIZES[kind] > 4096 * 8 * 7168:
        tokens = max(1, tokens * 3 // 4)
        width = max(8, width * 3 // 4)
    padded = min(padded, tokens // 2)
    to = rng.choice([kind, "fp32"]) if op == "combine" else kind
    return _move("", op, tokens, topk, experts, width, kind, to, padded, dropped,
                 op == "grad" or op == "combine" and rng.random() < 0.8, op == "combine" and rng.random() < 0.5)


# ---------------------------------------------------------------- inputs ----


def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEVICE)


def _codes(g, rows, cols):
    """E4M3 codes as absmax scales leave them: the largest of a row of normal values is the format's."""
    out = torch.empty((rows, cols), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 28) // max(1, cols))
    for r in range(0, rows, step):
        x = _randn(g, min(step, rows - r), cols).mul_(TOP / 4.2).clamp_(-TOP, TOP)
        out[r:r + step] = x.to(E4M3).view(torch.uint8)
    return out


def _popularity(experts):
    p = torch.arange(1, experts + 1, dtype=torch.float64) ** -1.1
    return p / p.sum()


def _choices(g, case):
    """int64 [tokens, topk]: distinct experts a token, popular ones more often; -1 for padding and dropped choices."""
    tokens, experts, topk = case["tokens"], case["experts"], case["topk"]
    order = torch.randperm(experts, generator=g, device=DEVICE)
    weight = _popularity(experts).float().to(DEVICE)[order]
    noise = torch.rand((tokens, experts), generator=g, device=DEVICE).clamp_(1e-9, 1 - 1e-6)
    ids = (weight.log() - (-noise.log()).log()).topk(topk, 1).indices
    if case["dropped"]:
        ids[torch.rand((tokens, topk), generator=g, device=DEVICE) < case["dropped"]] = -1
    if case["padded"]:
        ids[tokens - case["padded"]:] = -1
    return ids


def _sorted(ids, experts):
    """(offsets, row_token, row_of) of the choices ids [tokens, topk], ties in the tokens' order."""
    tokens, topk = ids.shape
    flat = ids.reshape(-1).long()
    live = (flat >= 0) & (flat < experts)
    key = torch.where(live, flat, experts)
    order = torch.argsort(key, stable=True)
    counts = (key[:, None] == torch.arange(experts, device=ids.device)).sum(0) if key.numel() * experts < 1 << 24 else \
        torch.bincount(key, minlength=experts + 1)[:experts]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    at = torch.arange(flat.numel(), device=ids.device)
    row_of = torch.empty_like(order)
    row_of[order] = at
    row_of = torch.where(live, row_of, -1).int().view(tokens, topk)
    row_token = torch.where(at < offsets[-1], order // topk, -1).int()
    return offsets, row_token, row_of


def _prepare_sort(case, g):
    ids = _choices(g, case)
    return {"ids": ids if case["wide"] else ids.int()}


def _prepare_move(case, g):
    tokens, width, topk = case["tokens"], case["width"], case["topk"]
    rows = tokens * topk
    _, _, row_of = _sorted(_choices(g, case), case["experts"])
    s = {"row_of": row_of, "rows": rows}
    kind = TYPES.get(case["type"])
    if case["op"] == "permute":
        if case["type"] == "e4m3":
            s["x"], s["s_tok"] = _codes(g, tokens, width), _randn(g, tokens).mul(0.2).exp().mul(4.2 / TOP)
            s["s_out"] = torch.zeros(rows, device=DEVICE)
        else:
            s["x"], s["s_tok"], s["s_out"] = _randn(g, tokens, width).to(kind), None, None
        s["out"] = torch.zeros((rows, width), dtype=s["x"].dtype, device=DEVICE)
        return s
    s["weights"] = torch.softmax(_randn(g, tokens, topk), 1) if case["weights"] else None
    s["y"] = _randn(g, rows, width).to(kind)
    if case["op"] == "combine":
        s["residual"] = _randn(g, tokens, width).mul(3).to(TYPES[case["to"]]) if case["residual"] else None
    else:
        s["dout"] = _randn(g, tokens, width).to(kind)
        s["dy"] = torch.zeros((rows, width), dtype=kind, device=DEVICE)
    return s


def _product_weights(g, n, k, experts=None):
    """Codes and channel scales of weights whose product with activations of unit spread has about unit spread too."""
    e = experts or 1
    qw = _codes(g, e * n, k)
    s_ch = _randn(g, e * n).mul(0.5).exp().mul(4.2 / TOP * 1.2 / math.sqrt(max(1, k)))
    return (qw.view(e, n, k), s_ch.view(e, n)) if experts else (qw, s_ch)


def _prepare_gemm(case, g):
    m, n, k = case["m"], case["n"], case["k"]
    qw, s_ch = _product_weights(g, n, k)
    return {"qa": _codes(g, m, k), "s_tok": _randn(g, m).mul(0.2).exp().mul(4.2 / TOP), "qw": qw, "s_ch": s_ch,
            "bias": _randn(g, n).mul(0.5) if case["bias"] else None,
            "residual": _randn(g, m, n).mul(2).to(TYPES[case["to"]]) if case["residual"] else None}


def _prepare_grouped(case, g):
    n, k, experts, tokens = case["n"], case["k"], case["experts"], case["tokens"]
    offsets, row_token, _ = _sorted(_choices(g, case), experts)
    qw, s_ch = _product_weights(g, n, k, experts)
    return {"qa": _codes(g, tokens, k), "s_tok": _randn(g, tokens).mul(0.2).exp().mul(4.2 / TOP), "qw": qw,
            "s_ch": s_ch, "offsets": offsets, "row_token": row_token, "most": int((offsets[1:] - offsets[:-1]).max()),
            "bias": _randn(g, experts, n).mul(0.5) if case["bias"] else None,
            "y": torch.zeros((tokens * case["topk"], n), dtype=TYPES[case["to"]], device=DEVICE)}


def _prepare_quantize(case, g):
    rows, width = case["rows"], case["width"]
    h = _randn(g, rows, width * 2 if case["gated"] else width)
    h *= _randn(g, h.shape[1]).mul(0.5).exp()  # channels differ in spread
    return {"h": h.to(TYPES[case["type"]]), "q": torch.zeros((rows, width), dtype=torch.uint8, device=DEVICE),
            "scales": torch.zeros(rows, device=DEVICE),
            "live": torch.tensor([case["live"]], dtype=torch.int32, device=DEVICE)}


PREPARE = {"sort": _prepare_sort, "permute": _prepare_move, "combine": _prepare_move, "grad": _prepare_move,
           "gemm": _prepare_gemm, "grouped": _prepare_grouped, "quantize": _prepare_quantize}


def prepare(case, seed):
    s = PREPARE[case["op"]](case, _gen(seed))
    s["case"] = case
    return s


# ---------------------------------------------------------------- the operators, plain ----


def _act(x, act):
    if act == "relu":
        return x.clamp_min(0.0)
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _sort_plain(s):
    return _sorted(s["ids"], s["case"]["experts"])


def _permute_plain(s):
    rows = s["row_of"].reshape(-1).long()
    live = rows >= 0
    rows, token = rows[live], (torch.arange(live.numel(), device=DEVICE) // s["case"]["topk"])[live]
    s["out"][rows] = s["x"][token]
    if s["s_tok"] is None:
        return s["out"]
    s["s_out"][rows] = s["s_tok"][token]
    return s["out"].view(E4M3), s["s_out"]


def _combine_plain(s):
    live = s["row_of"] >= 0
    y = s["y"][s["row_of"].clamp_min(0).long()].float()
    if s["weights"] is not None:
        y = y * s["weights"][..., None]
    y = torch.where(live[..., None], y, 0.0).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(TYPES[s["case"]["to"]])


def _grad_plain(s):
    live = s["row_of"] >= 0
    at = s["row_of"].clamp_min(0).long()
    d = s["dout"].float()[:, None, :]
    dw = torch.where(live, (s["y"][at].float() * d).sum(-1), 0.0)
    dy = (s["weights"][..., None] * d).to(s["dy"].dtype)
    s["dy"][at[live]] = dy[live]
    return s["dy"], dw


def _gemm_plain(s):
    y = torch.matmul(s["qa"].view(E4M3).float(), s["qw"].view(E4M3).float().t())
    y = y * (s["s_tok"][:, None] * s["s_ch"])
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _act(y, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(TYPES[s["case"]["to"]])


def _grouped_plain(s):
    offsets = s["offsets"].long()
    at = offsets[:-1, None] + torch.arange(s["most"], device=DEVICE)  # [experts, most] rows, padded
    live = at < offsets[1:, None]
    token = s["row_token"].long()[torch.where(live, at, 0)].clamp_min(0)
    x = s["qa"].view(E4M3).float()[token]
    y = torch.matmul(x, s["qw"].view(E4M3).float().transpose(1, 2))
    y = y * (s["s_tok"][token][..., None] * s["s_ch"][:, None, :])
    if s["bias"] is not None:
        y = y + s["bias"][:, None, :]
    s["y"][at[live]] = _act(y[live], s["case"]["act"]).to(s["y"].dtype)
    return s["y"]


def _quantize_plain(s):
    case = s["case"]
    width, live = case["width"], case["live"]
    h = s["h"][:live].float()
    v = _act(h[:, :width], case["act"])
    if case["gated"]:
        v = v * h[:, width:]
    scale = (v.abs().amax(1) / TOP).clamp_min(1e-12)
    s["q"][:live] = (v / scale[:, None]).clamp(-TOP, TOP).to(E4M3).view(torch.uint8)
    s["scales"][:live] = scale
    return s["q"].view(E4M3), s["scales"]


# ---------------------------------------------------------------- the operators, by this package ----


def _package():
    import fp8_w8a8_quantized_quantize_amd as fp8

    return fp8


def _sort_own(s):
    return _package().fp8_moe_sort(s["ids"], s["case"]["experts"])


def _permute_own(s):
    got = _package().fp8_moe_permute(s["x"], s["row_of"], s_tok=s["s_tok"], out=s["out"], s_out=s["s_out"])
    return got if s["s_tok"] is None else (got[0].view(E4M3), got[1])


def _combine_own(s):
    return _package().fp8_moe_combine(s["y"], s["row_of"], weights=s["weights"], residual=s["residual"],
                                      out_dtype=TYPES[s["case"]["to"]])


def _grad_own(s):
    return _package().fp8_moe_combine_grad(s["dout"], s["y"], s["row_of"], weights=s["weights"], dy=s["dy"])


def _gemm_own(s):
    return _package().fp8_gemm_scaled_act(s["qa"], s["s_tok"], s["qw"], s["s_ch"], bias=s["bias"], act=s["case"]["act"],
                                          residual=s["residual"], y_dtype=TYPES[s["case"]["to"]])


def _grouped_own(s):
    return _package().fp8_gemm_grouped_scaled_act(s["qa"], s["s_tok"], s["row_token"], s["offsets"], s["qw"], s["s_ch"],
                                                  bias=s["bias"], act=s["case"]["act"], y=s["y"])


def _quantize_own(s):
    case = s["case"]
    q, scales = _package().fp8_act_quantize(s["h"], act=case["act"], gated=case["gated"], q=s["q"], scales=s["scales"],
                                            live_rows=s["live"])
    return q.view(E4M3), scales


def run(state):
    op = state["case"]["op"]
    if own:
        return {"sort": _sort_own, "permute": _permute_own, "combine": _combine_own, "grad": _grad_own,
                "gemm": _gemm_own, "grouped": _grouped_own, "quantize": _quantize_own}[op](state)
    return {"sort": _sort_plain, "permute": _permute_plain, "combine": _combine_plain, "grad": _grad_plain,
            "gemm": _gemm_plain, "grouped": _grouped_plain, "quantize": _quantize_plain}[op](state)


# ---------------------------------------------------------------- what a pass needs ----


def work(case):
    op = case["op"]
    if op == "gemm":
        m, n, k, size = case["m"], case["n"], case["k"], SIZES[case["to"]]
        return {"bytes": m * k + n * k + 4 * (m + n + n * case["bias"]) + m * n * size * (1 + case["residual"]),
                "flops": 2 * m * n * k}
    if op == "quantize":
        width = case["width"]
        return {"bytes": case["live"] * (width * (1 + case["gated"]) * SIZES[case["type"]] + width + 4) + 4,
                "flops": case["live"] * width * 12}
    tokens, topk, experts = case["tokens"], case["topk"], case["experts"]
    rows = tokens * topk
    live = int((tokens - case["padded"]) * topk * (1 - case["dropped"]))
    if op == "sort":
        return {"bytes": rows * (16 if case["wide"] else 12) + 4 * (experts + 1), "flops": rows}
    if op == "grouped":
        n, k = case["n"], case["k"]
        # the weights of the experts that are chosen at all
        chosen = float((1 - (1 - (topk * _popularity(experts)).clamp_max(1.0)) ** (tokens - case["padded"])).sum())
        return {"bytes": int(chosen * n * (k + 4 + 4 * case["bias"])) + tokens * (k + 4) + 4 * rows
                + live * n * SIZES[case["to"]], "flops": 2 * live * n * k}
    width, size = case["width"], SIZES[case["type"]]
    if op == "permute":
        scales = 4 if case["type"] == "e4m3" else 0
        return {"bytes": (tokens - case["padded"] + live) * (width * size + scales) + 4 * rows, "flops": 0}
    if op == "combine":
        out = tokens * width * SIZES[case["to"]]
        return {"bytes": live * width * size + out * (1 + case["residual"]) + rows * (4 + 4 * case["weights"]),
                "flops": 2 * live * width}
    return {"bytes": (tokens - case["padded"] + 2 * live) * width * size + 12 * rows, "flops": 3 * live * width}


# ---------------------------------------------------------------- the definition, in 64 bits ----


def _exact_act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, 0.0)
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return 0.5 * x * torch.special.erfc(-x / math.sqrt(2.0))
    if act == "gelu_tanh":
        return x * torch.sigmoid(math.sqrt(8.0 / math.pi) * (x + 0.044715 * x ** 3))
    return x


def _round_e4m3(x):
    """The nearest E4M3 value to each of x (float64), ties to even, held at the largest finite one."""
    x = x.clamp(-TOP, TOP)
    step = torch.exp2((torch.frexp(x)[1].double() - 1).clamp_min(-6) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    op = case["op"]
    if op == "sort":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "quantize":
        live, width = case["live"], case["width"]
        h = s["h"][:live].double()
        v = _exact_act(h[:, :width], case["act"])
        if case["gated"]:
            v = v * h[:, width:]
        scales, q = s["scales"].double(), s["q"].double()
        scales[:live] = torch.maximum(v.abs().amax(1) / TOP, torch.tensor(1e-12, device=DEVICE).double())
        q[:live] = _round_e4m3(v / scales[:live, None])
        return q, scales
    if op == "gemm":
        y = (s["qa"].view(E4M3).double() * s["s_tok"].double()[:, None]) @ s["qw"].view(E4M3).double().t()
        y = y * s["s_ch"].double()
        y = _exact_act(y if s["bias"] is None else y + s["bias"].double(), case["act"])
        return y if s["residual"] is None else y + s["residual"].double()
    if op == "grouped":
        out = s["y"].double()
        ends = s["offsets"].tolist()
        x = s["qa"].view(E4M3).double() * s["s_tok"].double()[:, None]
        for e in range(case["experts"]):
            a, b = ends[e], ends[e + 1]
            if b > a:
                w = s["qw"][e].view(E4M3).double() * s["s_ch"][e].double()[:, None]
                y = x[s["row_token"][a:b].long()] @ w.t()
                out[a:b] = _exact_act(y if s["bias"] is None else y + s["bias"][e].double(), case["act"])
        return out
    topk = case["topk"]
    if op == "permute":
        out = (s["x"].view(E4M3) if case["type"] == "e4m3" else s["x"]).double()
        out = out.new_zeros((s["rows"], case["width"])).index_copy_(0, *_live(s["row_of"], out))
        if s["s_tok"] is None:
            return out
        scales = s["s_tok"].double()[:, None]
        return out, scales.new_zeros((s["rows"], 1)).index_copy_(0, *_live(s["row_of"], scales))[:, 0]
    if op == "combine":
        out = torch.zeros((case["tokens"], case["width"]), dtype=torch.float64, device=DEVICE)
        if s["residual"] is not None:
            out += s["residual"].double()
        for j in range(topk):
            at = (s["row_of"][:, j] >= 0).nonzero()[:, 0]
            y = s["y"][s["row_of"][at, j].long()].double()
            out[at] += y if s["weights"] is None else y * s["weights"][at, j].double()[:, None]
        return out
    dy, dw = s["dy"].double(), torch.zeros((case["tokens"], topk), dtype=torch.float64, device=DEVICE)
    for j in range(topk):
        at = (s["row_of"][:, j] >= 0).nonzero()[:, 0]
        d, rows = s["dout"][at].double(), s["row_of"][at, j].long()
        dy[rows] = d * s["weights"][at, j].double()[:, None]
        dw[at, j] = (d * s["y"][rows].double()).sum(1)
    return dy, dw


def _live(row_of, x):
    """(rows, the tokens' values) of the choices that are not dropped."""
    t, j = (row_of >= 0).nonzero(as_tuple=True)
    return row_of[t, j].long(), x[t]
