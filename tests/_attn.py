"""Plain 64-bit attention over a paged FP8 cache, and random caches for its tests."""
import math

import numpy as np
import torch

F8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
NAN_CODE = {"e4m3": 0x7F, "e5m2": 0x7D}
EPS_HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make(lens, Hq, Hkv, D, block, fmt, dtype, seed, new=None, extra_pages=3, width_extra=1, dev="cpu"):
    """A cache with `lens` tokens per sequence in permuted pages, every other byte (rows behind a sequence's end,
    pages no sequence owns) a NaN code; queries for `new` rows per sequence (one when None)."""
    g = torch.Generator().manual_seed(seed)
    f8, top = F8[fmt]
    C = 2 * Hkv * D
    pages = [(n + block - 1) // block for n in lens]
    nb = sum(pages) + extra_pages
    order = torch.randperm(nb, generator=g).to(torch.int32)
    width = max(pages + [0]) + width_extra
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    cache = torch.full((nb * block, C), NAN_CODE[fmt], dtype=torch.uint8)
    used = 0
    for b, n in enumerate(lens):
        table[b, :pages[b]] = order[used:used + pages[b]]
        used += pages[b]
        if n:
            j = torch.arange(n)
            slot = table[b, (j // block).long()].long() * block + j % block
            x = (torch.randn((n, C), generator=g) * (top / 5)).clamp(-top, top)
            cache[slot] = x.to(f8).view(torch.uint8)
    scales = (torch.randn(C, generator=g) * 0.4).exp() * (5 / top)
    rows = len(lens) if new is None else sum(new)
    q = (torch.randn((rows, Hq, D), generator=g) * 1.4).to(dtype)
    cu = torch.tensor([0] + list(np.cumsum(new if new is not None else [1] * len(lens))), dtype=torch.int32)
    return dict(q=q, cache=cache, table=table, lens=torch.tensor(lens, dtype=torch.int32), scales=scales, cu=cu,
                block=block, fmt=fmt, Hq=Hq, Hkv=Hkv, D=D)


def reference(s, causal=True, softcap=0.0, alibi=None, window=0, prefix=None, sm_scale=None, lse=True):
    """(out, lse, tol) in float64.  tol: how far out may be off, elementwise, for an output of q's type.

    The operator's own arithmetic, against the exact value: q times the key scale and p each go through one fp16 term
    where the output is bf16 and lse is not asked for (off by half a step, 2^-11 relative) and two otherwise (2^-22),
    `term` below, a score is a sum of D products in fp32 (at most (D + 8) roundings of 2^-24 of sum |q k|, twice for the two
    terms), its exponential is good to 2^-22 plus the rounding of its argument
    (2^-23 of |score| in base 2, under 2^-22 of the natural one), the cap and the bias add roundings of their own
    magnitude (2^-20 of the cap: 1 - 2 / (e + 1) and two approximations of 1 ulp; 2^-23 of the bias).  With ds the sum
    of those, p is off by the factor 1 +- ds, numerator and denominator both, so out by 2 ds * A with
    A = sum p |v| / sum p; the fp32 sums over n keys add n 2^-24 A at the most, and the value scale and the
    division 2^-22 A.  Then one rounding to the type.  s["lse_tol"] receives the same for lse."""
    term = 2.0 ** -11 if s["q"].dtype == torch.bfloat16 and not lse else 2.0 ** -22
    q, D, Hq, Hkv, block = s["q"].double(), s["D"], s["Hq"], s["Hkv"], s["block"]
    G = Hq // Hkv
    scale = D ** -0.5 if sm_scale is None else sm_scale
    sc = s["scales"].double().clamp_min(1e-12).view(2, Hkv, D)
    f8 = F8[s["fmt"]][0]
    nb = s["cache"].shape[0] // block
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    lse_tol = s["lse_tol"] = torch.zeros(q.shape[:2], dtype=torch.float64)
    for b in range(s["lens"].numel()):
        r0, r1 = int(s["cu"][b]), int(s["cu"][b + 1])
        n, L = r1 - r0, max(0, min(int(s["lens"][b]), s["table"].shape[1] * block))
        if n <= 0 or L == 0:
            continue
        j = torch.arange(L)
        page = s["table"][b, (j // block).long()].long()
        here = (page >= 0) & (page < nb)
        codes = s["cache"][torch.where(here, page * block + j % block, 0)].view(f8).double().view(L, 2, Hkv, D)
        codes[~here] = 0
        pos = torch.arange(L - n, L)[:, None]
        see = (j[None, :] <= pos) if causal else torch.ones((n, L), dtype=torch.bool)
        if causal and prefix is not None:
            see = see | (j < int(prefix[b]))[None, :]
        if window:
            see = see & (pos - j[None, :] < window)
        see = see & here[None, :]
        for h in range(Hq):
            k, v = codes[:, 0, h // G] * sc[0, h // G], codes[:, 1, h // G] * sc[1, h // G]
            x = q[r0:r1, h]
            w = x @ k.T * scale
            mag = x.abs() @ k.abs().T * abs(scale)
            ds = mag * (term + 2.0 ** -22 + 2 * (D + 8) * 2.0 ** -24)
            if softcap:
                w = softcap * torch.tanh(w / softcap)
                ds = ds + softcap * 2.0 ** -20
            if alibi is not None:
                bias = float(alibi[h]) * (j[None, :] - pos)
                w = w + bias
                ds = ds + bias.abs() * 2.0 ** -23
            ds = ds + w.abs() * 2.0 ** -22 + term + 2.0 ** -21
            w = torch.where(see, w, -math.inf)
            any_ = see.any(1)
            m = torch.where(any_, w.max(1).values, 0.0)[:, None]
            p = torch.where(see, torch.exp(w - m), 0.0)
            l = p.sum(1, keepdim=True)
            li = torch.where(l > 0, l, 1.0)
            out[r0:r1, h] = p @ v / li
            # a weight's own error counts by its weight
            A = p @ v.abs() / li
            E = (p * ds) @ v.abs() / li + A * ((p * ds).sum(1, keepdim=True) / li)
            tol[r0:r1, h] = E + A * (L * 2.0 ** -24 + 2.0 ** -21)
            lse[r0:r1, h] = torch.where(any_, (m + torch.log(li))[:, 0], -math.inf)
            # the sum's relative error, then the logarithm, the maximum's own units and the store in fp32
            lse_tol[r0:r1, h] = (p * ds).sum(1) / li[:, 0] + L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -21 * m[:, 0].abs()
    tol = tol + (out.abs() + tol) * EPS_HALF[s["q"].dtype]
    if s["q"].dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half a step of fp16's smallest values
    return out, lse, tol


def assert_close(got, want, tol, what):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= tol)
    if bool(bad.any()):
        i = tuple(int(x) for x in torch.nonzero(bad)[0])
        worst = float(((got - want).abs() / tol.clamp_min(1e-300))[bad].max())
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} off; first at {i}: got {float(got[i])!r}, want "
                             f"{float(want[i])!r} +- {float(tol[i]):.3g}; worst {worst:.3g} x the tolerance")


def assert_lse(got, want, s, what):
    """got against want, within what reference(s) left for it."""
    got = got.double().cpu()
    assert torch.equal(torch.isneginf(got), torch.isneginf(want)), what
    fine = ~torch.isneginf(want)
    bad = ~((got - want)[fine].abs() <= s["lse_tol"][fine])
    assert not bool(bad.any()), f"{what}: lse off by {float((got - want)[fine][bad].abs().max()):.3g}"
