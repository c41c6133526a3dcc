"""How far paged attention's outputs are off in the mean square, by a model of its roundings, and an emulation of them.

Worst-case bounds of long sums leave room for operands of a few bits; the mean square of the error does not.  Model,
per query and key: the scaled query goes through `terms` fp16 terms, a relative rounding of at most 2^-11 or 2^-22 each,
uniform, so 1 / sqrt(3) of that in the mean square, independent over the channels: the score is off by that times
sqrt(sum (q_c k_c)^2); p by its own rounding, the same.  fp32 adds: sums of D products rounded on the way (random steps
of 2^-24 of partial sums no larger than |score| + sqrt(sum (q_c k_c)^2), 2 D of them), the score's argument and its
exponential (2^-22 (1 + |score|)), a cap up to 256 by its formula (2^-22 of the cap).  With e_j all of that and weights
w_j = p_j / sum p, an output is off by sum_j w_j (v_j - out) e_j, whose variance is sum_j (w_j (v_j - out) e_j)^2 for
errors that do not know of each other; the sums over keys add sqrt(n) 2^-24 of sum w |v|.  Twice that is allowed.
"""
import math

import torch

from tests._attn import F8

EPS_HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def fp16_terms(x, terms, bits=11):
    """x as the sum of fp16-like terms of `bits` bits each (float64; the exponent range is scaled away by the kernels)."""
    left, total = x, torch.zeros_like(x)
    for _ in range(terms):
        m, e = torch.frexp(left)
        t = torch.ldexp(torch.round(m * 2.0 ** bits), e - bits)
        total, left = total + t, left - t
    return total


def _rows(s, causal, window, prefix):
    """(sequence's rows, its keys and values as codes and scales, visible pairs, positions) of every sequence."""
    D, Hkv, block = s["D"], s["Hkv"], s["block"]
    for b in range(s["lens"].numel()):
        r0, r1, L = int(s["cu"][b]), int(s["cu"][b + 1]), int(s["lens"][b])
        n = r1 - r0
        if n <= 0 or L <= 0:
            continue
        j = torch.arange(L)
        codes = s["cache"][s["table"][b, (j // block).long()].long() * block + j % block].view(F8[s["fmt"]][0]).double()
        pos = torch.arange(L - n, L)[:, None]
        see = (j[None, :] <= pos) if causal else torch.ones((n, L), dtype=torch.bool)
        if causal and prefix is not None:
            see = see | (j < int(prefix[b]))[None, :]
        if window:
            see = see & (pos - j[None, :] < window)
        yield r0, r1, codes.view(L, 2, Hkv, D), see, j[None, :] - pos


def model(s, terms, causal=True, softcap=0.0, alibi=None, window=0, prefix=None, emulate=None):
    """(out, variance of out, lse, variance of lse) in float64; emulate: (terms, bits) of the operands, instead of exact
    ones, for the same as a kernel with those roundings computes it in 64 bits otherwise."""
    q, D, Hq = s["q"].double(), s["D"], s["Hq"]
    G, scale = Hq // s["Hkv"], D ** -0.5
    sc = s["scales"].double().clamp_min(1e-12).view(2, s["Hkv"], D)
    out, var = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    lvar = torch.zeros(q.shape[:2], dtype=torch.float64)
    term = 2.0 ** (-11 * terms) / math.sqrt(3)
    for r0, r1, codes, see, dist in _rows(s, causal, window, prefix):
        n = codes.shape[0]
        for h in range(Hq):
            k, v = codes[:, 0, h // G], codes[:, 1, h // G] * sc[1, h // G]
            x = q[r0:r1, h] * sc[0, h // G]
            if emulate:
                x = fp16_terms(x, *emulate)
            w = x @ k.T * scale
            spread = (x * x @ (k * k).T).sqrt() * abs(scale)
            e2 = (spread * term) ** 2 + term ** 2
            e2 = e2 + ((w.abs() + spread) * 2.0 ** -24) ** 2 * 2 * D + (2.0 ** -22 * (1 + w.abs())) ** 2
            if softcap:
                w = softcap * torch.tanh(w / softcap)
                e2 = e2 + (2.0 ** -22 * min(softcap, 256.0)) ** 2
            if alibi is not None:
                bias = float(alibi[h]) * dist
                w, e2 = w + bias, e2 + (2.0 ** -23 * bias.abs()) ** 2
            w = torch.where(see, w, -math.inf)
            some = see.any(1)
            top = torch.where(some, w.max(1).values, 0.0)[:, None]
            p = torch.where(see, torch.exp(w - top), 0.0)
            if emulate:
                p = fp16_terms(p, *emulate)
            l = p.sum(1, keepdim=True)
            l = torch.where(l > 0, l, 1.0)
            o = p @ v / l
            we = (p / l) ** 2 * e2
            out[r0:r1, h] = o
            var[r0:r1, h] = (we @ v ** 2 - 2 * o * (we @ v) + o ** 2 * we.sum(1, keepdim=True)).clamp_min(0)
            var[r0:r1, h] += n * (2.0 ** -24 * (p @ v.abs() / l)) ** 2 + (2.0 ** -22 * o) ** 2
            lse[r0:r1, h] = torch.where(some, (top + torch.log(l))[:, 0], -math.inf)
            lvar[r0:r1, h] = we.sum(1) + n * 2.0 ** -48 + (2.0 ** -22 * (1 + lse[r0:r1, h].abs().nan_to_num(0, 0, 0))) ** 2
    return out, var, lse, lvar


def excess(got, want, var, dtype):
    """The error's mean square over what the model allows, 4 times its variance: the outputs' own rounding, which want
    rounded to the type has too, is taken out of it.  (An output that rounds the other way lies half a step on either
    side of its midpoint, so the difference of squares is that of the errors before the rounding, not of the step.)"""
    got = got.double().cpu()
    own = want.to(dtype).double() - want
    square = float(((got - want) ** 2).sum() - (own ** 2).sum())
    return square / float(4 * var.sum() + 1e-3 * (own ** 2).sum())


def assert_rms(got, want, var, dtype, what):
    x = excess(got, want, var, dtype)
    assert x <= 1, f"{what}: the error's mean square is {x:.3g} of what its roundings explain"


def lse_excess(got, want, var):
    fine = ~torch.isneginf(want)
    return float(((got.double().cpu() - want)[fine] ** 2).sum()) / float(4 * var[fine].sum())
