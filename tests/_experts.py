"""Plain 64-bit forms of the expert-row operators, the activations and the product epilogues, and the bounds that the
kernels' roundings give.

u = 2^-24 is fp32's rounding, half a step; the output's type adds eps / 2 of the value."""
import math

import numpy as np
import torch

from tests._gpu import DEV

U = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}  # smallest steps
F8 = torch.float8_e4m3fn


def randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def choices(seed, T, topk, E, dropped=0.0, padded=0):
    """int64 [T, topk] on the host: distinct experts a token, some of the choices outside [0, E)."""
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(T)]) if T else np.zeros((0, topk), np.int64)
    ids = ids.astype(np.int64)
    out = rng.random(ids.shape) < dropped
    ids[out] = rng.choice([-1, E, E + 7, -12345], size=int(out.sum()))
    if padded:
        ids[T - padded:] = -1
    return ids


def sorted_rows(ids, E):
    """(offsets, row_token, row_of) by numpy's stable sort."""
    T, topk = ids.shape
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])]).astype(np.int32)
    row_of = np.empty(T * topk, np.int32)
    row_of[order] = np.arange(T * topk)
    row_of[key == E] = -1
    row_token = (order // max(topk, 1)).astype(np.int32)
    row_token[offsets[-1]:] = -1
    return offsets, row_token, row_of.reshape(T, topk)


def act64(x, act):
    if act == "relu":
        return torch.where(x < 0, 0.0, x)
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return 0.5 * x * torch.special.erfc(-x / math.sqrt(2.0))
    if act == "gelu_tanh":
        return x * torch.sigmoid(math.sqrt(8.0 / math.pi) * (x + 0.044715 * x ** 3))
    return x


def act_bound(x, act, fine):
    """How far act(x) in fp32 may be from its value, for the fp32 x itself.  One hardware 2^t or reciprocal is off by
    2 u of its value.
    fine (fp32 outputs):
      silu: e^-x 2 u (2^t), 2 u (two products), 2 u (the argument's second term); 1 + e^-x u; reciprocal 2 u; product
        u: 10 u, taken as 12.
      gelu_tanh: the same and the argument's four roundings (constants, square, fma, product), each u of an argument a
        whose relative change enters the result as |a| times it: 12 + 4 |a|.
      gelu: t has 3 u (constant and sum u each at most, reciprocal 2 u) and t P(t) at most doubles it, Horner's steps add
        less than 10 u (alternating signs at most triple the later terms), the exponential 6 u, products 3 u and the fit
        1.4e-8 < u: 26 u, taken as 32.
    Otherwise the exponent's argument is one product, with u of itself and u of its constant, and gelu's fit is 4.7e-6 <
    80 u: silu 8 + 2 |x|, gelu_tanh 8 + 6 |a|, gelu 112 + 2 x^2 / 2.
    Below 2^-126 the hardware's results may be 0."""
    v = act64(x, act).abs()
    if act in ("none", "relu"):
        return torch.zeros_like(v)
    if act == "silu":
        k = 12 if fine else 8 + 2 * x.abs().clamp_max(200.0)
    elif act == "gelu":
        k = 32 if fine else 112 + x.abs().clamp_max(20.0) ** 2
    else:
        a = (math.sqrt(8.0 / math.pi) * (x + 0.044715 * x ** 3)).abs().clamp_max(200.0)
        k = 12 + 4 * a if fine else 8 + 6 * a
    return k * U * v + 2.0 ** -126 * (x.abs() + 1)


def round_bound(ref, dtype):
    return ref.abs() * torch.finfo(dtype).eps / 2 + TINY[dtype] / 2


def check(got, ref, bound, what):
    """|got - ref| <= bound everywhere, finite."""
    assert torch.isfinite(got.double()).all(), f"{what}: values that are not finite"
    over = (got.double() - ref).abs() - bound
    worst = over.max().item() if over.numel() else -1.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} outside, by {worst:.3g} at {int(over.argmax())}"


def codes(seed, rows, cols, nan_from=None):
    """E4M3 codes of normal values; columns from nan_from on are NaN codes."""
    q = (randn(seed, rows, cols) * 100).clamp(-448, 448).to(F8).view(torch.uint8)
    if nan_from is not None:
        q[:, nan_from:] = 0x7F
    return q


def product64(qa, st, qw, sc):
    """(values, sums of magnitudes) of the scaled product in 64 bits."""
    a, w = qa.view(F8).double(), qw.view(F8).double()
    s = st.double()[:, None] * sc.double()
    return (a @ w.t()) * s, (a.abs() @ w.abs().t()) * s


def product_bound(absref, K, dtype):
    """How far the product may be off before the epilogue.  16-bit outputs: the FP8 matrix instructions keep 13 bits
    below the leading one of 8 products, so a group loses at most 8 * 2^-13 of its largest one, 2^-10 of the sum of the
    magnitudes.  fp32 outputs: exact products of fp16 values, K / 8 groups joined by additions that may cut 2 u of the
    running sum (at most the sum of the magnitudes) and lose as much inside.  Scales and their product: 3 u."""
    if dtype is torch.float32:
        return absref * (K / 8 * 4 + 3 + 8) * U
    return absref * (2.0 ** -10 + (K / 8 + 3) * 2 * U)
