"""The sort of a router's choices, tokens moved to the experts' rows, the rows combined and the gradient of that, against
plain 64-bit forms."""
import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._experts import U, check, choices, randn, round_bound, sorted_rows
from tests._gpu import DEV, log

pytestmark = pytest.mark.gpu
BF, HF, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8


def sort(ids, E, **kw):
    return [t.cpu().numpy() for t in fp8.fp8_moe_sort(ids, E, **kw)]


def sort_matches(ids, E, what):
    log(f"sort {what}: {ids.shape} of {E}")
    want = sorted_rows(ids, E)
    for kind in (torch.int32, torch.int64):
        got = sort(torch.from_numpy(ids).to(DEV).to(kind), E)
        for g, w, name in zip(got, want, ("expert_offsets", "row_token", "row_of")):
            assert np.array_equal(g, w), f"{what} {kind}: {name}"


@pytest.mark.parametrize("T,topk,E,dropped,padded", [
    (0, 2, 4, 0, 0), (1, 1, 1, 0, 0), (1, 8, 64, 0, 0), (8, 8, 64, 0, 0), (63, 3, 5, 0.2, 4), (64, 1, 7, 0, 0),
    (65, 1, 7, 0.5, 0), (257, 10, 100, 0.1, 13), (1000, 4, 4, 0, 0), (1024, 4, 9, 0, 0), (1025, 4, 9, 0.05, 0),
    (4096, 8, 64, 0.02, 100), (5461, 12, 12, 0, 0), (5462, 12, 30, 0.1, 0), (300, 2, 1024, 0, 0), (4097, 1, 1024, 0.1, 7),
    (30000, 3, 1024, 0.01, 999), (70000, 5, 33, 0.3, 0), (131072, 8, 256, 0, 4000), (66000, 1, 1, 0, 0)])
def test_sort(T, topk, E, dropped, padded):
    sort_matches(choices(T + E, T, topk, E, dropped, padded), E, "random")


@pytest.mark.parametrize("T", [5, 3000, 40000])
def test_sort_one_sided(T):
    sort_matches(np.full((T, 3), 6, np.int64), 17, "one expert")
    sort_matches(np.full((T, 3), -1, np.int64), 17, "no expert")
    sort_matches(np.full((T, 3), 17, np.int64), 17, "past the last")
    ids = np.zeros((T, 2), np.int64)
    ids[:, 1] = 16
    sort_matches(ids, 17, "first and last")
    sort_matches(np.arange(2 * T).reshape(T, 2)[::-1] % 17, 17, "falling")
    sort_matches(np.zeros((T, 1), np.int64), 0, "no experts at all")


def test_sort_wide_ids_are_not_cut():
    ids = torch.tensor([[1 << 32, 3], [(1 << 32) + 2, -(1 << 32)], [2, (1 << 62) + 1]], device=DEV)
    off, tok, of = sort(ids, 4)
    assert off.tolist() == [0, 0, 0, 1, 2] and of.tolist() == [[-1, 1], [-1, -1], [0, -1]]
    assert tok.tolist() == [2, 0, -1, -1, -1, -1]


def test_sort_outputs_and_workspace_of_the_caller():
    T, topk, E = 40000, 4, 50
    ids = choices(3, T, topk, E, 0.1)
    d = torch.from_numpy(ids).to(DEV).int()
    ws = torch.full((fp8.fp8_moe_sort_workspace_bytes(T, topk, E),), 255, dtype=U8, device=DEV)
    off = torch.full((E + 1,), -7, dtype=torch.int32, device=DEV)
    tok, of = torch.full((T * topk,), -7, dtype=torch.int32, device=DEV), torch.full((T, topk), -7, dtype=torch.int32, device=DEV)
    got = fp8.fp8_moe_sort(d, E, expert_offsets=off, row_token=tok, row_of=of, ws=ws)
    assert got[0] is off and got[1] is tok and got[2] is of
    for g, w in zip(got, sorted_rows(ids, E)):
        assert np.array_equal(g.cpu().numpy(), w)
    with pytest.raises(fp8.Fp8Error):
        fp8.fp8_moe_sort(d, E, ws=ws[:-1])
    with pytest.raises(ValueError):
        fp8.fp8_moe_sort(d.t(), E)
    with pytest.raises(TypeError):
        fp8.fp8_moe_sort(d.short(), E)
    with pytest.raises(fp8.Fp8Error):
        fp8.fp8_moe_sort(d, 1025)


def rows_of(seed, T, topk, E, dropped=0.0, padded=0):
    off, tok, of = sorted_rows(choices(seed, T, topk, E, dropped, padded), E)
    return torch.from_numpy(of).to(DEV)


SHAPES = [  # T, topk, E, H
    (1, 1, 1, 1), (1, 8, 64, 7168), (3, 2, 5, 7), (5, 3, 9, 8), (7, 6, 20, 15), (4, 4, 4, 16), (33, 9, 30, 129),
    (64, 1, 8, 512), (9, 10, 12, 1000), (130, 5, 40, 2049), (12, 17, 40, 333), (300, 2, 3, 65), (2, 3, 4, 30001)]


@pytest.mark.parametrize("kind", [U8, BF, HF, F32])
@pytest.mark.parametrize("T,topk,E,H", SHAPES)
def test_permute(T, topk, E, H, kind):
    row_of = rows_of(T * H, T, topk, E, 0.15, T // 5)
    x = torch.randint(0, 256, (T, H * kind.itemsize), dtype=U8, device=DEV).view(kind)
    s = randn(1, T)
    R = T * topk
    out, s_out = torch.full((R, H * kind.itemsize), 0xA5, dtype=U8, device=DEV), torch.full((R,), -3.0, device=DEV)
    got = fp8.fp8_moe_permute(x, row_of, s_tok=s, out=out.view(kind), s_out=s_out)
    want, want_s = torch.full_like(out, 0xA5), torch.full_like(s_out, -3.0)
    t, j = (row_of >= 0).nonzero(as_tuple=True)
    want[row_of[t, j].long()] = x.view(U8)[t]
    want_s[row_of[t, j].long()] = s[t]
    assert got[1] is s_out and torch.equal(out, want) and torch.equal(s_out, want_s)
    assert fp8.fp8_moe_permute(x, row_of).shape == (R, H)


def test_permute_strides_and_entries_outside():
    x = randn(2, 10, 40, dtype=BF)[:, :33]
    out = torch.full((6, 50), 7.0, dtype=BF, device=DEV)
    row_of = torch.tensor([[0, 6], [5, -1], [1 << 30, 2], [-(1 << 31), 4]] + [[-1, -1]] * 6, dtype=torch.int32, device=DEV)
    fp8.fp8_moe_permute(x, row_of, out=out[:, :33], num_rows=6)
    want = torch.full_like(out, 7.0)
    for t, r in ((0, 0), (1, 5), (2, 2), (3, 4)):
        want[r, :33] = x[t]
    assert torch.equal(out, want)
    with pytest.raises(ValueError):
        fp8.fp8_moe_permute(x, row_of, out=out[:, :33], num_rows=7)
    with pytest.raises(ValueError):
        fp8.fp8_moe_permute(x, row_of, s_out=torch.ones(20, device=DEV))


def test_permute_and_combine_past_four_gigabytes():
    T, topk, H = 70000, 8, 8200
    log("4.6 GB of rows")
    row_of = torch.randperm(T * topk, device=DEV).int().view(T, topk)
    x = torch.randint(0, 255, (T, H), dtype=U8, device=DEV)
    out = fp8.fp8_moe_permute(x, row_of)
    at = torch.cat([torch.arange(100), torch.arange(T - 100, T)]).to(DEV)
    for j in (0, 7):
        assert torch.equal(out[row_of[at, j].long()], x[at])
    del out
    y = torch.empty((T * topk, 4100), dtype=HF, device=DEV)
    y.copy_((torch.arange(T * topk, device=DEV) % 1021)[:, None].expand(-1, 4100))
    got = fp8.fp8_moe_combine(y, row_of, out_dtype=F32)
    want = (row_of.long() % 1021).sum(1).float()
    assert torch.equal(got, want[:, None].expand(-1, 4100))


def combine_ref(y, row_of, weights, residual):
    """(values, bound on the fp32 sum's error) in 64 bits."""
    T, topk = row_of.shape
    out = torch.zeros((T, y.shape[1]), dtype=torch.float64, device=DEV) if residual is None else residual.double()
    size = out.abs()
    for j in range(topk):
        at = (row_of[:, j] >= 0).nonzero()[:, 0]
        v = y[row_of[at, j].long()].double()
        v = v if weights is None else v * weights[at, j].double()[:, None]
        out[at] += v
        size[at] += v.abs()
    return out, size * (topk + 1) * U


@pytest.mark.parametrize("kind,to", [(BF, BF), (HF, HF), (F32, F32), (BF, F32), (F32, BF), (F32, HF), (HF, F32), (BF, HF), (HF, BF)])
@pytest.mark.parametrize("T,topk,E,H", SHAPES)
def test_combine(T, topk, E, H, kind, to):
    row_of = rows_of(T + H, T, topk, E, 0.15, T // 5)
    y, w, res = randn(1, T * topk, H, dtype=kind), randn(2, T, topk), randn(3, T, H, dtype=to)
    for weights, residual in ((w, None), (None, res), (w, res)):
        got = fp8.fp8_moe_combine(y, row_of, weights=weights, residual=residual, out_dtype=to)
        ref, bound = combine_ref(y, row_of, weights, residual)
        assert got.dtype is to
        check(got, ref, bound + round_bound(ref, to), f"combine {T, topk, H, kind, to}")
        if residual is not None:
            own = residual.clone()
            assert fp8.fp8_moe_combine(y, row_of, weights=weights, residual=own, out=own) is own
            assert torch.equal(own, got)


def test_combine_leaves_out_what_is_dropped():
    row_of = torch.tensor([[0, -1], [-1, -1], [3, 9], [1, 2]], dtype=torch.int32, device=DEV)
    y, w = torch.ones((4, 24), dtype=BF, device=DEV), torch.full((4, 2), 2.0, device=DEV)
    w[0, 1] = w[1, 0] = w[2, 1] = float("nan")
    y[2] = float("inf")
    out = fp8.fp8_moe_combine(y, row_of, weights=w)
    assert (out[0] == 2).all() and (out[1] == 0).all() and (out[2] == 2).all() and (out[3] == float("inf")).all()
    y[0] = float("nan")  # a row that is used; no other token's choice may touch it
    out = fp8.fp8_moe_combine(y, row_of, weights=w)
    assert out[0].isnan().all() and (out[1] == 0).all() and (out[2] == 2).all()
    none = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    res = randn(5, 3, 24, dtype=BF)
    assert torch.equal(fp8.fp8_moe_combine(y[:0], none, residual=res), res)
    assert torch.equal(fp8.fp8_moe_combine(y, none[:, :0], residual=res), res)
    assert (fp8.fp8_moe_combine(y[:0], none) == 0).all()


def test_combine_strides():
    row_of = rows_of(5, 40, 3, 8, 0.1)
    for H in (64, 61):
        y, res = randn(1, 120, 70, dtype=BF)[:, :H], randn(2, 40, 77)[:, :H]
        out = torch.full((40, 90), 5.0, device=DEV)
        fp8.fp8_moe_combine(y, row_of, residual=res, out=out[:, :H])
        ref, bound = combine_ref(y, row_of, None, res)
        check(out[:, :H], ref, bound + round_bound(ref, F32), f"strided {H}")
        assert (out[:, H:] == 5).all()


@pytest.mark.parametrize("dk,yk", [(BF, BF), (HF, HF), (F32, F32), (F32, BF), (BF, F32), (HF, BF), (F32, HF), (BF, HF), (HF, F32)])
@pytest.mark.parametrize("T,topk,E,H", SHAPES)
def test_grad(T, topk, E, H, dk, yk):
    row_of = rows_of(T + 2 * H, T, topk, E, 0.15, T // 5)
    d, y, w = randn(1, T, H, dtype=dk), randn(2, T * topk, H, dtype=yk), randn(3, T, topk)
    dy = torch.full((T * topk, H), 9.0, dtype=yk, device=DEV)
    dw = torch.full((T, topk), 9.0, device=DEV)
    got = fp8.fp8_moe_combine_grad(d, y, row_of, weights=w, dy=dy, dweights=dw)
    assert got[0] is dy and got[1] is dw
    want, live = torch.full((T * topk, H), 9.0, dtype=torch.float64, device=DEV), row_of >= 0
    t, j = live.nonzero(as_tuple=True)
    r = row_of[t, j].long()
    want[r] = w[t, j].double()[:, None] * d[t].double()
    check(dy, want, want.abs() * U + round_bound(want, yk), "dy")
    ref, size = torch.zeros_like(dw, dtype=torch.float64), torch.zeros_like(dw, dtype=torch.float64)
    prod = d[t].double() * y[r].double()
    ref[t, j], size[t, j] = prod.sum(1), prod.abs().sum(1)
    # every term passes through the additions of its own thread, the exchanges of a wave and the waves' sums
    check(dw, ref, size * (H / 8 + 8 + 8 + 8) * U, "dweights")
    assert (dw[~live] == 0).all()
    plain, _ = fp8.fp8_moe_combine_grad(d, y, row_of, need_dweights=False)
    assert torch.equal(plain[r], d[t].to(yk))
    none, only = fp8.fp8_moe_combine_grad(d, y, row_of, weights=w, need_dy=False)
    assert none is None and torch.equal(only, dw)
    own = y.clone()
    fp8.fp8_moe_combine_grad(d, own, row_of, weights=w, dy=own, dweights=dw)
    assert torch.equal(own[r], dy[r]) and torch.equal(dw, only)


def test_grad_against_differences():
    """combine is linear in the weights, the rows and the residual: a change of one of them by delta changes <dout, out>
    by <gradient, delta>, in exact arithmetic; both sides in 64 bits from the kernels' fp32 outputs."""
    T, topk, E, H = 37, 4, 11, 300
    row_of = rows_of(8, T, topk, E, 0.1)
    y, w, d = randn(1, T * topk, H), randn(2, T, topk), randn(3, T, H)
    dy = torch.zeros_like(y)
    _, dw = fp8.fp8_moe_combine_grad(d, y, row_of, weights=w, dy=dy)
    base = fp8.fp8_moe_combine(y, row_of, weights=w)

    def moved(y2, w2):
        a, b = fp8.fp8_moe_combine(y2, row_of, weights=w2), base
        # each fp32 output is off by (topk + 1) u of its terms' magnitudes
        size = combine_ref(y2, row_of, w2, None)[1] + combine_ref(y, row_of, w, None)[1]
        return (d.double() * (a.double() - b.double())).sum(), (d.double().abs() * size).sum()

    t, j = (row_of >= 0).nonzero(as_tuple=True)
    size_dw = torch.zeros((T, topk), dtype=torch.float64, device=DEV)
    size_dw[t, j] = (d[t].double() * y[row_of[t, j].long()].double()).abs().sum(1)
    for seed in range(4):
        got, slack = moved(y, w + randn(10 + seed, T, topk))
        change = (w + randn(10 + seed, T, topk)).double() - w.double()
        want = (dw.double() * change).sum()
        slack = slack + (size_dw * (H / 8 + 24) * U * change.abs()).sum()  # dweights' own bound, as in test_grad
        assert abs(got - want) <= slack, (got, want, slack)
        got, slack = moved(y + randn(20 + seed, T * topk, H), w)
        change = (y + randn(20 + seed, T * topk, H)).double() - y.double()
        want = (dy.double() * change).sum()
        assert abs(got - want) <= slack + (dy.double() * change).abs().sum() * U, (got, want, slack)
    # permute's gradient is combine without weights: <permute(x), g> = <x, combine(g)>
    x, g = randn(4, T, H), randn(5, T * topk, H)
    out = fp8.fp8_moe_permute(x, row_of, out=torch.zeros((T * topk, H), device=DEV))
    left = (out.double() * g.double()).sum()
    back = fp8.fp8_moe_combine(g, row_of)
    bound = (x.double().abs() * combine_ref(g, row_of, None, None)[1]).sum()
    assert abs(left - (x.double() * back.double()).sum()) <= bound


def test_grad_of_rows_past_four_gigabytes():
    T, topk, H, ld = 2, 2, 1003, (1 << 30) + 40
    row_of = torch.tensor([[3, 0], [1, 2]], dtype=torch.int32, device=DEV)
    dout, y, w = randn(1, T, H, dtype=HF), randn(2, T * topk, H, dtype=HF), randn(3, T, topk)
    far = torch.empty(3 * ld + H, dtype=HF, device=DEV).as_strided((4, H), (ld, 1))
    far.copy_(y)
    log("rows 2^30 elements apart")
    want_y, want_w = fp8.fp8_moe_combine_grad(dout, y, row_of, w)
    dy, dw = fp8.fp8_moe_combine_grad(dout, far, row_of, w, dy=far)
    assert torch.equal(dy, want_y) and torch.equal(dw, want_w)


def test_refused_arguments():
    row_of = rows_of(1, 6, 2, 3)
    y, x = randn(1, 12, 32, dtype=BF), randn(2, 6, 32, dtype=BF)
    for f in (lambda: fp8.fp8_moe_combine(y, row_of.long()), lambda: fp8.fp8_moe_combine(y.double(), row_of),
              lambda: fp8.fp8_moe_combine(y, row_of, weights=torch.ones((6, 2), device=DEV, dtype=BF)),
              lambda: fp8.fp8_moe_combine(y, row_of, residual=x, out_dtype=F32),
              lambda: fp8.fp8_moe_permute(x.double(), row_of), lambda: fp8.fp8_moe_permute(x, row_of.cpu())):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: fp8.fp8_moe_combine(y.t(), row_of), lambda: fp8.fp8_moe_combine(y, row_of, residual=x[:5]),
              lambda: fp8.fp8_moe_combine(y, row_of.t()), lambda: fp8.fp8_moe_permute(x[:5], row_of),
              lambda: fp8.fp8_moe_combine_grad(x[:, :31], y, row_of), lambda: fp8.fp8_moe_combine(y, row_of, weights=torch.ones(5, device=DEV))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(fp8.Fp8Error):  # not 16-byte aligned
        fp8.fp8_moe_combine(y[:, 1:], row_of)
