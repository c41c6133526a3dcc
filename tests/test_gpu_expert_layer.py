"""The operators around the experts' products run together, as an expert layer's forward pass: sort, both products, the
activation between them, the way back to the tokens -- eagerly, captured and replayed, on another stream."""
import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_quantize_amd as fp8
from tests._experts import U, check, choices, codes, product_bound, randn, round_bound, sorted_rows
from tests._gpu import DEV, to_host
from tests.test_gpu_act_quantize import quantize_ok
from tests.test_gpu_expert_rows import combine_ref
from tests.test_gpu_gemm_act import grouped_expect, scales

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Layer:
    def __init__(self, T, topk, E, H, F, seed=0):
        self.E, self.R = E, T * topk
        self.ids_host = choices(seed, T, topk, E, 0.1, T // 8)
        self.ids = torch.from_numpy(self.ids_host).to(DEV)
        self.x, self.stream = randn(seed + 1, T, H), randn(seed + 2, T, H)
        self.weights = torch.softmax(randn(seed + 3, T, topk), 1)
        self.w1, self.s1 = codes(seed + 4, E * 2 * F, H).view(E, 2 * F, H), scales(5, E * 2 * F, H).view(E, 2 * F)
        self.w2, self.s2 = codes(seed + 6, E * H, F).view(E, H, F), scales(7, E * H, F).view(E, H)
        self.b1, self.b2 = randn(8, E, 2 * F) * 0.3, randn(9, E, H) * 0.3
        self.every = torch.arange(self.R, dtype=torch.int32, device=DEV)
        new = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
        self.up, self.down, self.out = new(self.R, 2 * F), new(self.R, H), new(T, H, dtype=torch.float32)
        self.q, self.s = new(self.R, F, dtype=torch.uint8), new(self.R, dtype=torch.float32)
        self.rows = None

    def run(self, **kw):
        qx, sx = fp8.fp8_quantize_per_token(self.x, **kw)
        off, tok, of = fp8.fp8_moe_sort(self.ids, self.E, **kw)
        fp8.fp8_gemm_grouped_scaled_act(qx, sx, tok, off, self.w1, self.s1, bias=self.b1, y=self.up, **kw)
        fp8.fp8_act_quantize(self.up, act="silu", gated=True, q=self.q, scales=self.s, live_rows=off[self.E:], **kw)
        fp8.fp8_gemm_grouped_scaled_act(self.q, self.s, self.every, off, self.w2, self.s2, bias=self.b2, y=self.down, **kw)
        fp8.fp8_moe_combine(self.down, of, weights=self.weights, residual=self.stream, out=self.out, **kw)
        self.mid = (qx, sx, off, tok, of)
        return self.out


@pytest.mark.parametrize("T,topk,E,H,F", [(1, 2, 8, 256, 128), (50, 4, 12, 384, 208), (333, 6, 32, 512, 256)])
def test_layer(T, topk, E, H, F):
    L = Layer(T, topk, E, H, F)
    out = L.run().clone()
    qx, sx, off, tok, of = L.mid
    want = sorted_rows(L.ids_host, E)
    for g, w in zip((off, tok, of), want):
        assert np.array_equal(g.cpu().numpy(), w)
    n = int(want[0][-1])
    # each step from the step before it, as the kernels left it
    ref, bound = grouped_expect(qx, sx, want[1], want[0], L.w1, L.s1, L.b1, "none", torch.zeros_like(L.up), BF)
    check(L.up, ref, bound, "first product")
    quantize_ok(L.up[:n], "silu", True, L.q[:n], L.s[:n], "activation")
    ref, bound = grouped_expect(L.q, L.s, np.arange(L.R, dtype=np.int32), want[0], L.w2, L.s2, L.b2, "none",
                                torch.zeros_like(L.down), BF)
    check(L.down, ref, bound, "second product")
    ref, bound = combine_ref(L.down, of, L.weights, L.stream)
    check(out, ref, bound + round_bound(ref, torch.float32), "combine")


def test_replays_match_eager():
    L = Layer(90, 4, 16, 256, 144, seed=3)
    eager = to_host(L.run()).copy()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.run()
    for r in range(3):
        L.out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(to_host(L.out), eager), f"replay {r}"
        # other choices in the same buffers, replayed and run eagerly
        L.ids.copy_(torch.from_numpy(choices(50 + r, 90, 4, 16, 0.2)))
        g.replay()
        torch.cuda.synchronize()
        got = to_host(L.out).copy()
        assert np.array_equal(got, to_host(L.run())) and not np.array_equal(got, eager)
        L.ids.copy_(torch.from_numpy(L.ids_host))


def test_large_sort_replays_match_eager():
    """The sort in two kernels over a workspace."""
    T, topk, E = 30000, 4, 60
    ids = torch.from_numpy(choices(1, T, topk, E, 0.1)).to(DEV)
    ws = torch.empty(fp8.fp8_moe_sort_workspace_bytes(T, topk, E), dtype=torch.uint8, device=DEV)
    bufs = [t.clone() for t in fp8.fp8_moe_sort(ids, E, ws=ws)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp8.fp8_moe_sort(ids, E, *bufs, ws=ws)
    for r in range(3):
        host = choices(r + 2, T, topk, E, 0.05 * r)
        ids.copy_(torch.from_numpy(host))
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        for b, w in zip(bufs, sorted_rows(host, E)):
            assert np.array_equal(b.cpu().numpy(), w), f"replay {r}"


def test_on_another_stream():
    L = Layer(60, 3, 8, 256, 128, seed=9)
    want = L.run().clone()
    side = torch.cuda.Stream()
    L.out.zero_()
    torch.cuda.synchronize()
    spin = torch.randn((4096, 4096), device=DEV)
    with torch.cuda.stream(side):
        for _ in range(20):
            spin = spin @ spin * 1e-3   # keeps the side stream busy
    x = L.x.clone()
    L.x.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            spin = spin @ spin * 1e-3
        L.x.copy_(x)                    # the calls see it only in this stream's order
        got = L.run()
    side.synchronize()
    assert torch.equal(got, want)
    # a stream named in the call: what it allocates belongs to that stream
    off, tok, of = fp8.fp8_moe_sort(L.ids, 8, stream=side)
    out = fp8.fp8_moe_combine(L.down, of, weights=L.weights, residual=L.stream, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
