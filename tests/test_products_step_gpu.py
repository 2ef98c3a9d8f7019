"""A training step of a mixture of experts in 8 bits as one captured graph: routing,
quantisation, both expert products, both gradients and the rows' own, replayed with
other tokens and other routing between eager work, against the same calls made
eagerly (bit for bit) and against the 64-bit gradient of the very values."""
import pytest
import torch

import bf16_activation_quantized_amd as w4
from products_ref import fp8_values

pytestmark = pytest.mark.gpu
DEV = "cuda"
T, K, G, H, F = 150, 3, 6, 256, 384      # tokens, slots per token, experts, widths


def rows(n):
    return torch.zeros(T * K, n, dtype=torch.bfloat16, device=DEV)


class Layer:
    """y = combine(relu(xs . W1^T) . W2^T), and the gradient with respect to x; every buffer kept."""

    def __init__(self):
        g = torch.Generator().manual_seed(0)
        w1 = (torch.randn(G * F, H, generator=g) * H ** -0.5).bfloat16()
        w2 = (torch.randn(G * H, F, generator=g) * F ** -0.5).bfloat16()
        q1, s1 = w4.w4a16_fp8_quantize(w1.to(DEV), block_rows=128)
        q2, s2 = w4.w4a16_fp8_quantize(w2.to(DEV), block_rows=128)
        self.w1, self.s1 = q1.view(G, F, H), s1.view(G, F // 128, H // 128)
        self.w2, self.s2 = q2.view(G, H, F), s2.view(G, H // 128, F // 128)

    def step(self, x, ids, weights, dy):
        o = {}
        _, pos, sizes = w4.w4a16_expert_sort(ids, G)
        xs = w4.w4a16_expert_gather(x, pos, xs=rows(H))
        q, s = w4.w4a16_fp8_quantize(xs)
        h = w4.w4a16_fp8_gemm_grouped(q, s, self.w1, self.s1, sizes, y=rows(F))
        a, sa = w4.w4a16_fp8_quantize(torch.relu(h))
        z = w4.w4a16_fp8_gemm_grouped(a, sa, self.w2, self.s2, sizes, y=rows(H))
        o["y"] = w4.w4a16_expert_combine(z, pos, weights)
        dz, o["dweights"] = w4.w4a16_expert_combine_grad(dy, z, pos, weights, dz=rows(H))
        d, sd = w4.w4a16_fp8_quantize(dz)
        da = w4.w4a16_fp8_gemm_grad(d, sd, self.w2, self.s2, m_sizes=sizes, dx=rows(F))
        e, se = w4.w4a16_fp8_quantize(torch.where(h > 0, da, torch.zeros_like(da)))
        dxs = w4.w4a16_fp8_gemm_grad(e, se, self.w1, self.s1, m_sizes=sizes, dx=rows(H))
        o["dx"] = w4.w4a16_expert_gather_grad(dxs, pos)
        o.update(sizes=sizes, q=q, s=s, h=h, a=a, sa=sa, z=z, d=d, sd=sd, da=da, e=e, se=se, dxs=dxs)
        return o


def inputs(seed):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, G, generator=g) + torch.randn(G, generator=g)
    top, ids = logits.topk(K, dim=1)
    ids = ids.int()
    ids[seed % 7::7] = -1                       # padded tokens
    return [t.to(DEV) for t in (torch.randn(T, H, generator=g).bfloat16(), ids, torch.softmax(top, 1),
                                (torch.randn(T, H, generator=g) * 1e-3).bfloat16())]


def check(layer, o, ids):
    """Each product and each gradient against the 64-bit one of the values that it was given."""
    n = o["sizes"].tolist()
    kept = sum(n)
    assert kept == int((ids >= 0).sum())
    w1 = [fp8_values(w.cpu(), s.cpu(), 128) for w, s in zip(layer.w1, layer.s1)]
    w2 = [fp8_values(w.cpu(), s.cpu(), 128) for w, s in zip(layer.w2, layer.s2)]
    for x, s, ws, got in (("q", "s", [w.t() for w in w1], "h"), ("a", "sa", [w.t() for w in w2], "z"),
                          ("d", "sd", w2, "da"), ("e", "se", w1, "dxs")):
        v = fp8_values(o[x].cpu(), o[s].cpu(), 1)
        at, want = 0, []
        for rows_, w in zip(n, ws):
            want.append(v[at:at + rows_] @ w)
            at += rows_
        want = torch.cat(want)
        y = o[got].double().cpu()
        # the rounding's 2^-8 and the matrix core's groups of 8, which lose at most 2^-10 of their magnitudes
        assert ((y[:kept] - want).norm() / want.norm()).item() < 2.0 ** -8 + 2.0 ** -10, got
        assert (y[kept:] == 0).all(), got


def test_captured_step():
    layer = Layer()
    x = inputs(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(*x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer.step(*x)
    for seed in range(1, 6):
        new = inputs(seed)
        for a, b in zip(x, new):
            a.copy_(b)
        graph.replay()
        eager = layer.step(*new)                # its own work beside the replay's outputs
        torch.cuda.synchronize()
        for name, v in eager.items():
            if v.element_size() == 1:
                assert torch.equal(captured[name].view(torch.uint8), v.view(torch.uint8)), (seed, name)
            else:
                assert torch.equal(captured[name], v), (seed, name)
        check(layer, captured, new[1])
