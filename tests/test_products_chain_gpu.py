"""The new calls as they are used together: a mixture of experts in 8 bits, and
the whole gradient of the 4-bit experts' layer."""
import pytest
import torch

import bf16_activation_quantized_amd as w4
from products_ref import fp8_values, int4_values

pytestmark = pytest.mark.gpu
DEV = "cuda"


def route(T, k, G, seed):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, G, generator=g)
    top, ids = logits.topk(k, dim=1)
    ids = ids.int()
    ids[::7] = -1                               # padded tokens
    return ids, torch.softmax(top, 1)


def test_experts_in_8_bits():
    """Sort, gather, quantise, product by expert, activation, quantise, product, combine; each product against the
    64-bit one of the very values it was given, the rest on bf16 values."""
    T, k, G, H, F = 150, 3, 6, 256, 384
    ids, weights = route(T, k, G, 1)
    x = torch.randn(T, H).bfloat16()
    w1, s1 = w4.w4a16_fp8_quantize((torch.randn(G * F, H) * H ** -0.5).bfloat16().to(DEV), block_rows=128)
    w2, s2 = w4.w4a16_fp8_quantize((torch.randn(G * H, F) * F ** -0.5).bfloat16().to(DEV), block_rows=128)
    w1, s1, w2, s2 = w1.view(G, F, H), s1.view(G, F // 128, H // 128), w2.view(G, H, F), s2.view(G, H // 128, F // 128)
    order, pos, sizes = w4.w4a16_expert_sort(ids.to(DEV), G)
    xs = torch.zeros(T * k, H, dtype=torch.bfloat16, device=DEV)
    w4.w4a16_expert_gather(x.to(DEV), pos, xs=xs)
    q, qs = w4.w4a16_fp8_quantize(xs)
    h = w4.w4a16_fp8_gemm_grouped(q, qs, w1, s1, sizes, y=torch.zeros(T * k, F, dtype=torch.bfloat16, device=DEV))
    a = torch.nn.functional.silu(h.float()).bfloat16()
    qa, qas = w4.w4a16_fp8_quantize(a)
    z = w4.w4a16_fp8_gemm_grouped(qa, qas, w2, s2, sizes, y=torch.zeros(T * k, H, dtype=torch.bfloat16, device=DEV))
    y = w4.w4a16_expert_combine(z, pos, weights.to(DEV))

    n = sizes.tolist()
    kept = sum(n)

    def by_expert(q, qs, w, s):
        v, out, r = fp8_values(q.cpu(), qs.cpu(), 1), [], 0
        for e in range(G):
            out.append(v[r:r + n[e]] @ fp8_values(w[e].cpu(), s[e].cpu(), 128).t())
            r += n[e]
        return torch.cat(out)
    for got, want in ((h, by_expert(q, qs, w1, s1)), (z, by_expert(qa, qas, w2, s2))):
        assert ((got[:kept].double().cpu() - want).norm() / want.norm()).item() < 2.0 ** -8 + 2.0 ** -10
        assert (got[kept:] == 0).all()
    # the layer as a whole against the definition on unquantised activations: two quantisations (2^-4 each at most)
    ref = torch.zeros(T, H, dtype=torch.float64)
    v1 = [fp8_values(w1[e].cpu(), s1[e].cpu(), 128) for e in range(G)]
    v2 = [fp8_values(w2[e].cpu(), s2[e].cpu(), 128) for e in range(G)]
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e >= 0:
                ref[t] += weights[t, j].double() * (torch.nn.functional.silu(x[t].double() @ v1[e].t()) @ v2[e].t())
    assert ((y.double().cpu() - ref).norm() / ref.norm()).item() < 2 * 2.0 ** -4
    assert (y[::7] == 0).all()


def test_gradient_of_the_4_bit_experts():
    """combine's gradient, the product's input gradient and gather's gradient in a row are the gradient of the layer
    x -> combine(product(gather(x))) with respect to x."""
    T, k, G, H, F, gs = 120, 2, 5, 256, 200, 32
    ids, weights = route(T, k, G, 2)
    x = torch.randn(T, H).bfloat16()
    w = torch.randint(0, 256, (G, F, H // 2), dtype=torch.uint8)
    s = (0.01 + 0.01 * torch.rand(G, F, H // gs)).bfloat16()
    dy = torch.randn(T, F).bfloat16()
    wd, sd, wt = w.to(DEV), s.to(DEV), weights.to(DEV)
    order, pos, sizes = w4.w4a16_expert_sort(ids.to(DEV), G)
    rows = lambda n: torch.zeros(T * k, n, dtype=torch.bfloat16, device=DEV)   # noqa: E731
    xs = w4.w4a16_expert_gather(x.to(DEV), pos, xs=rows(H))
    z = w4.w4a16_gemm_grouped(xs, wd, sd, sizes, y=rows(F), group_size=gs)
    dz, dw = w4.w4a16_expert_combine_grad(dy.to(DEV), z, pos, wt, dz=rows(F))
    dxs = w4.w4a16_gemm_grad(dz, wd, sd, m_sizes=sizes, dx=rows(H), group_size=gs)
    dx = w4.w4a16_expert_gather_grad(dxs, pos)

    xr = x.double().requires_grad_()
    out = []
    v = [int4_values(w[e], s[e], gs) for e in range(G)]
    for t in range(T):
        y = torch.zeros(F, dtype=torch.float64)
        for j in range(k):
            e = int(ids[t, j])
            if e >= 0:
                y = y + weights[t, j].double() * (v[e] @ xr[t])
        out.append(y)
    (torch.stack(out) * dy.double()).sum().backward()
    # three roundings to bf16: of dz, of dxs and of the sum
    assert ((dx.double().cpu() - xr.grad).norm() / xr.grad.norm()).item() < 3 * 2.0 ** -8
    assert (dx[::7] == 0).all()
