"""The input gradient of the 4-bit products on the GPU against its 64-bit definition.

Small whole numbers in dY (times a power of two per row) and powers of two as
scales: every sum is exact in fp32, so the output is the exact result rounded
once, bit for bit. Random values: dY and s (q - 8) are exact in the matrix
core's operands, so what is left are its fp32 additions (at most 2^-23 of the
magnitudes each: the 32 elements of a step at a time, the steps and the slices)
and the rounding to bf16 (2^-8).
"""
import pytest
import torch

import bf16_activation_quantized_amd as w4
from products_ref import grouped_ref, int4_values

pytestmark = pytest.mark.gpu
DEV = "cuda"
HEIGHTS = (16, 32, 64, 96, 128, 160, 192, 224, 256)
TILES = [None] + [(h, 1) for h in HEIGHTS] + [(16, 4), (32, 16), (64, 2), (96, 3), (192, 5), (256, 16)]


class Case:
    def __init__(self, M, N, K, gs=128, sizes=None, exact=True, seed=0):
        g = torch.Generator().manual_seed(seed + 7919 * M + 31 * N + K)
        lead = () if sizes is None else (len(sizes),)
        self.gs, self.sizes, self.K = gs, sizes, K
        self.w = torch.randint(0, 256, (*lead, N, K // 2), generator=g, dtype=torch.uint8)
        if exact:
            self.dy = torch.randint(-8, 9, (M, N), generator=g).float()
            self.dy *= torch.ldexp(torch.ones(M, 1), torch.randint(-60, 61, (M, 1), generator=g))
            self.s = torch.ldexp(torch.ones(*lead, N, K // gs), torch.randint(-2, 3, (*lead, N, K // gs), generator=g))
        else:
            self.dy = torch.randn(M, N, generator=g) * torch.exp(4 * torch.randn(M, 1, generator=g) - 10)
            self.s = 0.005 + 0.015 * torch.rand(*lead, N, K // gs, generator=g)
        self.dy, self.s = self.dy.bfloat16(), self.s.bfloat16()
        self.dev = [t.to(DEV) for t in (self.dy, self.w, self.s)]
        self.m = None if sizes is None else torch.tensor(sizes, dtype=torch.int32, device=DEV)

    def want(self):
        w, s = (self.w, self.s) if self.sizes is not None else (self.w[None], self.s[None])
        return grouped_ref(self.dy.double(), [int4_values(a, b, self.gs) for a, b in zip(w, s)],
                           [self.dy.shape[0]] if self.sizes is None else self.sizes, self.K)

    def run(self, tile=None, dx=None, **kw):
        if dx is None:
            dx = torch.full((self.dy.shape[0], self.K), float("nan"), dtype=torch.bfloat16, device=DEV)
        return w4.w4a16_gemm_grad(*self.dev, m_sizes=self.m, dx=dx, group_size=self.gs, tile=tile, **kw)


SHAPES = [(1, 8, 128), (1, 4096, 256), (3, 56, 384), (16, 64, 512), (17, 200, 640), (63, 264, 256), (64, 1000, 128),
          (65, 128, 896), (129, 72, 384), (200, 520, 1152), (257, 192, 256), (300, 1032, 384)]


@pytest.mark.parametrize("tile", TILES, ids=str)
@pytest.mark.parametrize("gs", [128, 32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact(M, N, K, gs, tile):
    c = Case(M, N, K, gs)
    assert torch.equal(c.run(tile).cpu(), c.want()[0].bfloat16())


@pytest.mark.parametrize("tile", [None] + [(h, 1) for h in HEIGHTS] + [(16, 3), (64, 4), (192, 2)], ids=str)
@pytest.mark.parametrize("gs", [128, 32])
@pytest.mark.parametrize("sizes", [[5], [0, 3], [40, 1, 0, 17, 100], [0, 0, 300, 20, 0], [0, 0], [1] * 70],
                         ids=lambda s: f"{len(s)}x{sum(s)}")
def test_grouped_exact(sizes, gs, tile):
    M = sum(sizes) + 5
    c = Case(M, 200, 384, gs, sizes)
    want = c.want()[0]
    dx = torch.full((M, 384), 7.0, dtype=torch.bfloat16, device=DEV)
    assert c.run(tile, dx) is dx
    assert torch.equal(dx[:-5].cpu(), want[:-5].bfloat16()) and (dx[-5:] == 7).all()


@pytest.mark.parametrize("tile", [None, (16, 1), (64, 1), (256, 1), (16, 2)], ids=str)
def test_few_rows_far_apart(tile):
    """One row of each of a few experts, the first and the last of many among them,
    so that every tile holds one row; then all rows with the last expert."""
    for sizes in ([1] + [0] * 198 + [1, 0, 0, 1, 1] + [0] * 95 + [1], [0] * 299 + [40], [40] + [0] * 299):
        c = Case(sum(sizes), 64, 128, 128, sizes)
        assert torch.equal(c.run(tile).cpu(), c.want()[0].bfloat16())


@pytest.mark.parametrize("gs,K", [(32, 4096), (32, 4224), (32, 8320), (128, 16384), (128, 16512), (128, 24704)])
def test_wide_rows_of_scales(gs, K):
    """Up to 128 scale groups the prepass reads them as one run, past that 64 at a time."""
    for N in (40, 264):
        c = Case(20, N, K, gs)
        assert torch.equal(c.run().cpu(), c.want()[0].bfloat16())
    c = Case(9, 136, K, gs, [3, 0, 4])
    assert torch.equal(c.run()[:7].cpu(), c.want()[0][:7].bfloat16())


@pytest.mark.parametrize("N", [20472, 20480, 20488, 41000])
def test_long_rows(N):
    """Rows that the prepass holds in registers, and longer ones, with the largest value in each part."""
    c = Case(4, N, 128)
    for m, n in enumerate((0, N - 1, N // 2, 20479 % N)):
        c.dy[m] = 0
        c.dy[m, n] = 3.0
        c.dy[m, (n + 77) % N] = -2.0 ** -10
    c.dev[0] = c.dy.to(DEV)
    assert torch.equal(c.run().cpu(), c.want()[0].bfloat16())


def test_negative_scales():
    c = Case(40, 200, 256, 32)
    c.s[::3] *= -1
    c.dev[2] = c.s.to(DEV)
    assert torch.equal(c.run().cpu(), c.want()[0].bfloat16())


@pytest.mark.parametrize("tile", [None, (16, 1), (32, 1), (64, 2), (128, 1), (192, 1), (256, 1)], ids=str)
@pytest.mark.parametrize("M,N,K,gs", [(1, 1000, 256, 128), (40, 2048, 384, 32), (300, 1032, 512, 128),
                                      (300, 1032, 512, 32)])
def test_random_values(M, N, K, gs, tile):
    c = Case(M, N, K, gs, exact=False)
    want, size = c.want()
    y = c.run(tile).double().cpu()
    lim = 2.0 ** -8 * want.abs() + 2.0 ** -23 * (32 + N // 32 + 20) * size
    assert ((y - want).abs() <= lim).all()
    assert ((y - want).norm(dim=1) <= 2.0 ** -8 * want.norm(dim=1)).all()      # row by row: they differ in size


def test_differences():
    """The gradient of sum(dY * (X . W^T)) against differences of the 4-bit product itself (exact inputs)."""
    M, N, K = 4, 128, 256
    c = Case(M, N, K)
    dy = torch.randint(-3, 4, (M, N)).float()
    c.dev[0] = dy.bfloat16().to(DEV)
    dx = c.run().float().cpu()
    x = torch.randint(-3, 4, (M, K)).float()
    for k in (0, 1, 127, 128, 200, 255):
        up, down = x.clone(), x.clone()
        up[:, k] += 4
        down[:, k] -= 4
        w = int4_values(c.w, c.s, c.gs)
        want = ((dy.double() * ((up - down).double() @ w.t())).sum(1) / 8).float()
        y = [w4.w4a16_gemm(v.bfloat16().to(DEV), c.dev[1], c.dev[2]).float().cpu() for v in (up, down)]
        diff = (dy * (y[0] - y[1])).sum(1) / 8
        assert torch.equal(dx[:, k], want.bfloat16().float())
        # each output of the product is rounded to bf16 on both sides
        assert ((diff - want).abs() <= 2.0 ** -8 * (dy.abs() * (y[0].abs() + y[1].abs())).sum(1) / 8 + 1e-3).all()


def test_wide_ranges():
    """Rows of very different size, tiny and huge scales, outliers within a row."""
    M, N, K = 70, 256, 512
    c = Case(M, N, K, 32, exact=False)
    c.dy = c.dy.float()
    c.dy /= c.dy.abs().amax(1, keepdim=True)
    c.dy *= torch.ldexp(torch.ones(M, 1), torch.randint(-110, 100, (M, 1)))
    c.dy[5, 7] *= 2.0 ** 20                    # an outlier: the others keep all their bits
    c.dy[6] = 0
    c.dy[7, 3:] = 0
    c.dy = c.dy.bfloat16()
    c.s = c.s.float() * torch.ldexp(torch.ones(1, K // 32), torch.randint(-6, 7, (1, K // 32)))
    c.s = c.s.bfloat16()
    c.dev = [t.to(DEV) for t in (c.dy, c.w, c.s)]
    want, size = c.want()
    for tile in TILES:
        y = c.run(tile).double().cpu()
        # below the smallest normal bf16 the rounding's half step is 2^-134
        assert ((y - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -23 * (32 + N // 32 + 20) * size + 2.0 ** -134).all()


def test_small_values_beside_large_ones():
    """A value is rounded to 2^-40 of its row's largest, a scale to 2^-35 of its column group's: the errors stay there."""
    M, N, K = 20, 128, 256
    c = Case(M, N, K, 128, exact=False)
    c.dy = c.dy.float()
    c.dy[:, 5] = c.dy.abs().amax(1) * 2.0 ** 34
    c.s = c.s.float()
    c.s[9, 1] = c.s[:, 1].max() * 2.0 ** 32
    c.dy, c.s = c.dy.bfloat16(), c.s.bfloat16()
    c.dev = [t.to(DEV) for t in (c.dy, c.w, c.s)]
    want, size = c.want()
    dtop = c.dy.double().abs().amax(1, keepdim=True) * 2.0 ** -40
    stop = (c.s.double().abs().amax(0, keepdim=True) * 2.0 ** -35).repeat_interleave(128, 1)
    w = int4_values(c.w, c.s, 128)
    lost = dtop * w.abs().sum(0, keepdim=True) + c.dy.double().abs().sum(1, keepdim=True) * 8 * stop + N * dtop * 8 * stop
    y = c.run().double().cpu()
    assert ((y - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -23 * (32 + N // 32 + 20) * size + lost).all()


@pytest.mark.parametrize("tile", TILES, ids=str)
def test_non_finite_values_stay_in_their_row_and_group(tile):
    c = Case(70, 200, 384, 32)
    base = c.run(tile).cpu()
    for v in (float("inf"), float("nan"), float("-inf")):
        dy, w, s = (t.clone() for t in c.dev)
        dy[69, 3] = v
        y = w4.w4a16_gemm_grad(dy, w, s, group_size=32, tile=tile).cpu()
        assert torch.equal(y[:69], base[:69]) and not y[69].isfinite().any()
        dy, w, s = (t.clone() for t in c.dev)
        s[199, 11] = v
        y = w4.w4a16_gemm_grad(dy, w, s, group_size=32, tile=tile).cpu()
        assert torch.equal(y[:, :352], base[:, :352]) and not y[:, 352:].isfinite().any()


def test_other_experts_do_not_reach_a_row():
    sizes = [19, 30, 0, 40]
    for tile in (None, (16, 1), (64, 1), (128, 1), (256, 1)):
        c = Case(95, 200, 256, 128, sizes)
        base = c.run(tile).clone()
        c.dev[0][19:49] = float("nan")
        c.dev[0][89:] = float("nan")
        c.dev[2][1:3] = float("nan")
        y = c.run(tile)
        assert torch.equal(y[:19], base[:19]) and torch.equal(y[49:89], base[49:89])
        assert y[19:49].isnan().all() and y[89:].isnan().all()


def test_no_rows():
    assert w4.w4a16_gemm_grad(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV),
                              torch.zeros(64, 64, dtype=torch.uint8, device=DEV),
                              torch.ones(64, 1, dtype=torch.bfloat16, device=DEV)).shape == (0, 128)


def test_weights_past_4_gib():
    G, N, K = 34, 16384, 16384
    w = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, device=DEV)
    s = (0.01 + 0.01 * torch.rand(G, N, K // 128, device=DEV)).bfloat16()
    sizes = [0] * (G - 2) + [3, 20]
    dy = torch.randn(23, N, device=DEV).bfloat16()
    d = w4.w4a16_gemm_grad(dy, w, s, m_sizes=torch.tensor(sizes, dtype=torch.int32, device=DEV), tile=(16, 1))
    for e, r in ((G - 2, slice(0, 3)), (G - 1, slice(3, 23))):
        assert torch.equal(d[r], w4.w4a16_gemm_grad(dy[r].clone(), w[e], s[e], tile=(16, 1)))


@pytest.mark.parametrize("M,N,K", [(140000, 64, 16384), (140000, 16384, 128)])
def test_rows_past_4_gib(M, N, K):
    """dX, then dY, of more than 2^32 bytes: some rows against calls of their own (whole numbers: exact)."""
    w = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.ones(N, K // 128, device=DEV).bfloat16()
    dy = torch.randint(-4, 5, (M, N), device=DEV, dtype=torch.int8).bfloat16()
    for sizes in (None, [M - 5]):
        m = None if sizes is None else torch.tensor(sizes, dtype=torch.int32, device=DEV)
        d = w4.w4a16_gemm_grad(dy, w if m is None else w[None], s if m is None else s[None], m_sizes=m,
                               dx=torch.full((M, K), 7.0, dtype=torch.bfloat16, device=DEV))
        last = M if m is None else M - 5
        for r in (0, 65500, 131000, last - 50):
            assert torch.equal(d[r:r + 50], w4.w4a16_gemm_grad(dy[r:r + 50], w, s))
        assert (d[last:] == 7).all()


@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (40, 2048, 256), (300, 512, 512)])
def test_captured_and_replayed(M, N, K):
    c = Case(M, N, K)
    wk = torch.empty(w4.w4a16_gemm_grad_workspace_bytes(1, M, N, K), dtype=torch.uint8, device=DEV)
    dx = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(None, dx, workspace=wk)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(None, dx, workspace=wk)
    for seed in range(1, 5):
        n = Case(M, N, K, seed=seed)
        for a, b in zip(c.dev, n.dev):
            a.copy_(b)
        dx.zero_()
        wk.fill_(255)
        graph.replay()
        eager = n.run()
        torch.cuda.synchronize()
        assert torch.equal(dx, eager) and torch.equal(eager.cpu(), n.want()[0].bfloat16()), seed


def test_streams_at_once_and_repeated():
    cases = [Case(200, 512, 1024, exact=False), Case(40, 2048, 256, 32, exact=False), Case(9, 64, 512, exact=False)]
    want = [c.run().clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for c, s in zip(cases, streams):
            y = torch.zeros(c.dy.shape[0], c.K, dtype=torch.bfloat16, device=DEV)
            s.wait_stream(torch.cuda.current_stream())
            outs.append(c.run(None, y, stream=s))
    torch.cuda.synchronize()
    for i, y in enumerate(outs):
        assert torch.equal(y, want[i % 3])
