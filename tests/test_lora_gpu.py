"""The projection with per-row low-rank adapters on the GPU against its 64-bit
definition, within the bound that operators_ref derives."""
import numpy as np
import pytest
import torch

import bf16_activation_quantized_amd as w4
import oracle
from gpu_util import bits_host, dev, nan_filled
from operators_ref import f64, lora_ref, sort_ref, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w4._lib()


class Case:
    def __init__(self, M, N, K, group, R, L, kind, seed, scaled=True):
        rng = np.random.default_rng(seed)
        self.group, self.M, self.N, self.K, self.R, self.L = group, M, N, K, R, L
        self.q = rng.integers(0, 16, (N, K), dtype=np.uint8)
        gen = torch.Generator().manual_seed(seed)
        self.x = torch.randn(M, K, generator=gen).bfloat16()
        self.s = (0.005 + 0.015 * torch.rand(N, K // group, generator=gen)).bfloat16()
        self.a = (torch.randn(L, R, K, generator=gen) * K ** -0.5).bfloat16()
        self.b = (torch.randn(L, N, R, generator=gen) * 0.3).bfloat16()
        self.sc = (0.5 + torch.rand(L, generator=gen)) if scaled else None
        if kind == "each":
            ids = np.arange(M) % L
        elif kind == "runs":
            ids = np.sort(rng.integers(0, L, M))
        elif kind == "none":
            ids = np.full(M, -1)
        else:
            ids = rng.integers(0, L, M)
        if kind == "holes":
            ids[rng.random(M) < 0.3] = -1
            ids[rng.random(M) < 0.1] = L
            ids[rng.random(M) < 0.1] = np.iinfo(np.int32).max
            ids[rng.random(M) < 0.1] = np.iinfo(np.int32).min
        self.ids = ids.astype(np.int32)
        d = dev()
        self.d = dict(x=self.x.to(d), w_packed=w4.w4a16_pack_int4(torch.from_numpy(self.q).to(d)), scales=self.s.to(d),
                      a=self.a.to(d), b=self.b.to(d), adapter_ids=torch.from_numpy(self.ids).to(d),
                      scaling=None if self.sc is None else self.sc.to(d))

    def run(self, **kw):
        return w4.w4a16_gemm_lora(**{**self.d, **kw}, group_size=self.group)

    def ref(self):
        sc = np.ones(self.L) if self.sc is None else f64(self.sc)
        return lora_ref(f64(self.x), self.q.astype(np.float64), f64(self.s), f64(self.a), f64(self.b), self.ids, sc,
                        self.group)


CASES = [
    # M, N, K, group, R, L, kind, split_k
    (1, 256, 512, 128, 16, 2, "each", 0),        # the tiny workload's size
    (1, 1, 128, 128, 8, 1, "each", 0),
    (1, 1001, 5120, 128, 16, 8, "rand", 0),
    (1, 777, 4096, 128, 64, 3, "rand", 2),
    (1, 1000, 1280, 128, 24, 3, "rand", 0),
    (1, 300, 9216, 128, 128, 2, "rand", 0),
    (1, 300, 1024, 128, 40, 2, "each", 16),
    (1, 64, 256, 128, 16, 2, "none", 0),
    (1, 4100, 512, 32, 16, 2, "each", 0),
    (2, 333, 640, 128, 32, 5, "each", 0),
    (3, 514, 1024, 128, 8, 2, "holes", 4),
    (7, 1023, 2048, 128, 72, 9, "holes", 0),
    (8, 512, 1152, 128, 128, 3, "rand", 1),
    (9, 257, 1024, 128, 16, 16, "each", 0),
    (13, 1030, 2560, 128, 56, 4, "holes", 2),
    (16, 2048, 4096, 128, 16, 16, "each", 0),
    (16, 96, 8192, 128, 128, 20, "holes", 8),
    (10, 100, 128, 128, 32, 3, "each", 0),       # 1, 3, 4, 5 and 12 stages of the LDS-staged kernel
    (11, 70, 1536, 128, 64, 11, "each", 0),
    (12, 1000, 2048, 128, 128, 4, "mixed", 1),
    (15, 130, 2560, 128, 96, 15, "each", 1),
    (16, 200, 6144, 128, 40, 7, "holes", 1),
    (16, 64, 1024, 128, 16, 16, "each", 16),     # more slices than groups
    (17, 640, 1024, 128, 16, 3, "runs", 0),
    (31, 1025, 896, 128, 48, 31, "each", 2),
    (33, 512, 1280, 128, 16, 4, "holes", 0),
    (48, 4096, 512, 128, 64, 6, "rand", 0),
    (49, 700, 384, 128, 16, 3, "rand", 0),
    (64, 896, 5120, 128, 32, 7, "holes", 0),
    (100, 257, 2048, 128, 128, 2, "runs", 4),
    (145, 1000, 640, 128, 104, 145, "each", 1),
    (200, 2048, 1024, 128, 16, 300, "rand", 0),
    (333, 8448, 256, 128, 64, 5, "runs", 1),     # row sums from the pre-pass
    (129, 8448, 384, 128, 8, 4, "holes", 2),
    (40, 257, 384, 32, 16, 3, "holes", 4),
    (5, 300, 128, 32, 8, 2, "rand", 0),
    (130, 2048, 512, 32, 64, 4, "runs", 2),
    (257, 513, 256, 32, 120, 6, "rand", 1),
    (300, 64, 128, 128, 16, 2, "none", 0),
    (1000, 40, 256, 128, 88, 3, "holes", 0),
    (4500, 48, 256, 128, 16, 5, "holes", 1),     # more rows than one grouping block
    (9000, 16, 128, 128, 8, 700, "rand", 0),
    (300, 64, 256, 128, 24, 9000, "holes", 0),   # more adapters than the grouping counts
    (70, 40, 640, 32, 8, 8193, "each", 0),
    (8, 520, 1024, 32, 128, 8, "each", 4),
]


@pytest.mark.parametrize("M,N,K,group,R,L,kind,sk", CASES)
def test_parity(M, N, K, group, R, L, kind, sk):
    c = Case(M, N, K, group, R, L, kind, seed=M * 3 + N + K + R, scaled=R % 16 == 0)
    buf = nan_filled((M * N + 64,))                     # guard behind the output
    buf[M * N:] = 7.0
    y = c.run(split_k=sk, y=buf[:M * N].view(M, N))
    torch.cuda.synchronize()
    ref, bound = c.ref()
    within(f64(y), ref, bound, f"lora {M}x{N}x{K}")
    assert oracle.gate(bits_host(y), ref)["ok"]
    assert (buf[M * N:] == 7.0).all()
    first = y.clone()
    assert torch.equal(first, c.run(split_k=sk))        # bitwise repeatable


@pytest.mark.parametrize("M,group,R", [(64, 128, 72), (128, 128, 40), (129, 32, 128), (191, 128, 24), (700, 128, 88)])
@pytest.mark.parametrize("sizes", [(1, 15, 16, 32), (17, 33, 14), (31, 1, 1, 1, 30), (48, 16), (64,), (63,), (2,) * 32])
def test_adapters_strewn_over_blocks(M, group, R, sizes):
    """Adapters with these numbers of rows, shuffled within each 64 rows (the
    rows behind them bare): x . A^T is formed in units of up to 16 such rows."""
    rng = np.random.default_rng(M + R + len(sizes))
    c = Case(M, 80, 384, group, R, len(sizes) + 2, "mixed", seed=M + R)
    ids = np.concatenate([rng.permutation(np.r_[np.repeat(rng.permutation(len(sizes) + 2)[:len(sizes)], sizes),
                                                np.full(64 - sum(sizes), -1)]) for _ in range(-(-M // 64))])[:M]
    c.ids = ids.astype(np.int32)
    ref, bound = c.ref()
    within(f64(c.run(adapter_ids=torch.from_numpy(c.ids).to(dev()))), ref, bound, f"strewn {M} {sizes}")


@pytest.mark.parametrize("M,group", [(1, 128), (6, 128), (14, 128), (30, 128), (45, 128), (333, 128), (333, 32),
                                     (2000, 128)])
@pytest.mark.parametrize("R", [8, 24, 40, 72, 88, 104, 120, 128])
@pytest.mark.parametrize("kind", ["mixed", "runs", "holes"])
def test_each_row_takes_its_own_scale(M, group, R, kind):
    """Scales that differ by adapter, at every kind of rank (the last rank tile
    full or half) and of row order."""
    c = Case(M, 96, 256, group, R, 5, kind, seed=M + R)
    c.sc = torch.tensor([1.0, -2.0, 4.0, 0.5, 8.0])
    ref, bound = c.ref()
    within(f64(c.run(scaling=c.sc.to(dev()))), ref, bound, f"scales {M} r{R}")


@pytest.mark.parametrize("M,N,K,group,sk", [(1, 512, 1024, 128, 0), (4, 512, 1024, 128, 0), (12, 512, 1024, 128, 2),
                                            (40, 512, 512, 128, 0), (100, 8448, 256, 128, 0), (100, 512, 256, 32, 2)])
def test_rows_without_adapter_equal_the_projection(M, N, K, group, sk):
    """A call whose rows have no adapter rounds the projection's own sum: the
    same values as w4a16_gemm, up to the order of its fp32 sums."""
    c = Case(M, N, K, group, 16, 2, "none", seed=M + N)
    ref, bound = c.ref()
    within(f64(c.run(split_k=sk)), ref, bound, "lora")
    y = w4.w4a16_gemm(c.d["x"], c.d["w_packed"], c.d["scales"], split_k=sk, group_size=group)
    within(f64(y), ref, bound, "gemm")


@pytest.mark.parametrize("M,N,K,group,R", [(1, 300, 512, 128, 16), (6, 300, 512, 128, 40), (14, 300, 512, 128, 16),
                                           (20, 300, 512, 128, 16), (150, 300, 512, 128, 64),
                                           (150, 300, 512, 32, 24)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_other_adapters_stay_out(M, N, K, group, R, bad):
    """Infinities and NaN in an adapter reach its own rows only (adapter 1 has
    them in A, adapter 3 in B and scaling; no row names adapter 4, all NaN)."""
    c = Case(M, N, K, group, R, 5, "rand", seed=M)
    c.ids[:] = np.arange(M) % 4
    if M == 1:
        c.ids[:] = 2
    c.d["adapter_ids"] = torch.from_numpy(c.ids).to(dev())
    want = c.run()
    a, b, sc = c.d["a"].clone(), c.d["b"].clone(), c.d["scaling"].clone()
    a[1, R - 1, 5] = bad
    b[3, 17] = bad
    a[4], b[4], sc[4] = float("nan"), float("nan"), float("nan")
    got = c.run(a=a, b=b, scaling=sc)
    clean = torch.from_numpy((c.ids == 0) | (c.ids == 2)).to(dev())
    assert torch.equal(got[clean], want[clean])
    for l in (1, 3):
        rows = torch.from_numpy(c.ids == l).to(dev())
        if rows.any():
            hit = got[rows] if l == 1 else got[rows][:, 17]
            assert not torch.isfinite(hit).any()
    # a bad row of x reaches no other row
    if M > 1:
        x = c.d["x"].clone()
        x[0] = bad
        got = c.run(x=x)
        assert torch.equal(got[1:], want[1:]) and not torch.isfinite(got[0]).any()


@pytest.mark.parametrize("M,N,K,group,R,sk", [(1, 300, 1024, 128, 16, 0), (1, 300, 1280, 128, 16, 0),
                                              (5, 300, 1024, 128, 40, 2), (14, 300, 512, 128, 128, 0),
                                              (40, 300, 512, 128, 128, 0), (100, 8448, 256, 128, 64, 1),
                                              (300, 300, 512, 32, 16, 4)])
def test_workspace_is_written_before_it_is_read(M, N, K, group, R, sk):
    """A workspace full of NaN, of the size asked for, gives the same result."""
    c = Case(M, N, K, group, R, 4, "holes", seed=M + R)
    if M == 1:
        c.d["adapter_ids"].fill_(2)
    need = w4.w4a16_gemm_lora_workspace_bytes(M, N, K, 4, R, sk, group)
    ws = torch.full((need // 4 + 16,), float("nan"), device=dev())
    ws[need // 4:] = 5.0
    got = c.run(split_k=sk, workspace=ws[:need // 4])
    assert torch.equal(got, c.run(split_k=sk)) and torch.isfinite(got).all()
    assert (ws[need // 4:] == 5.0).all()


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own."""
    cases = [Case(200, 2048, 1024, 128, 32, 6, "mixed", seed=1), Case(12, 4096, 2048, 128, 16, 12, "each", seed=2)]
    want = [c.run().clone() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, c in enumerate(cases):
            got[i].append(c.run(stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in (0, 1) for y in got[i])


def test_binding_refuses_what_does_not_fit():
    c = Case(4, 64, 256, 128, 8, 2, "each", seed=3)
    d = c.d
    for kw in (dict(x=d["x"][:, :128]), dict(x=d["x"][0]), dict(w_packed=d["w_packed"][:, :64].contiguous()),
               dict(scales=d["scales"][:32]), dict(a=d["a"][:1]), dict(a=d["a"][0]), dict(b=d["b"].transpose(1, 2)),
               dict(adapter_ids=d["adapter_ids"][:3]), dict(scaling=d["scaling"][:1]),
               dict(y=torch.empty(4, 65, dtype=torch.bfloat16, device=dev())), dict(x=d["x"].cpu()),
               dict(scaling=d["scaling"].cpu())):
        with pytest.raises(ValueError):
            c.run(**kw)
    for kw in (dict(x=d["x"].half()), dict(adapter_ids=d["adapter_ids"].long()), dict(scaling=d["scaling"].double()),
               dict(a=None), dict(workspace=torch.zeros(1 << 16, dtype=torch.int32, device=dev()))):
        with pytest.raises(TypeError):
            c.run(**kw)
    with pytest.raises(w4.W4A16Error) as e:
        c.run(workspace=torch.zeros(4, device=dev()))
    assert e.value.status == 5
    with pytest.raises(w4.W4A16Error) as e:
        c.run(a=d["a"][:, :4].contiguous(), b=d["b"][:, :, :4].contiguous())    # rank 4
    assert e.value.status == 2


def test_no_rows():
    c = Case(4, 64, 128, 128, 8, 2, "each", seed=1)
    y = c.run(x=c.d["x"][:0], adapter_ids=c.d["adapter_ids"][:0])
    assert y.shape == (0, 64)


def test_adapters_past_32_bit_offsets():
    """5.4 GB of A: the last adapter is found."""
    L, R, K, N = 5200, 128, 4096, 128
    c = Case(3, N, K, 128, R, 2, "each", seed=5)
    a = torch.zeros(L, R, K, dtype=torch.bfloat16, device=dev())
    b = torch.zeros(L, N, R, dtype=torch.bfloat16, device=dev())
    sc = torch.zeros(L, device=dev())
    a[-1], b[-1], sc[-1] = c.d["a"][1], c.d["b"][1], c.d["scaling"][1]
    a[-2], b[-2], sc[-2] = c.d["a"][0], c.d["b"][0], c.d["scaling"][0]
    ids = c.d["adapter_ids"] + (L - 2)
    assert torch.equal(c.run(a=a, b=b, scaling=sc, adapter_ids=ids), c.run())


@pytest.mark.parametrize("M,N,K", [(1, 1024, 2560), (16, 1024, 2048), (40, 1024, 1024), (300, 8448, 512)])
def test_side_stream_and_graph_replays(M, N, K):
    c = Case(M, N, K, 128, 32, 6, "holes", seed=M)
    want = c.run().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = c.run(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = c.run()
    for _ in range(4):
        cap.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap, want)
        c.run()
        torch.cuda.synchronize()


def test_experts_and_adapters_together():
    """As used: a shared projection with the requests' adapters, its rows sorted
    by expert (two of six, some tokens padded), gathered, multiplied by the
    experts' grouped weights, combined with the router's weights; then the
    gradients back to the rows of the projection."""
    M, N1, K, G, N2, k = 70, 256, 384, 6, 200, 2
    c = Case(M, N1, K, 128, 16, 3, "holes", seed=77)
    h = c.run()
    rng = np.random.default_rng(7)
    ids = rng.integers(0, G, (M, k)).astype(np.int32)
    ids[ids == 4] = 5                                   # an expert without rows
    ids[rng.random(M) < 0.2] = -1
    q = rng.integers(0, 16, (G, N2, N1), dtype=np.uint8)
    s = (0.005 + 0.015 * torch.rand(G, N2, N1 // 128, generator=torch.Generator().manual_seed(3))).bfloat16()
    w = torch.softmax(torch.randn(M, k, generator=torch.Generator().manual_seed(4)), dim=1)
    order, pos, sizes = w4.w4a16_expert_sort(torch.from_numpy(ids).to(dev()), G)
    ro, rp, rs = sort_ref(ids, G)
    kept = int(rs.sum())
    xs = w4.w4a16_expert_gather(h, pos)
    z = torch.full((M * k, N2), 7.0, dtype=torch.bfloat16, device=dev())
    w4.w4a16_gemm_grouped(xs, w4.w4a16_pack_int4(torch.from_numpy(q).to(dev())), s.to(dev()), sizes, y=z)
    y = w4.w4a16_expert_combine(z, pos, w.to(dev()))
    assert (z[kept:] == 7.0).all()                      # rows behind the last expert: left as they were

    # the same in 64 bits from the bf16 rows of the step before
    hd = f64(h)
    sf = np.repeat(f64(s), 128, axis=2)
    zr = np.zeros((kept, N2))
    for r in range(kept):
        t = ro[r] // k
        g = ids[t, ro[r] % k]
        zr[r] = (sf[g] * (q[g] - 8.0)) @ hd[t]
    got = f64(z[:kept])
    assert np.max(np.abs(got - zr)) <= 4e-3 * np.max(np.abs(zr)) + 1e-3
    yr = np.zeros((M, N2))
    for t in range(M):
        for j in range(k):
            if rp[t, j] >= 0:
                yr[t] += float(w[t, j]) * got[rp[t, j]]
    assert np.max(np.abs(f64(y) - yr)) <= 2.0 ** -8 * np.max(np.abs(yr)) + 1e-5
    dy = torch.randn(M, N2, generator=torch.Generator().manual_seed(5)).bfloat16().to(dev())
    dz, dw = w4.w4a16_expert_combine_grad(dy, z, pos, w.to(dev()))
    dwr = np.array([[np.dot(f64(dy)[t], got[rp[t, j]]) if rp[t, j] >= 0 else 0.0 for j in range(k)] for t in range(M)])
    assert np.max(np.abs(f64(dw) - dwr)) <= N2 * 2.0 ** -24 * np.max(np.abs(f64(dy))) * np.max(np.abs(got)) * N2
    assert torch.isfinite(dz[:kept]).all()
