"""sort, gather, grouped product and combine as one run, every step held to a
bound that is derived: the projection's of operators_ref for the grouped
product, from the gathered rows themselves."""
import numpy as np
import pytest
import torch

import bf16_activation_quantized_amd as w4
from gpu_util import dev
from operators_ref import combine_ref, f64, gather_ref, lora_ref, sort_ref, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w4._lib()


@pytest.mark.parametrize("T,k,G,K,N,group", [
    (70, 2, 6, 256, 200, 128), (1, 4, 8, 640, 96, 128), (333, 3, 7, 5376, 264, 128), (300, 4, 16, 512, 520, 32),
    (1000, 2, 3, 384, 72, 128), (40, 8, 100, 256, 64, 32),
])
def test_run_of_all_four(T, k, G, K, N, group):
    rng = np.random.default_rng(T + G)
    ids = rng.integers(0, G, (T, k)).astype(np.int32)
    ids[ids == G // 2] = (G // 2 + 1) % G                # an expert without rows
    ids[rng.random((T, k)) < 0.15] = -1
    ids[0, 0] = 0
    gen = torch.Generator().manual_seed(T)
    x = torch.randn(T, K, generator=gen).bfloat16()
    q = rng.integers(0, 16, (G, N, K), dtype=np.uint8)
    s = (0.005 + 0.015 * torch.rand(G, N, K // group, generator=gen)).bfloat16()
    w = torch.softmax(torch.randn(T, k, generator=gen), dim=1)
    order, pos, sizes = w4.w4a16_expert_sort(torch.from_numpy(ids).to(dev()), G)
    ro, rp, rs = sort_ref(ids, G)
    assert np.array_equal(order.cpu().numpy(), ro) and np.array_equal(pos.cpu().numpy(), rp)
    assert np.array_equal(sizes.cpu().numpy(), rs)
    xs = w4.w4a16_expert_gather(x.to(dev()), pos, xs=torch.full((T * k, K), 7.0, dtype=torch.bfloat16, device=dev()))
    assert np.array_equal(f64(xs), gather_ref(f64(x), rp, np.full((T * k, K), 7.0)))
    z = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device=dev())
    w4.w4a16_gemm_grouped(xs, w4.w4a16_pack_int4(torch.from_numpy(q).to(dev())), s.to(dev()), sizes, y=z,
                          group_size=group)
    r0, none = 0, np.zeros(0)
    for g in range(G):                                   # each expert's rows: a projection without adapters
        r1 = r0 + int(rs[g])
        if r1 > r0:
            ref, bound = lora_ref(f64(xs[r0:r1]), q[g].astype(np.float64), f64(s[g]), np.zeros((1, 8, K)),
                                  np.zeros((1, N, 8)), np.full(r1 - r0, -1), none, group)
            within(f64(z[r0:r1]), ref, bound, f"expert {g}")
        r0 = r1
    assert (z[r0:] == 7.0).all()                         # rows behind the last expert: left as they were
    y = w4.w4a16_expert_combine(z, pos, w.to(dev()))
    within(f64(y), *combine_ref(f64(z), rp, f64(w)), "combine")


def test_streams_by_address_and_threads():
    """A stream given by its address (and 0, the default stream), outputs made by
    the calls; no weights; and two host threads, each on a stream of its own."""
    import threading

    T, k, G, width = 500, 3, 9, 520
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(T, width, generator=gen).bfloat16().to(dev())
    ids = torch.randint(-1, G + 1, (T, k), generator=gen, dtype=torch.int32).to(dev())
    a, b = (torch.randn(4, *s, generator=gen).bfloat16().to(dev()) for s in ((16, 512), (64, 16)))
    q = torch.randint(0, 256, (64, 256), generator=gen, dtype=torch.uint8).to(dev())
    s = torch.ones(64, 4, dtype=torch.bfloat16, device=dev())
    who = (torch.arange(T) % 5).int().to(dev())
    xc = x[:, :512].contiguous()

    def calls(stream):
        order, pos, sizes = w4.w4a16_expert_sort(ids, G, stream=stream)
        kept = int((pos >= 0).sum()) if stream is None else None
        xs = w4.w4a16_expert_gather(x, pos, stream=stream)
        y = w4.w4a16_expert_combine(xs, pos, stream=stream)
        return kept, (order, pos, sizes, y, w4.w4a16_gemm_lora(xc, q, s, a, b, who, stream=stream))

    kept, want = calls(None)
    torch.cuda.synchronize()
    ro, rp, rs = sort_ref(ids.cpu().numpy(), G)
    assert kept == rs.sum()
    xs = gather_ref(f64(x), rp, np.zeros((T * k, width)))
    within(f64(want[3]), *combine_ref(xs, rp, None), "combine without weights")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side.cuda_stream, 0):
        torch.cuda.synchronize()
        got = calls(stream)[1]
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(want, got))
    bad = []

    def work():
        mine = torch.cuda.Stream()
        with torch.cuda.stream(mine):
            for _ in range(20):
                got = calls(mine)[1]
                mine.synchronize()
                if not all(torch.equal(u, v) for u, v in zip(want, got)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
