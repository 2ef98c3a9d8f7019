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
