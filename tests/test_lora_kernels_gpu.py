"""The projection with adapters in every kernel that its automatic choice can
reach: each tile height, each GEMV geometry with and without the ring, each
small-batch instance, and both kernels of x . A^T on both sides of their
borders. The choice is asserted, so that a change of it cannot drop a kernel
from here unnoticed."""
import math

import numpy as np
import pytest
import torch

import bf16_activation_quantized_amd as w4
from gpu_util import dev, nan_filled
from operators_ref import f64, lora_ref, within
from test_lora_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w4._lib()


def check(c, sk=0, cols=None):
    """The call against the 64-bit definition, in full or at some columns
    (columns do not depend on each other), with guard rows behind."""
    M, N = c.M, c.N
    buf = nan_filled((M * N + 64,))
    buf[M * N:] = 7.0
    y = c.run(split_k=sk, y=buf[:M * N].view(M, N))
    cols = np.arange(N) if cols is None else cols
    sc = np.ones(c.L) if c.sc is None else f64(c.sc)
    t = torch.from_numpy(cols)
    ref, bound = lora_ref(f64(c.x), c.q[cols].astype(np.float64), f64(c.s[t]), f64(c.a), f64(c.b[:, t]), c.ids, sc,
                          c.group)
    within(f64(y[:, t.to(dev())]), ref, bound, f"lora {M}x{N}x{c.K} g{c.group} r{c.R}")
    assert torch.isfinite(y).all() and (buf[M * N:] == 7.0).all()


def some(N, n=160):
    """The first and last columns, and some between."""
    return np.unique(np.r_[np.arange(24), np.linspace(0, N - 1, n).astype(int), np.arange(N - 24, N)])


HEIGHTS = [
    # group, rows of a tile, M, N, K; up to 31 column tiles at group 128 and 7 at
    # group 32 the kernel forms the row sums itself, above they come from ahead
    (128, 48, 200, 776, 384), (128, 64, 6178, 264, 128), (128, 80, 8252, 264, 128), (128, 96, 5141, 776, 128),
    (128, 112, 6178, 776, 128), (128, 128, 7215, 776, 128), (128, 144, 8252, 776, 128),
    (128, 48, 200, 8200, 384), (128, 64, 383, 8200, 128), (128, 80, 505, 8200, 256), (128, 96, 566, 8200, 384),
    (128, 112, 688, 8200, 256), (128, 128, 810, 8200, 384), (128, 144, 932, 8200, 256),
    (32, 80, 200, 264, 256), (32, 96, 5141, 776, 128), (32, 112, 6178, 776, 128), (32, 128, 7215, 776, 128),
    (32, 80, 200, 2304, 384), (32, 96, 566, 8200, 256), (32, 112, 688, 8200, 128), (32, 128, 810, 8200, 256),
]


@pytest.mark.parametrize("group,rows,M,N,K", HEIGHTS)
@pytest.mark.parametrize("R,L,kind", [(24, 11, "holes"), (64, 4, "runs"), (128, 5, "holes")])
def test_every_tile_height(group, rows, M, N, K, R, L, kind):
    """More adapters than are in flight at once, mixed with bare rows; requests
    one after the other; and a last tile that is not full."""
    assert w4.w4a16_gemm_auto_config(M, N, K, group) == (w4.PATH_TILE, rows, 1)
    assert M % rows != 0
    check(Case(M, N, K, group, R, L, kind, seed=M + rows + R), cols=some(N))


@pytest.mark.parametrize("M,N,K,group,R,L,kind,rows,sk", [
    (1322, 19456, 2560, 128, 64, 4, "runs", 144, 1), (512, 8192, 8192, 128, 64, 8, "mixed", 128, 2),
    (1000, 5120, 5120, 128, 128, 8, "mixed", 96, 1), (200, 4096, 4096, 128, 128, 8, "holes", 64, 4),
    (333, 2560, 9728, 32, 24, 5, "holes", 112, 8),
])
def test_whole_projections(M, N, K, group, R, L, kind, rows, sk):
    """The sizes of the measured workloads, long K among them."""
    assert w4.w4a16_gemm_auto_config(M, N, K, group) == (w4.PATH_TILE, rows, sk)
    check(Case(M, N, K, group, R, L, kind, seed=M), cols=some(N))


def gemv_rows(gps):
    """Weight rows of a block of the GEMV's matrix-core layout for slices of gps
    groups, or 0 where it has none and the small-batch kernel takes the call."""
    r = 16 // math.gcd(gps, 16)
    return r if r <= 4 and r * gps <= 128 else 0


GEMV_GROUPS = [16, 32, 48, 64, 8, 24, 40, 56, 4, 12, 20, 28]


@pytest.mark.parametrize("gps", GEMV_GROUPS)
@pytest.mark.parametrize("ring", [False, True])
def test_every_gemv_geometry(gps, ring):
    """One request: few blocks of rows per wave, or two and more, where the next
    block is requested before the current one is consumed."""
    rows = gemv_rows(gps)
    N, K = (4099 if ring else 250) * rows + 1, 128 * gps
    assert rows > 0 and w4.w4a16_gemm_auto_config(1, N, K) == (w4.PATH_GEMV, 0, 1)
    R = (8, 24, 64, 128)[GEMV_GROUPS.index(gps) % 4]
    check(Case(1, N, K, 128, R, 3, "rand", seed=gps + ring, scaled=True), cols=some(N))


@pytest.mark.parametrize("N,K,R,sk", [
    (17408, 5120, 16, 0), (17408, 5120, 128, 0),    # pieces of B past one per thread
    (70001, 512, 64, 0), (130001, 512, 128, 0),     # more columns than 256 for each compute unit
    (131073, 1024, 128, 2), (70000, 2048, 72, 0),
    (1000, 6656, 40, 16),                           # 13 slices with groups, 3 without
    (333, 2048, 128, 4), (333, 8192, 16, 16),
])
def test_gemv_of_many_columns_and_slices(N, K, R, sk):
    path, variant, split = w4.w4a16_gemm_auto_config(1, N, K)
    assert path == w4.PATH_GEMV and gemv_rows(-(-(K // 128) // (sk or split))) > 0
    c = Case(1, N, K, 128, R, 2, "rand", seed=N + R)
    check(c, sk, cols=some(N))
    need = w4.w4a16_gemm_lora_workspace_bytes(1, N, K, 2, R, sk)
    ws = torch.full((need // 4 + 16,), float("nan"), device=dev())
    got = c.run(split_k=sk, workspace=ws[:need // 4])
    assert torch.equal(got, c.run(split_k=sk)) and torch.isnan(ws[need // 4:]).all()


@pytest.mark.parametrize("K", [512, 1024, 2560])
@pytest.mark.parametrize("R", [8, 24, 72, 128])
def test_gemv_takes_its_adapters_scale(K, R):
    for l in range(5):
        c = Case(1, 333, K, 128, R, 5, "rand", seed=K + R)
        c.sc = torch.tensor([1.0, -2.0, 4.0, 0.5, 8.0])
        c.d["scaling"] = c.sc.to(dev())
        c.ids[:] = l
        c.d["adapter_ids"].fill_(l)
        check(c)


@pytest.mark.parametrize("M", [1, 3, 7, 9, 16, 20, 30, 36, 45])
@pytest.mark.parametrize("R", [24, 64, 128])
@pytest.mark.parametrize("K", [640, 33024])
def test_every_small_batch_instance(M, R, K):
    """Each number of row quads and of rank steps; 33024: more scale groups than
    the kernel keeps in LDS."""
    path, _, split = w4.w4a16_gemm_auto_config(M, 72, K, 128)
    assert path == (w4.PATH_GEMV if M == 1 else w4.PATH_SKINNY)
    assert M > 1 or gemv_rows(-(-(K // 128) // split)) == 0      # a slice that the GEMV has no adapters for
    check(Case(M, 72, K, 128, R, 7, "holes" if M > 1 else "rand", seed=M + R + K), sk=1 if M > 1 else 0)


@pytest.mark.parametrize("N,group", [(64, 128), (8448, 128), (2048, 32), (72, 32)])
@pytest.mark.parametrize("M", [63, 64, 127, 128, 255, 256, 512, 513])
def test_borders_of_the_first_product(M, N, group):
    """504 to 4104 rows times ranks, on both sides of each number of ranks per
    workgroup and of the row tiles, alone and with the row sums in one launch."""
    check(Case(M, N, 256, group, 8, 9, "holes", seed=M + N), sk=1, cols=some(N))


@pytest.mark.parametrize("M,R,L", [(2500, 128, 64), (2500, 128, 700), (1337, 128, 3), (5000, 64, 40), (300, 24, 9000)])
@pytest.mark.parametrize("group", [128, 32])
def test_blocks_of_more_units_than_workgroups(M, R, L, group):
    """Up to 64 adapters strewn over each 64 rows, taken in turns by fewer
    workgroups; ids of up to 14 bits."""
    check(Case(M, 40, 256, group, R, L, "holes", seed=M + L), sk=1)
