"""The 8-bit product of up to 16 rows where each workgroup takes several column
tiles one after the other (more than two tiles of 16 columns per compute unit),
whole numbers bit for bit: one block per wave and tile and several, contractions
that end within the waves, the last round with and without a tile for each
workgroup, rows that leave one workgroup per compute unit."""
import ctypes

import pytest
import torch

import bf16_activation_quantized_amd as w4
from test_fp8_gpu import DEV, Case, same

pytestmark = pytest.mark.gpu


def columns_in_flight():
    """Output columns that all workgroups take at once, two per compute unit."""
    return 2 * 16 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("K", [128, 1024, 1152, 2176, 4224])
@pytest.mark.parametrize("over", [1, 16 * 7 + 5, None], ids=str)
def test_several_column_tiles(K, over):
    """A tile more than the workgroups, a few more and one that is not whole, two rounds more and a bit."""
    n = columns_in_flight()
    N = n + over if over is not None else 3 * n + 100
    full = Case(16, N, K)
    want = full.want()[0]
    x, xs, w, ws = full.dev
    for M in (1, 2, 7, 8, 9, 15, 16):
        bm, sk = ctypes.c_int32(), ctypes.c_int32()
        assert w4._lib().w4a16_fp8_gemm_auto(0, 0, 1, M, N, K, ctypes.byref(bm), ctypes.byref(sk)) == 0 and bm.value == 16
        y = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
        w4.w4a16_fp8_gemm(x[:M], xs[:M], w, ws, y=y[:M])
        assert same(y[:M], want[:M]) and (y[M] == 7).all(), M


@pytest.mark.parametrize("M,K", [(8, 9728), (16, 8192), (16, 9216), (5, 16384)])
def test_rows_that_leave_one_workgroup_per_compute_unit(M, K):
    N = columns_in_flight() + 37
    c = Case(M, N, K)
    assert same(c.run(), c.want()[0])


def test_the_ends_of_every_array():
    """Scales, weights and rows that end where other tensors' NaN begin: nothing behind them reaches an output."""
    N, K, M = 2 * columns_in_flight() + 3, 1152, 11
    c = Case(M, N, K)
    want = c.want()[0]

    def framed(t):
        wide = torch.full((t.numel() + 65536,), 0x7F, dtype=torch.uint8, device=DEV).view(t.dtype) \
            if t.element_size() == 1 else torch.full((t.numel() + 65536,), float("nan"), device=DEV)
        wide[:t.numel()] = t.reshape(-1)
        return wide[:t.numel()].view(t.shape)
    c.dev = [framed(t) for t in c.dev]
    assert same(c.run(), want)
