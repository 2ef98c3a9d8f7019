"""The widest rows of the 8-bit products and the input gradients (CPU only: no
kernel is launched). The tile kernels address the rows of a tile with 32-bit
offsets, those past the last row too: one that wrapped would come to lie in the
rows that are there. And the most tiles: a launch of 2^32 threads or more is cut
short without an error."""
import ctypes
import os

import pytest
import torch

import bf16_activation_quantized_amd as w4

OK, ERR_SHAPE = 0, 2
LIMIT = (1 << 32) - 1


@pytest.fixture()
def lib():
    # fake device pointers that validation must reject: only where no GPU could run them
    if torch.cuda.is_available():
        pytest.skip("host-only checks: a GPU is visible")
    if not os.path.exists(w4.LIB_PATH):
        pytest.skip("libw4a16.so not built")
    return w4._lib()


def choice(f, *args):
    bm, sk = ctypes.c_int32(-1), ctypes.c_int32(-1)
    return f(*args, ctypes.byref(bm), ctypes.byref(sk)), bm.value


FP8 = [  # grad, G (0: plain), M, N, K
    (0, 0, 65, 33038208, 128), (0, 0, 130, 16500000, 128), (0, 2, 70, 30000000, 128), (1, 0, 65, 128, 33030144),
    (1, 0, 33, 33030144, 128), (0, 0, 17, 33554304, 128), (0, 0, 255, 8421376, 128), (1, 3, 40, 128, 33030144),
    (0, 0, 20, 8, (1 << 24) - 128), (0, 0, 1, 128, 9728), (0, 0, 1, 128, 1 << 14),
]


@pytest.mark.parametrize("grad,G,M,N,K", FP8)
def test_rows_of_a_tile_fit_its_offsets(lib, grad, G, M, N, K):
    status, bm = choice(lib.w4a16_fp8_gemm_auto, grad, int(G > 0), max(G, 1), M, N, K)
    assert status == OK
    row = max(N, 2 * K) if grad else max(K, 2 * N)
    assert bm == 16 and M <= 16 * max(G, 1) or bm * row <= LIMIT
    assert grad or (64 if bm == 16 else 256) * K <= LIMIT


@pytest.mark.parametrize("G,M,N,K,gs", [(1, 65, 8, 33030144, 128), (1, 33, 33030144, 128, 32), (1, 1, 8, (1 << 27) - 128, 128),
                                        (4, 200, 10000000, 128, 128), (1, 130, 8, 16500096, 32)])
def test_rows_of_a_gradients_tile_fit_its_offsets(lib, G, M, N, K, gs):
    status, bm = choice(lib.w4a16_gemm_grad_auto, int(G > 1), G, M, N, K, gs)
    assert status == OK
    assert bm * 2 * max(-(-N // 128) * 128, K) <= LIMIT


A = ctypes.c_void_p(0x10000)


@pytest.mark.parametrize("grad,M,N,K,bm", [
    (1, 1, 128, 1 << 26, 0),                            # 32 rows of dX: 2^32 bytes
    (0, 1, 8, 1 << 28, 0), (0, 17, 8, 1 << 24, 0),   # 256 columns' weights
    (0, 65, 33038208, 128, 96), (1, 65, 128, 33030144, 256),
])
def test_wider_rows_are_refused(lib, grad, M, N, K, bm):
    assert lib.w4a16_fp8_gemm_ex(grad, A, A, A, A, None, A, 1, M, N, K, bm, 1, None, 0, None) == ERR_SHAPE
    if bm == 0:
        assert choice(lib.w4a16_fp8_gemm_auto, grad, 0, 1, M, N, K)[0] == ERR_SHAPE
        size = lib.w4a16_fp8_gemm_grad_workspace_bytes if grad else lib.w4a16_fp8_gemm_workspace_bytes
        assert size(M, N, K) == 0


def test_wider_rows_by_expert_are_refused(lib):
    # (2^26 and more: 64 columns' weights of the kernel for few rows)
    assert lib.w4a16_fp8_gemm_grouped(A, A, A, A, A, A, 3, 20, 8, 1 << 26, None) == ERR_SHAPE
    assert choice(lib.w4a16_fp8_gemm_auto, 0, 1, 3, 20, 8, (1 << 26) - 128) == (OK, 16)


@pytest.mark.parametrize("M,N,K,bm", [(1, 8, 1 << 28, 0), (65, 8, 33030144, 96), (33, 33030144, 128, 128)])
def test_a_gradients_wider_rows_are_refused(lib, M, N, K, bm):
    assert lib.w4a16_gemm_grad_ex(A, A, A, None, A, 1, M, N, K, 128, bm, 1, A, 1 << 60, None) == ERR_SHAPE
    assert lib.w4a16_gemm_grad_workspace_bytes_ex(1, M, N, K, 128, bm, 1) == 0
    if bm == 0:
        assert choice(lib.w4a16_gemm_grad_auto, 0, 1, M, N, K, 128)[0] == ERR_SHAPE


# ------------------------------------------------------------------ threads of a launch

BLOCKS = 1 << 23      # workgroups of 512 threads


def tiles_bound(M, bm, G):
    return (M + (bm - 1) * min(G, M)) // bm


@pytest.mark.parametrize("grad,G,M,N,K", [
    (0, 1 << 17, 1 << 17, 4096, 128),         # one row each: 2^17 tiles of 16 rows, 64 of 64 columns
    (0, 1 << 20, 1 << 24, 512, 128),          # 16 rows each
    (0, 1 << 19, 1 << 24, 2048, 128),         # 32 rows each: all heights of the tile kernel
    (1, 1 << 19, 1 << 24, 128, 2048), (1, 1 << 19, 1 << 24, 128, 2176), (1, 1 << 21, 1 << 21, 128, 1024),
])
def test_more_tiles_than_a_launch_takes_are_refused(lib, grad, G, M, N, K):
    status, bm = choice(lib.w4a16_fp8_gemm_auto, grad, 1, G, M, N, K)
    # (32 rows each: 2^19 + 31 / 32 2^19 tiles at most, just below the limit with 8 of 256 columns)
    least, cols = (32, 256) if grad else (16, 64)
    if tiles_bound(M, least, G) * -(-(K if grad else N) // cols) >= BLOCKS:
        assert lib.w4a16_fp8_gemm_ex(grad, A, A, A, A, A, A, G, M, N, K, least, 0, None, 0, None) == ERR_SHAPE
    if status == OK:          # (a taller tile)
        assert bm >= 32 and tiles_bound(M, bm, G) * -(-(K if grad else N) // 256) < BLOCKS
    else:
        assert status == ERR_SHAPE
        call = lib.w4a16_fp8_gemm_grouped(A, A, A, A, A, A, G, M, N, K, None) if not grad else \
            lib.w4a16_fp8_gemm_grad(A, A, A, A, A, A, G, M, N, K, None, 0, None)
        assert call == ERR_SHAPE


def test_the_most_tiles_that_a_launch_takes(lib):
    G = (1 << 17) - 1
    assert choice(lib.w4a16_fp8_gemm_auto, 0, 1, G, G, 4096, 128) == (OK, 16)          # 64 G workgroups
    assert choice(lib.w4a16_fp8_gemm_auto, 0, 1, G + 1, G + 1, 4096, 128)[1] != 16


def test_rows_of_a_forced_height(lib):
    # the kernel for few rows takes 16 rows per y of its grid
    assert lib.w4a16_fp8_gemm_ex(0, A, A, A, A, None, A, 1, 16 * 65535 + 1, 64, 128, 16, 0, None, 0, None) == ERR_SHAPE


@pytest.mark.parametrize("G,M,N,K,gs", [
    (1 << 21, 1 << 21, 8, 1024, 128),         # tiles: 4 columns of each expert's one row
    (1 << 20, 64, 1024, 128, 128),            # blocks of scales
    (64, 64, 1 << 24, 128, 128),              # as many by longer rows
    (1 << 17, 64, 128, 131072, 32),           # by wider rows of scales
])
def test_a_gradients_launches(lib, G, M, N, K, gs):
    assert choice(lib.w4a16_gemm_grad_auto, 1, G, M, N, K, gs)[0] == ERR_SHAPE
    assert lib.w4a16_gemm_grad(A, A, A, A, A, G, M, N, K, gs, A, 1 << 60, None) == ERR_SHAPE
    assert lib.w4a16_gemm_grad_workspace_bytes(G, M, N, K, gs) == 0


def test_the_most_scales_of_a_launch(lib):
    # 2^20 - 1 experts of 8 blocks of 128 x 1, and 2 workgroups of rows
    assert choice(lib.w4a16_gemm_grad_auto, 1, (1 << 20) - 1, 16, 1024, 128, 128)[0] == OK
