"""Which kernel, tile height and split the 8-bit products and the input gradients
take by themselves (CPU only; 256 compute units, as where no device is)."""
import ctypes
import os

import pytest
import torch

import bf16_activation_quantized_amd as w4

HEIGHTS = (16, 32, 64, 96, 128, 160, 192, 224, 256)


@pytest.fixture()
def lib():
    if torch.cuda.is_available():
        pytest.skip("the choice goes by the device's compute units")
    if not os.path.exists(w4.LIB_PATH):
        pytest.skip("libw4a16.so not built")
    return w4._lib()


def choice(f, *args):
    bm, sk = ctypes.c_int32(), ctypes.c_int32()
    assert f(*args, ctypes.byref(bm), ctypes.byref(sk)) == 0
    return bm.value, sk.value


def fp8(lib, grad, G, M, N, K):
    return choice(lib.w4a16_fp8_gemm_auto, grad, int(G > 0), max(G, 1), M, N, K)


def w4_grad(lib, G, M, N, K, gs=128):
    return choice(lib.w4a16_gemm_grad_auto, int(G > 0), max(G, 1), M, N, K, gs)


@pytest.mark.parametrize("args,want", [
    ((0, 0, 1, 17408, 5120), (16, 1)), ((0, 0, 16, 8192, 8192), (16, 1)), ((0, 0, 1322, 19456, 2560), (256, 1)),
    ((0, 0, 8192, 8192, 8192), (256, 1)), ((0, 64, 96, 2048, 4096), (16, 1)), ((0, 32, 16384, 2048, 4096), (256, 1)),
    ((1, 0, 777, 9728, 2560), (160, 5)), ((1, 8, 4096, 2048, 4096), (160, 1)),
])
def test_the_8_bit_calls_of_the_design_notes(lib, args, want):
    assert fp8(lib, *args) == want


def test_the_4_bit_gradients_of_the_design_notes(lib):
    assert w4_grad(lib, 0, 1322, 19456, 2560) == (224, 4)
    assert w4_grad(lib, 8, 2048, 2048, 4096, 32) == (192, 1)


@pytest.mark.parametrize("N,K", [(17408, 5120), (8192, 8192), (100, 128), (4096, 9728)])
def test_up_to_16_rows_take_their_kernel_where_they_fit(lib, N, K):
    for M in range(1, 17):
        fits = 16384 + (K // 128 + 1) * (8 if M <= 8 else 16) * 128 + K // 128 * (8 if M <= 8 else 16) * 4 <= 160 * 1024
        bm, sk = fp8(lib, 0, 0, M, N, K)
        assert (bm == 16 and sk == 1) if fits else bm in (32, 64)
    assert fp8(lib, 0, 0, 17, N, K)[0] > 16 and fp8(lib, 1, 0, 1, N // 128 * 128 or 128, K)[0] > 16
    for G in (1, 8, 100):
        assert fp8(lib, 0, G, 16 * G, N, K) == (16, 1) and fp8(lib, 0, G, 16 * G + 1, N, K)[0] > 16


@pytest.mark.parametrize("M", [1, 20, 64, 100, 300, 777, 2048, 5000])
@pytest.mark.parametrize("N,K", [(128, 128), (2560, 9728), (9728, 2560), (8192, 8192), (512, 16384)])
def test_splits_fit_one_round_and_their_workspace(lib, M, N, K):
    for grad in (0, 1):
        bm, sk = fp8(lib, grad, 0, M, N, K)
        out, steps = (K, N // 128) if grad else (N, K // 128)
        assert bm in HEIGHTS and 1 <= sk <= 16
        if sk > 1:
            assert -(-M // bm) * -(-out // 256) * sk <= 256 and -(-steps // sk) >= 4
        size = (w4.w4a16_fp8_gemm_grad_workspace_bytes if grad else w4.w4a16_fp8_gemm_workspace_bytes)(M, N, K)
        assert size == (0 if sk == 1 else -(-sk * M * out * 4 // 256) * 256)
    for gs in (128, 32):
        bm, sk = w4_grad(lib, 0, M, N, K, gs)
        assert bm in HEIGHTS and 1 <= sk <= 16
        if sk > 1:
            assert -(-M // bm) * -(-K // 256) * sk <= 256 and -(-(N // 64) // sk) >= 8
        up = lambda v: -(-v // 256) * 256   # noqa: E731
        parts = up(2 * M * N) + up(4 * M) + up(2 * N * (K // gs)) + up(2 * (N // 128) * (K // gs))
        assert w4.w4a16_gemm_grad_workspace_bytes(1, M, N, K, gs) == parts + (up(4 * sk * M * K) if sk > 1 else 0)


@pytest.mark.parametrize("G,M,N,K", [(8, 4096, 2048, 4096), (64, 3000, 512, 1024), (2, 1, 256, 256), (300, 700, 128, 128)])
def test_by_expert_only_the_4_bit_gradient_splits(lib, G, M, N, K):
    assert fp8(lib, 0, G, M, N, K)[1] == 1 and fp8(lib, 1, G, M, N, K)[1] == 1
    bm, sk = w4_grad(lib, G, M, N, K)
    most = (M + (bm - 1) * min(G, M)) // bm * -(-K // 256)
    assert sk == 1 or most * sk <= 256
