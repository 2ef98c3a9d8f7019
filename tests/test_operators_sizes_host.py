"""Workspace of the adapter projection, to the byte (CPU only)."""
import os

import pytest

import bf16_activation_quantized_amd as w4

CASES = [(1, 64, 512, 128, 16, 0), (1, 64, 512, 128, 8, 2), (1, 1, 6656, 128, 40, 16), (1, 17408, 5120, 128, 16, 0),
         (5, 300, 1024, 128, 24, 0), (16, 512, 1024, 128, 16, 2), (16, 512, 1024, 128, 16, 16), (20, 96, 512, 128, 8, 0),
         (40, 512, 1024, 128, 8, 0), (45, 96, 512, 128, 128, 4), (64, 8192, 8192, 128, 16, 0), (100, 8448, 256, 128, 128, 0),
         (100, 8448, 256, 128, 128, 8), (333, 2560, 9728, 32, 24, 0), (64, 512, 256, 32, 16, 4), (1322, 19456, 2560, 128, 64, 0)]


@pytest.fixture(autouse=True)
def _built():
    if not os.path.exists(w4.LIB_PATH):
        pytest.skip("libw4a16.so not built")


@pytest.mark.parametrize("M,N,K,group,R,sk", CASES)
@pytest.mark.parametrize("L", [1, 700])
def test_workspace_is_h_and_the_projections_own(M, N, K, group, R, sk, L):
    """Both parts of h (2 bytes each), rounded up to 256, then what w4a16_gemm
    uses at the same sizes: partials and row sums."""
    h = (M * R * 4 + 255) // 256 * 256
    assert w4.w4a16_gemm_lora_workspace_bytes(M, N, K, L, R, sk, group) == \
        h + w4.w4a16_gemm_workspace_bytes(M, N, K, sk, group_size=group)


@pytest.mark.parametrize("N,K,sk", [(64, 1280, 0), (64, 1024, 16), (300, 9216, 0), (4096, 640, 2), (77, 33024, 0)])
def test_one_row_of_a_length_without_gemv_takes_the_small_batch_plan(N, K, sk):
    """The only other plan: slices for which the GEMV takes no adapters."""
    assert w4.w4a16_gemm_auto_config(1, N, K)[0] == w4.PATH_GEMV
    assert w4.w4a16_gemm_lora_workspace_bytes(1, N, K, 3, 16, sk) == \
        256 + w4.w4a16_gemm_workspace_bytes(1, N, K, sk, path=w4.PATH_SKINNY)
