"""What the 8-bit operators answer to sizes near the end of 32 bits, where counts of tiles and squares rounded up would
wrap around: refused before anything is launched (addresses here are fake).  And which products are cut into K slices."""
import ctypes

import pytest

import compressed_sparse_attention_09_b200 as csa

UNSUPPORTED, WORKSPACE = 2, 7
P = ctypes.c_void_p(1 << 20)
TOP = 2 ** 31 - 1
ROWS, WIDTH = 1 << 30, 1 << 28


def gemm(M, N, K, ws_bytes=1 << 40):
    n0 = csa.csa_launch_count()
    rc = csa.lib().csa_gemm_f8(csa.CSA_BF16, P, 1 << 32, P, 1 << 28, P, 1 << 32, P, 1 << 28, M, N, K, P, 1 << 32, P, ws_bytes, None)
    assert csa.csa_launch_count() == n0
    return rc


@pytest.mark.parametrize("M,N,K", [(TOP, 128, 128), (ROWS + 1, 1, 16), (1, TOP, 4096), (64, TOP - 127, 1024), (1, ROWS + 1, 4096),
                                   (1, 1, TOP), (1, 128, WIDTH + 16), (TOP, TOP, TOP)])
def test_product_refuses_sizes_that_wrap_around(M, N, K):
    assert gemm(M, N, K) == UNSUPPORTED
    assert csa.csa_gemm_f8_workspace_bytes(M, N, K) == 0


def test_product_takes_the_largest_sizes():
    """(as far as the check of its workspace, which comes after that of the sizes)"""
    need = csa.csa_gemm_f8_workspace_bytes(64, 2048, WIDTH)
    assert need == 8 * 2048 * 64 * 4
    assert gemm(64, 2048, WIDTH, need - 1) == WORKSPACE
    assert csa.csa_gemm_f8_workspace_bytes(1, ROWS, 4096) == 0


@pytest.mark.parametrize("N", [TOP, TOP - 127, TOP - 65535 * 128 + 1, ROWS + 1])
def test_weight_quantiser_refuses_rows_that_wrap_around(N):
    n0 = csa.csa_launch_count()
    assert csa.lib().csa_quantize_weight_f8(csa.CSA_BF16, P, 256, N, 256, P, 256, P, 2, None) == UNSUPPORTED
    assert csa.csa_launch_count() == n0


@pytest.mark.parametrize("M,N,K,slices", [(64, 4160, 4096, 4), (1, 4160, 4096, 4), (64, 2304, 4096, 8), (64, 300, 8192, 8),
                                          (64, 9472, 1024, 1), (64, 9472, 8192, 1), (64, 4160, 2048, 1), (5, 1000, 2048, 1),
                                          (64, 4160, 4224, 1), (65, 4160, 4096, 1)])
def test_products_are_sliced_where_that_pays(M, N, K, slices):
    """Deep products in four or eight slices; shallow ones, and wide ones that would get two, are faster whole."""
    need = slices * -(-N // 128) * 128 * M * 4 if slices > 1 else 0
    assert csa.csa_gemm_f8_workspace_bytes(M, N, K) == -(-need // 256) * 256
