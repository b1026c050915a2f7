"""Which tile the E4M3 products with a scale per block of 128 take (host code alone)."""
import pytest

import test_gpu_fp8_large as large


@pytest.mark.parametrize("rows,N,K,E", [(8, 4096, 4096, 32), (16, 4096, 4096, 32), (8, 2048, 4096, 64), (32, 2048, 4096, 64),
                                        (4, 14336, 4096, 8), (64, 2048, 4096, 64), (2, 4096, 2048, 8)])
def test_few_rows_over_many_experts(rows, N, K, E):
    """Where memory bounds the product, tiles of 16 x 16 (more of them than of 16 x 32, at the
    same time each) are the slower ones: 8 rows over 32 experts of 4096 x 4096 38 and 27 us."""
    assert large.load_choice()(rows, N, K, E) == "16x32"


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 4096, 4096), (16, 2048, 8192), (16, 1024, 2048), (9, 4000, 4000)])
def test_few_rows_and_columns(M, N, K):
    """Where 16 x 32 leaves CUs without a tile, 16 x 16 is the faster one."""
    assert large.load_choice()(M, N, K) == "16x16"


def test_gradient_cases_take_every_form_in_three_terms():
    """dY in fp32, which is three terms: large tiles, small ones, and rows in parts."""
    import ctypes
    import os

    import test_gpu_fp8_grad as grad

    lib = ctypes.CDLL(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libfp8_choice.so"))
    lib.fp8_grad_choice.argtypes = [ctypes.c_int64] * 4 + [ctypes.c_int]
    taken = {lib.fp8_grad_choice(M, N, K, 1, 3) for M, N, K in grad.SIZES}
    assert {0, 1} <= taken and len(taken) >= 4
    rows = len(grad.COUNTS)
    assert lib.fp8_grad_choice(sum(grad.COUNTS), 2020, 992, rows, 3) == 0
    assert lib.fp8_grad_choice(sum(grad.COUNTS), 300, 400, rows, 3) >= 1
