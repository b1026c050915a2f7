"""The flag for scales of any kind at the weight gradients' C entries: it changes no
refusal (all return from argument validation), and its kernels keep their LDS order."""
import os
import re

import pytest

import asm_hazards as H
from test_abi_fp8 import A, EALIGN, EINVAL
from test_kernel_asm_fp8 import CSRC, pytestmark, unordered  # noqa: F401  (the mark: hipcc is there)

FLAG = 16


@pytest.fixture(scope="module")
def lib():
    from block_scaled_precision_mxgemm_amd import mxgemm

    assert mxgemm.GRAD_ANY_SCALE == FLAG
    return mxgemm.raw_library()


def test_header():
    header = open(os.path.join(os.path.dirname(CSRC), os.pardir, "include", "mxgemm.h")).read()
    assert "#define MXG_GRAD_ANY_SCALE %d" % FLAG in header


@pytest.mark.parametrize("kind,dC,want", [(FLAG + 3, A, EINVAL), (FLAG + 15, A, EINVAL), (2 * FLAG, A, EINVAL), (3 * FLAG, A, EINVAL),
                                          (FLAG - 32, A, EINVAL), (-1, A, EINVAL), (FLAG, None, EINVAL), (FLAG, A + 8, EALIGN),
                                          (FLAG + 1, A + 2, EALIGN), (FLAG + 2, A + 4, EALIGN)])
def test_refusals(lib, kind, dC, want):
    assert lib.fp8gemm_weight_grad(dC, kind, 8, 4, A, A, 64, A, 0, A, None) == want
    assert lib.fp8gemm_weight_grad_grouped(dC, kind, 8, 4, A, A, 8, 64, 2, A, None, 1, A, 0, A, None) == want


@pytest.mark.parametrize("M,N,K,E", [(16384, 16, 64, 1), (16384, 1024, 1024, 1), (8192, 4096, 4096, 1), (5000, 64, 128, 4)])
def test_workspace_holds_its_parts(lib, M, N, K, E):
    """As many parts of the rows as three terms take, or none where those take large tiles."""
    import ctypes

    choice = ctypes.CDLL(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libfp8_choice.so"))
    choice.fp8_grad_choice.argtypes = [ctypes.c_int64] * 4 + [ctypes.c_int]
    splits = choice.fp8_grad_choice(M, N, K, E, 3)
    if splits > 1:
        assert lib.fp8gemm_weight_grad_workspace(M, N, K, E) >= splits * E * N * K * 4


def test_its_kernels_keep_their_lds_order():
    from block_scaled_precision_mxgemm_amd import build as B

    text = H.compile_to_asm(os.path.join(CSRC, "fp8_weight_grad.hip"), B.FLAGS, B.HIPCC)
    seen = 0
    for m in re.finditer(r"^(_ZN\S*fp8_weight_grad_any_kernel\S*):", text, re.M):
        body = text[m.end():text.index(".Lfunc_end", m.end())]
        runs, bad = unordered(body)
        assert bad == 0 and runs >= 4, (m.group(1), runs, bad)
        assert "scratch_" not in body
        seen += 1
    assert seen == 6
