"""Results of the largest tile for rows that start anywhere in a line: both ways of storing
16-bit results, whole and ragged tiles, bit for bit."""
import pytest
import torch

import fp8_ref as ref
from gpu_util import binding, poison_lds, say
from test_gpu_fp8 import DEV, TYPES, exact_codes, gen
from test_gpu_fp8_large import load_choice

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert binding().mxgemm_device_supported()
    yield


@pytest.mark.parametrize("columns", [0, 1, 7, 8, 16, 31, 32, 33, 40, 48, 63])
@pytest.mark.parametrize("M", [5120, 5127])
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_rows_from_any_place_of_a_line(columns, M, kind):
    say("fp8 rows from any place of a line", columns, M, kind)
    N, K = 5120 + columns, 272
    assert load_choice()(M, N, K) == "256x256"
    g = gen(columns)
    a, a_s = exact_codes(g, M, K)
    b, b_s = exact_codes(g, N, K, 128)
    out = torch.full((M + 1, N), -7.0, dtype=TYPES[kind], device=DEV)
    poison_lds()
    binding().fp8gemm_run(a, a_s, b, b_s, out=out[:M], out_type=kind)
    want = (ref.dequantize(a, a_s) @ ref.dequantize(b, b_s, 128).t()).to(TYPES[kind])
    assert torch.equal(out[:M], want)
    assert bool((out[M] == -7.0).all())
