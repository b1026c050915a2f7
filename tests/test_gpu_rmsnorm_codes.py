"""The norm's codes are, bit for bit, those that the quantizers give its fp32 y."""
import pytest
import torch

import fp8_ref as ref
from gpu_util import binding, say
from test_gpu_fp8 import DEV, U, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert binding().mxgemm_device_supported()
    yield


SIZES = [(1, 16), (9, 48), (700, 144), (64, 256), (33, 512), (300, 544), (40, 1024), (17, 2064), (500, 4096), (20, 8192),
         (11, 14336), (5, 16416), (3, 32768), (2, 131072), (1, 1048576)]


@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("quant", [1, 2, 3, 4])
@pytest.mark.parametrize("residual", [False, True])
def test_codes_are_those_of_y(rows, K, quant, residual):
    """fp32 rows, so that y is seen as it is.  y itself: the sum in 64 bits has 2^-29 of
    half a step at K = 2^20, the product with the rest of rstd 2^-47."""
    say("norm codes of y", rows, K, quant, residual)
    bn = binding()
    if quant == bn.QUANT_MXFP8 and K % 32:      # blocks of 32
        with pytest.raises(bn.MXGemmError):
            bn.rmsnorm_quantize(torch.ones(rows, K, device=DEV), torch.ones(K, device=DEV), quant=quant)
        return
    g = gen(rows + K + quant)
    x = randn(g, rows, K) * torch.exp2(torch.randint(-6, 4, (rows, 1), generator=g, device=DEV).float())
    x[rows // 2, K // 2:] = 0.0           # blocks of zeros
    r = randn(g, rows, K) * (x != 0) if residual else None
    w = 1 + 0.2 * randn(g, K)
    q, s, h, y, _ = bn.rmsnorm_quantize(x, w, residual=r, quant=quant, with_y=True)
    want = ref.norm(h, w, 1e-6)[1]
    assert bool(((y.double() - want).abs() <= want.abs() * (U * (1 + 2.0 ** -16)) + 2.0 ** -149).all())
    if quant == bn.QUANT_INT8:
        wq, ws = bn.int8gemm_quantize(y)
    elif quant == bn.QUANT_MXFP8:
        wq, ws = bn.mxgemm_quantize(y)
    else:
        wq, ws = ref.quantize(y, 1, quant == bn.QUANT_FP8_POW2)
    assert torch.equal(q, wq) and torch.equal(s, ws)
