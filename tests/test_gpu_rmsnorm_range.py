"""The norm of rows whose 1 / sqrt(mean square) lies at the ends of fp32's range or
beyond it, against the 64-bit form."""
import pytest
import torch

import fp8_ref as ref
from gpu_util import binding, say
from test_gpu_fp8 import DEV, TYPES, U, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert binding().mxgemm_device_supported()
    yield


@pytest.mark.parametrize("K", [16, 512, 4096, 14336, 32768, 131072])
@pytest.mark.parametrize("exponent", [-140, -128, -110, 90, 110, 126])
@pytest.mark.parametrize("kind", [0, 1])
def test_rows_of_any_size(K, exponent, kind):
    """Rows of 1 .. 1.9 times 2^exponent, no eps: rstd is the nearest fp32 value (an infinity
    beyond the largest), y that of the real product: it is formed from rstd with its rest, up
    to 2^-40 of half a step.  (bf16 has no 2^-140: those are rows of zeros, whose y is NaN.)"""
    say("norm of rows of any size", K, exponent, kind)
    bn = binding()
    g = gen(K + exponent)
    x = 1.0 + 0.9 * torch.rand(3, K, generator=g, device=DEV, dtype=torch.float64)
    x = x * (2.0 * torch.randint(0, 2, (3, K), generator=g, device=DEV) - 1.0) * 2.0 ** exponent
    x = x.to(TYPES[kind])
    w = 1 + 0.2 * randn(g, K)
    _, _, _, y, rstd = bn.rmsnorm_quantize(x, w, quant=0, eps=0.0)
    real, want = ref.norm(x, w, 0.0)
    assert torch.equal(rstd, real.float())
    t = torch.finfo(TYPES[kind])
    # y in fp32, then in the rows' type
    off = (y.double() - want).abs()
    step = U if kind == 0 else U + t.eps / 2
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert bool(((off <= want.abs() * (step * (1 + 2.0 ** -7)) + 2.0 ** -133) | torch.isnan(want)).all())


@pytest.mark.parametrize("quant", [1, 2, 3, 4])
def test_codes_of_tiny_rows(quant):
    """The codes of rows of 2^-135 are those of the same rows times 2^135, no eps."""
    say("norm codes of tiny rows", quant)
    bn = binding()
    g = gen(quant)
    x = torch.randint(-2000, 2001, (5, 544), generator=g, device=DEV).float() * 2.0 ** -8
    w = randn(g, 544)
    q, s, _, _, rstd = bn.rmsnorm_quantize(x * 2.0 ** -135, w, quant=quant, eps=0.0)
    want = bn.rmsnorm_quantize(x, w, quant=quant, eps=0.0)
    assert bool(torch.isinf(rstd).all())
    assert torch.equal(q, want[0]) and torch.equal(s, want[1])
