"""Products by expert of so many few-row tiles that their grid takes its second dimension
(more than 2^20 of them), every result compared bit for bit."""
import ctypes
import os

import pytest
import torch

import fp8_ref as ref
from gpu_util import binding, say
from test_gpu_fp8 import DEV, exact_codes, gen
from test_gpu_fp8_large import load_choice

pytestmark = pytest.mark.gpu

# rows, N, K, E: 64 experts with a tile of 16 rows or less each, 32 GiB of weights
M, N, K, E = 100, 1 << 19, 1024, 64


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert binding().mxgemm_device_supported()
    yield


def tiles(bm, bn):
    """Tiles that the launch provides for."""
    return min(-(-M // bm) + E - 1, M) * -(-N // bn)


def plan(g):
    expert = torch.randint(0, E, (M,), generator=g, device=DEV).sort()[0]
    return expert, torch.searchsorted(expert, torch.arange(E + 1, device=DEV)).int()


@pytest.mark.parametrize("gather", [False, True])
def test_fp8(gather):
    say("fp8 tiles in two dimensions", gather)
    assert load_choice()(M, N, K, E) == "16x32" and tiles(16, 32) > 1 << 20
    g = gen(21)
    a, a_s = exact_codes(g, M, K)
    b = torch.randint(0, 3, (E, N, K), generator=g, device=DEV, dtype=torch.uint8).mul_(8).add_(0x30)   # 1/2, 1, 2
    b_s = torch.exp2(torch.randint(-1, 2, (E, N // 128, K // 128), generator=g, device=DEV).float())
    expert, off = plan(g)
    index = torch.randperm(M, generator=g, device=DEV).int() if gather else None
    got = binding().fp8gemm_run_grouped(a, a_s, b, b_s, off, index=index)
    rows = torch.arange(M, device=DEV) if index is None else index.long()
    x = ref.dequantize(a, a_s)[rows]
    for e in expert.unique().tolist():
        at = expert == e
        for n in range(0, N, N // 4):
            to = slice(n, n + N // 4)
            want = x[at] @ ref.dequantize(b[e, to], b_s[e, n // 128:(n + N // 4) // 128], 128).t()
            assert torch.equal(got[at, to].double(), want), (e, n)


@pytest.mark.parametrize("gather", [False, True])
def test_int8(gather):
    say("int8 tiles in two dimensions", gather)
    lib = ctypes.CDLL(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libint8_choice.so"))
    lib.int8_choice.argtypes = [ctypes.c_int64] * 4
    v = lib.int8_choice(M, N, K, E)
    assert v < 2 and tiles(16, (16, 32)[v]) > 1 << 20
    g = gen(22)
    a = torch.randint(-8, 9, (M, K), generator=g, device=DEV).to(torch.int8)
    b = torch.randint(0, 17, (E, N, K), generator=g, device=DEV, dtype=torch.uint8).view(torch.int8).sub_(8)
    a_s = torch.exp2(torch.randint(-2, 3, (M,), generator=g, device=DEV).float())
    b_s = torch.exp2(torch.randint(-2, 3, (E, N), generator=g, device=DEV).float())
    expert, off = plan(g)
    index = torch.randperm(M, generator=g, device=DEV).int() if gather else None
    got = binding().int8gemm_run_grouped(a, a_s, b, b_s, off, index=index)
    rows = torch.arange(M, device=DEV) if index is None else index.long()
    x = (a.double() * a_s.double()[:, None])[rows]
    for e in expert.unique().tolist():
        at = expert == e
        for n in range(0, N, N // 4):
            to = slice(n, n + N // 4)
            want = x[at] @ (b[e, to].double() * b_s[e, to].double()[:, None]).t()
            assert torch.equal(got[at, to].double(), want), (e, n)
