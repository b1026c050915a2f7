"""Gradients of the weights from codes whose scales are no powers of two: applied in fp32
(any_scale), and how far the rounding to bfloat16 without it goes; against the gradient
of the dequantized activations in 64 bits."""
import pytest
import torch

import fp8_ref as ref
from gpu_util import binding, poison_lds, say
from test_gpu_fp8 import DEV, TYPES, U, exact_codes, gen, randn
from test_gpu_fp8_grad import COUNTS, EXPERTS, SIZES, exact_d, expert_grad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert binding().mxgemm_device_supported()
    yield


def real_grad(d, a, a_s):
    """dW and sum |terms|, nothing rounded."""
    x = ref.dequantize(a, a_s)
    return d.double().t() @ x, d.double().abs().t() @ x.abs()


def sum_error(M, terms):
    """Products of bf16 values and codes are exact in fp32; their sum of M rows of `terms` is
    off by at most terms M 2^-24 of the sum of their sizes, the further terms of a row at
    most 2^-8 of the first."""
    return (M * terms + 9) * U * (1 + 2.0 ** -7)


@pytest.mark.parametrize("M,N,K", [(1, 40, 128), (100, 300, 272), (700, 520, 1040), (3000, 136, 256), (2500, 1100, 640), (513, 129, 48)])
@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("out", [0, 1, 2])
def test_any_scale(M, N, K, kind, out):
    """dC times the scale is rounded to fp32 once (2^-24, in the 9 above); three bf16 values
    hold it."""
    say("weight grad any scale", M, N, K, kind, out)
    g = gen(M + N)
    a, a_s = ref.quantize(randn(g, M, K) * torch.exp2(torch.randint(-8, 8, (M, 1), generator=g, device=DEV).float()))
    d = (randn(g, M, N) * 0.1).to(TYPES[kind])
    y, mass = real_grad(d, a, a_s)
    got = binding().fp8gemm_weight_grad(d, a, a_s, out_type=out, any_scale=True).double()
    err = mass * sum_error(M, 3)
    tol = err + torch.finfo(TYPES[out]).eps / 2 * (y.abs() + err) + (2.0 ** -25 if out == 2 else 2.0 ** -120)
    off = (got - y).abs()
    say("  error / bound %.3g" % (off / tol).max().item())
    assert bool((off <= tol).all())
    if out == 0:
        rms = ((got - y).square().mean() / y.square().mean()).sqrt().item()
        say("  rms %.3g" % rms)
        assert rms <= 2.0 ** -20


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_rounded_activations(kind):
    """Without any_scale x is rounded to bf16: at most 2^-8 of each term (half a step)."""
    say("weight grad rounded activations", kind)
    g = gen(kind)
    M, N, K = 2047, 300, 640
    a, a_s = ref.quantize(randn(g, M, K))
    d = randn(g, M, N).to(TYPES[kind])
    y, mass = real_grad(d, a, a_s)
    got = binding().fp8gemm_weight_grad(d, a, a_s).double()
    off = (got - y).abs()
    assert bool((off <= mass * (2.0 ** -8 + sum_error(M, (3, 1, 2)[kind]) * (1 + 2.0 ** -8))).all())
    say("  rms %.3g" % (off.square().mean() / y.square().mean()).sqrt().item())


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_exact(M, N, K, kind):
    """Scales 3/2, 3 and 3/4: sums of multiples of 3/32 below 2^21, equal in any order."""
    say("weight grad any scale exact", M, N, K, kind)
    g = gen(M + N + K)
    a, a_s = exact_codes(g, M, K)
    a_s = a_s * 1.5
    d = exact_d(g, M, N, kind)
    poison_lds()
    got = binding().fp8gemm_weight_grad(d, a, a_s, any_scale=True)
    assert torch.equal(got.double(), real_grad(d, a, a_s)[0])


@pytest.mark.parametrize("E,tokens,k,N,K", EXPERTS)
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_experts(E, tokens, k, N, K, kind):
    say("weight grad any scale experts", E, tokens, k, N, K, kind)
    g = gen(E + tokens + N)
    bn = binding()
    a, a_s = exact_codes(g, tokens, K)
    a_s = a_s * 1.5
    ids = torch.rand(tokens, E, generator=g, device=DEV).topk(k, 1).indices.int()
    offsets, order, _ = bn.expert_plan(ids, E)
    d = exact_d(g, tokens * k, N, kind)
    out = torch.full((E, N, K), float("nan"), device=DEV)
    bn.fp8gemm_weight_grad_grouped(d, a, a_s, offsets, index=order, index_div=k, out=out, any_scale=True)
    want = expert_grad(d, a, a_s, offsets, order, k, E)
    assert torch.equal(out.double(), want)
    at = (order // k).long()
    got = bn.fp8gemm_weight_grad_grouped(d, a[at], a_s[at], offsets, out_type=1, any_scale=True)
    assert torch.equal(got, want.float().bfloat16())


@pytest.mark.parametrize("N,K", [(1010, 1264), (300, 400)])
@pytest.mark.parametrize("kind,out", [(1, 0), (0, 1), (2, 2)])
@pytest.mark.parametrize("gather", [True, False])
def test_experts_of_every_size(N, K, kind, out, gather):
    say("weight grad any scale, experts of every size", N, K, kind, out, gather)
    g = gen(N + K)
    E, rows, T = len(COUNTS), sum(COUNTS), 900
    offsets = torch.tensor([0] + COUNTS, device=DEV).cumsum(0).int()
    a, a_s = exact_codes(g, T if gather else rows, K)
    a_s = a_s * 1.5
    index = torch.randint(0, 3 * T, (rows,), generator=g, device=DEV).int() if gather else None
    d = exact_d(g, rows, N, kind)
    want = expert_grad(d, a, a_s, offsets, index, 3, E)
    poison_lds()
    got = torch.full((E, N, K), float("nan"), dtype=TYPES[out], device=DEV)
    binding().fp8gemm_weight_grad_grouped(d, a, a_s, offsets, index=index, index_div=3, out=got, out_type=out, any_scale=True)
    assert torch.equal(got, want.float().to(TYPES[out]))


def test_offsets_and_index():
    """Rows behind the experts are not read into a sum, indices outside A give NaN."""
    say("weight grad any scale, offsets and index")
    E, N, K, T, rows = 5, 140, 272, 40, 300
    g = gen(rows)
    a, a_s = exact_codes(g, T, K)
    a_s = a_s * 1.5
    d = exact_d(g, rows, N, 1)
    index = torch.randint(0, 2 * T, (rows,), generator=g, device=DEV).int()
    index[11], index[290], index[291] = -1, 2 * T, 2 ** 31 - 1
    d[290:] = float("nan")
    for offsets in ([2, 2, 7, 9, 15, 290], [0] * 6, [0, 0, 0, 290, 290, 290], [-5, 3, 1, 12, 10, 280], [290] * 6,
                    [-2 ** 31, -1, 0, 1, 2, 3]):
        off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        got = binding().fp8gemm_weight_grad_grouped(d, a, a_s, off, index=index, index_div=2, any_scale=True)
        want = expert_grad(d, a, a_s, off, index, 2, E)
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan) and torch.equal(nan.all((1, 2)), nan.any((1, 2)))
        assert torch.equal(got[~nan].double(), want[~nan])


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_specials(kind):
    """Infinities and NaNs of gradient, scales and codes are where the formula has them,
    scales of 0 too; a value beyond bf16's range stays finite."""
    say("weight grad any scale specials", kind)
    g = gen(2)
    a, a_s = exact_codes(g, 90, 160)
    a[a == 0] = 0x38
    a_s = a_s * 1.5
    d = exact_d(g, 90, 60, kind)
    d[d == 0] = 1.0
    a_s[5, 1] = float("nan")
    a_s[9, 0] = float("inf")
    a_s[11, 1] = 0.0
    a_s[12] = 0.0
    a[7, 3] = 0x7F
    a[13, 9] = 0x80                # -0 against an infinite gradient below
    d[13, 8] = float("inf")
    d[20, 2] = float("inf")
    d[21, 4] = float("nan")
    if kind == 0:
        d[22, 6] = torch.finfo(torch.float32).max
        a[22], a_s[22] = 0x30, 0.75
    x = ref.dequantize(a, a_s)
    y = d.double().t() @ x
    got = binding().fp8gemm_weight_grad(d, a, a_s, any_scale=True).double()
    assert torch.equal(torch.isnan(got), torch.isnan(y))
    assert torch.equal(torch.isinf(got), torch.isinf(y)) and torch.equal(got[torch.isinf(y)], y[torch.isinf(y)])
    ok = torch.isfinite(y)
    ok[6] = False
    assert torch.equal(got[ok], y[ok])
    if kind == 0:
        fine = torch.isfinite(y[6])
        assert bool(((got[6] - y[6]).abs()[fine] <= 4 * U * y[6].abs()[fine]).all())


def test_replay_and_streams():
    say("weight grad any scale, replay and streams")
    bn = binding()
    g = gen(3)
    a, a_s = ref.quantize(randn(g, 5000, 256))
    d = randn(g, 5000, 200).bfloat16()
    off = torch.tensor([0, 100, 100, 2000, 5000], dtype=torch.int32, device=DEV)

    def work(stream=None):
        return (bn.fp8gemm_weight_grad(d, a, a_s, any_scale=True, stream=stream),
                bn.fp8gemm_weight_grad_grouped(d, a, a_s, off, any_scale=True, stream=stream))

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for _ in range(4):
        d.copy_(randn(g, 5000, 200))
        graph.replay()
        got = [t.clone() for t in held]
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    many = [work(st) for st in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for m in many for p, q in zip(m, want))
