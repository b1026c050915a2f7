"""Gradients of the weights of the E4M3 products from the activations' codes,
dense and by expert, and a step of a layer that uses them, against the 64-bit forms."""
import pytest
import torch

import fp8_ref as ref
from gpu_util import binding, poison_lds, say
from test_gpu_fp8 import DEV, TYPES, U, exact_codes, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert binding().mxgemm_device_supported()
    yield


def exact_d(g, rows, N, kind):
    """Multiples of 1/4 up to 2."""
    return (torch.randint(-8, 9, (rows, N), generator=g, device=DEV).float() / 4).to(TYPES[kind])


SIZES = [(1, 1, 16), (1, 130, 128), (2, 16, 144), (31, 7, 272), (32, 128, 256), (33, 129, 1040), (64, 100, 96), (65, 257, 384),
         (127, 300, 640), (200, 64, 2064), (513, 384, 512), (1000, 1030, 400), (2047, 515, 304), (4096, 256, 256), (9000, 24, 48),
         (300, 2050, 1168), (8200, 136, 128), (700, 4096, 2064), (130, 4100, 4112), (5000, 1000, 1040)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_exact(M, N, K, kind):
    """Sums of multiples of 1/16 below 2^20: equal, in any order, from every kernel."""
    say("weight grad exact", M, N, K, kind)
    g = gen(M + N + K)
    a, a_s = exact_codes(g, M, K)
    d = exact_d(g, M, N, kind)
    got = binding().fp8gemm_weight_grad(d, a, a_s)
    assert torch.equal(got.double(), d.double().t() @ ref.dequantize(a, a_s))


@pytest.mark.parametrize("M,N,K", [(1, 40, 128), (100, 300, 272), (700, 520, 1040), (3000, 136, 256), (2500, 1100, 640)])
@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("out", [0, 1, 2])
@pytest.mark.parametrize("pow2", [True, False])
def test_normal(M, N, K, kind, out, pow2):
    """Products of bf16 values are exact in fp32; their sum of M terms is off by at
    most M 2^-24 of the sum of their sizes.  fp16 and fp32 go in as two and three bf16
    values, exactly: as many more terms, the further ones at most 2^-8 of the first."""
    say("weight grad", M, N, K, kind, out, pow2)
    g = gen(M + N)
    a, a_s = ref.quantize(randn(g, M, K) * torch.exp2(torch.randint(-8, 8, (M, 1), generator=g, device=DEV).float()), 1, pow2)
    d = (randn(g, M, N) * 0.1).to(TYPES[kind])
    x = (ref.decode(a).float() * ref.expand(a_s, M, K, 1)).to(torch.bfloat16)
    if pow2:
        assert torch.equal(x.double(), ref.dequantize(a, a_s))
    y, mass = ref.bf16_grad(d, x)
    got = binding().fp8gemm_weight_grad(d, a, a_s, out_type=out).double()
    err = mass * ((M * (3, 1, 2)[kind] + 8) * U * (1 + 2.0 ** -7))
    tol = err + torch.finfo(TYPES[out]).eps / 2 * (y.abs() + err) + (2.0 ** -25 if out == 2 else 2.0 ** -140)
    off = (got - y).abs()
    say("  error / bound %.3g" % (off / tol).max().item())
    assert bool((off <= tol).all())
    if out == 0:
        rms = ((got - y).square().mean() / y.square().mean()).sqrt().item()
        say("  rms %.3g" % rms)
        assert rms <= 2.0 ** -20


def test_specials():
    """Infinities and NaNs of the gradient and of the codes stay in their row and
    column; a finite value beyond bf16's range stays finite."""
    say("weight grad specials")
    g = gen(2)
    for kind in (0, 1, 2):
        a, a_s = exact_codes(g, 90, 160)
        a[a == 0] = 0x38                # ones: no infinity times zero
        a_s[5, 1] = float("nan")
        a[7, 3] = 0x7F
        d = exact_d(g, 90, 60, kind)
        d[d == 0] = 1.0
        d[20, 2] = float("inf")
        d[21, 4] = float("nan")
        if kind == 0:
            d[22, 6] = torch.finfo(torch.float32).max
            a[22], a_s[22] = 0x30, 1.0   # 1/2
        y = d.double().t() @ ref.dequantize(a, a_s)
        got = binding().fp8gemm_weight_grad(d, a, a_s).double()
        assert torch.equal(torch.isnan(got), torch.isnan(y))
        assert torch.equal(torch.isinf(got), torch.isinf(y))
        ok = torch.isfinite(y)
        ok[6] = False
        assert torch.equal(got[ok], y[ok])
        if kind == 0:
            fine = torch.isfinite(y[6])
            assert bool(((got[6] - y[6]).abs()[fine] <= 2.0 ** -15 * y[6].abs()[fine]).all())


def expert_grad(d, a, a_s, offsets, index, div, E):
    x = ref.dequantize(a, a_s)
    out = torch.zeros(E, d.shape[1], a.shape[1], dtype=torch.float64, device=d.device)
    for e, (lo, hi) in enumerate(ref.rows_of_experts(offsets.tolist(), d.shape[0])):
        at = torch.arange(lo, hi, device=d.device)
        if index is not None:
            at = torch.where(index[lo:hi] < 0, -1, torch.div(index[lo:hi], div, rounding_mode="floor")).long()
        good = (at >= 0) & (at < a.shape[0])
        out[e] = d[lo:hi].double().t() @ torch.where(good[:, None], x[at.clamp(0, a.shape[0] - 1)], float("nan"))
    return out


EXPERTS = [(1, 1, 1, 16, 128), (4, 3, 2, 130, 144), (8, 16, 2, 300, 400), (64, 16, 4, 128, 256), (7, 100, 3, 257, 272),
           (16, 300, 4, 520, 640), (2, 1000, 2, 256, 256), (130, 40, 8, 64, 128), (1024, 30, 2, 32, 48), (16, 1024, 4, 512, 512),
           (6, 700, 2, 2100, 1552), (3, 5000, 2, 136, 272), (16, 600, 3, 2048, 1024)]


@pytest.mark.parametrize("E,tokens,k,N,K", EXPERTS)
@pytest.mark.parametrize("kind", [0, 1])
def test_experts(E, tokens, k, N, K, kind):
    say("weight grad experts", E, tokens, k, N, K, kind)
    g = gen(E + tokens + N)
    bn = binding()
    a, a_s = exact_codes(g, tokens, K)
    ids = torch.rand(tokens, E, generator=g, device=DEV).topk(k, 1).indices.int()
    offsets, order, _ = bn.expert_plan(ids, E)
    d = exact_d(g, tokens * k, N, kind)
    out = torch.full((E, N, K), float("nan"), device=DEV)
    bn.fp8gemm_weight_grad_grouped(d, a, a_s, offsets, index=order, index_div=k, out=out)
    want = expert_grad(d, a, a_s, offsets, order, k, E)
    assert torch.equal(out.double(), want)
    at = (order // k).long()
    got = bn.fp8gemm_weight_grad_grouped(d, a[at], a_s[at], offsets, out_type=1)
    assert torch.equal(got, want.float().bfloat16())


def test_experts_offsets_and_index():
    say("weight grad offsets and index")
    E, N, K, T, rows = 5, 140, 272, 40, 300
    g = gen(rows)
    a, a_s = exact_codes(g, T, K)
    d = exact_d(g, rows, N, 1)
    index = torch.randint(0, 2 * T, (rows,), generator=g, device=DEV).int()
    index[11], index[290] = -1, 2 * T
    index[291] = 2 ** 31 - 1
    # rows behind the last expert are not read into a sum
    d[290:] = float("nan")
    for offsets in ([2, 2, 7, 9, 15, 290], [0] * 6, [0, 0, 0, 290, 290, 290], [-5, 3, 1, 12, 10, 280],
                    [290, 290, 290, 290, 290, 290], [-2 ** 31, -1, 0, 1, 2, 3]):
        off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        got = binding().fp8gemm_weight_grad_grouped(d, a, a_s, off, index=index, index_div=2)
        want = expert_grad(d, a, a_s, off, index, 2, E)
        nan = torch.isnan(want)   # the expert of row 11, whose index is none
        assert torch.equal(torch.isnan(got), nan) and torch.equal(nan.all((1, 2)), nan.any((1, 2)))
        assert torch.equal(got[~nan].double(), want[~nan])
    off = torch.tensor([4, 2 ** 31 - 1, 5, 6, 7, 8], dtype=torch.int32, device=DEV)
    got = binding().fp8gemm_weight_grad_grouped(d, a, a_s, off, index=index, index_div=2)
    assert torch.isnan(got[0]).all() and bool((got[1:] == 0).all())


def test_gradient_past_4_gib():
    """dC and A of more than 4 GiB."""
    say("weight grad rows past 4 GiB")
    g = gen(4)
    rows, N, K = 2 ** 20 + 300, 2304, 4224
    a = torch.zeros(rows, K, dtype=torch.uint8, device=DEV)
    a_s = torch.ones(rows, 33, device=DEV)
    d = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 5, 2 ** 19 + 77, 2 ** 20 + 1, rows - 1], device=DEV)
    q, s = exact_codes(g, 5, K)
    a[at], a_s[at] = q, s
    d[at] = exact_d(g, 5, N, 1)
    got = binding().fp8gemm_weight_grad(d, a, a_s)
    assert torch.equal(got.double(), d[at].double().t() @ ref.dequantize(q, s))


def test_graph_replay():
    say("graph replay weight grad")
    bn = binding()
    g = gen(3)
    a, a_s = exact_codes(g, 3000, 256)
    d = exact_d(g, 3000, 200, 1)
    off = torch.tensor([0, 100, 100, 2000, 3000], dtype=torch.int32, device=DEV)

    def work():
        return bn.fp8gemm_weight_grad(d, a, a_s), bn.fp8gemm_weight_grad_grouped(d, a, a_s, off)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for _ in range(4):
        d.copy_(exact_d(g, 3000, 200, 1))
        graph.replay()
        got = [t.clone() for t in held]
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert torch.equal(got[0].double(), d.double().t() @ ref.dequantize(a, a_s))


def test_side_streams():
    """Two calls at once have a workspace each."""
    say("weight grad streams")
    bn = binding()
    g = gen(7)
    sets = []
    for M, N, K in ((5000, 64, 128), (5000, 64, 128), (700, 300, 512)):
        a, a_s = exact_codes(g, M, K)
        sets.append((exact_d(g, M, N, 1), a, a_s))
    want = [bn.fp8gemm_weight_grad(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[bn.fp8gemm_weight_grad(*s, stream=st) for _ in range(5)] for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        assert all(torch.equal(w, m) for m in many)


def test_binding_refusals():
    bn = binding()
    g = gen(6)
    a, a_s = exact_codes(g, 8, 256)
    d = exact_d(g, 8, 30, 1)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    for call in (lambda: bn.fp8gemm_weight_grad(d[:7], a, a_s), lambda: bn.fp8gemm_weight_grad(d, a, a_s[:, :1]),
                 lambda: bn.fp8gemm_weight_grad(d, a, a_s, out_type=4), lambda: bn.fp8gemm_weight_grad(d.t(), a, a_s),
                 lambda: bn.fp8gemm_weight_grad_grouped(d, a[:4], a_s[:4], off),
                 lambda: bn.fp8gemm_weight_grad_grouped(d, a, a_s, off, index=off),
                 lambda: bn.fp8gemm_weight_grad_grouped(d, a, a_s, off[:1]),
                 lambda: bn.fp8gemm_weight_grad(d, a, a_s, out=torch.empty(30, 255, device=DEV))):
        with pytest.raises((ValueError, bn.MXGemmError)):
            call()
    with pytest.raises(TypeError):
        bn.fp8gemm_weight_grad(d.double(), a, a_s)


# ---- together ---------------------------------------------------------------------


def test_layer_step():
    """Norm, product, and the gradients of weights, activations and the norm, as a
    training step makes them, each against 64 bits on what the step before gave."""
    say("layer step")
    bn = binding()
    g = gen(12)
    T, K, N = 300, 512, 384
    x, r = randn(g, T, K).bfloat16(), randn(g, T, K).bfloat16()
    gain = (1 + 0.1 * randn(g, K)).bfloat16()
    weight = 0.05 * randn(g, N, K)
    w_q, w_s = bn.fp8gemm_quantize(weight, 128, pow2=True)
    wt_q, wt_s = bn.fp8gemm_quantize(weight.t().contiguous(), 128, pow2=True)
    assert torch.equal(wt_q, w_q.t()) and torch.equal(wt_s, w_s.t())

    q, s, h, _, rstd = bn.rmsnorm_quantize(x, gain, residual=r, quant=bn.QUANT_FP8_POW2)
    c = bn.fp8gemm_run(q, s, w_q, w_s, out_type=1)
    y = ref.dequantize(q, s) @ ref.dequantize(w_q, w_s, 128).t()
    assert ((c.double() - y).norm() / y.norm()).item() < 2.0 ** -9
    d_c = randn(g, T, N).bfloat16()
    d_w = bn.fp8gemm_weight_grad(d_c, q, s)
    want = d_c.double().t() @ ref.dequantize(q, s)
    assert ((d_w.double() - want).norm() / want.norm()).item() < 2.0 ** -20
    dq, ds = bn.fp8gemm_quantize(d_c, pow2=True)
    d_y = bn.fp8gemm_run(dq, ds, wt_q, wt_s, out_type=1)
    want = ref.dequantize(dq, ds) @ ref.dequantize(w_q, w_s, 128)
    assert ((d_y.double() - want).norm() / want.norm()).item() < 2.0 ** -9
    d_h = randn(g, T, K).bfloat16()
    d_x, d_gain = bn.rmsnorm_backward(d_y, h, gain, rstd, d_h=d_h)
    wx, wg = ref.norm_backward(d_y, h, gain, 1e-6, d_h)
    assert ((d_x.double() - wx).norm() / wx.norm()).item() < 2.0 ** -9
    assert ((d_gain.double() - wg).norm() / wg.norm()).item() < 2.0 ** -18


def test_expert_layer_step():
    """Forward and weight gradients of a layer of experts over one plan, captured
    into a graph and replayed."""
    say("expert layer step")
    bn = binding()
    g = gen(13)
    T, K, N, E, k = 200, 256, 384, 6, 2
    x = randn(g, T, K).bfloat16()
    gain = torch.ones(K, device=DEV)
    logits = randn(g, T, E)
    up_q, up_s = bn.fp8gemm_quantize(0.05 * randn(g, E, N, K), 128)
    down_q, down_s = bn.fp8gemm_quantize(0.05 * randn(g, E, K, N), 128)
    d_out = randn(g, T, K).bfloat16()
    d_y = torch.zeros(T * k, K, dtype=torch.bfloat16, device=DEV)

    def work():
        ids, w = bn.expert_route(logits, k)
        offsets, order, position = bn.expert_plan(ids, E)
        q, s, _, _, _ = bn.rmsnorm_quantize(x, gain, quant=bn.QUANT_FP8_POW2)
        h = bn.fp8gemm_run_grouped(q, s, up_q, up_s, offsets, index=order, index_div=k, act=1, out_type=1)
        hq, hs = bn.fp8gemm_quantize(h, pow2=True)
        y = bn.fp8gemm_run_grouped(hq, hs, down_q, down_s, offsets, out_type=1)
        out = bn.expert_combine(y, position, w)
        bn.expert_combine_backward(d_out, y, position, w, d_y=d_y)
        d_down = bn.fp8gemm_weight_grad_grouped(d_y, hq, hs, offsets)
        d_up = bn.fp8gemm_weight_grad_grouped(h, q, s, offsets, index=order, index_div=k)
        return ids, offsets, order, q, s, h, hq, hs, y, out, d_y.clone(), d_down, d_up

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for _ in range(3):
        logits.copy_(randn(g, T, E))
        graph.replay()
        got = [t.clone() for t in held]
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        ids, offsets, order, q, s, h, hq, hs, y, out, dy, d_down, d_up = got
        e = ids.reshape(-1)[order.long()].long()
        for i in range(E):
            at = e == i
            xe = ref.dequantize(q, s)[(order[at] // k).long()]
            u = ref.gelu(xe @ ref.dequantize(up_q[i], up_s[i], 128).t())
            assert ((h[at].double() - u).norm() / u.norm()).item() < 2.0 ** -8
            he = ref.dequantize(hq, hs)[at]
            want = he @ ref.dequantize(down_q[i], down_s[i], 128).t()
            assert ((y[at].double() - want).norm() / want.norm()).item() < 2.0 ** -8
            want = dy[at].double().t() @ he
            assert ((d_down[i].double() - want).norm() / want.norm()).item() < 2.0 ** -20
            want = h[at].double().t() @ xe
            assert ((d_up[i].double() - want).norm() / want.norm()).item() < 2.0 ** -20


# rows of experts: none, part of a slice of 64, odd and even numbers of slices
COUNTS = [0, 1, 64, 500, 65, 448, 449, 512, 0, 513, 576, 577, 640, 129, 1000, 128, 1024, 1, 700, 192, 193, 0]


@pytest.mark.parametrize("N,K", [(1010, 1264), (1024, 1280), (2020, 992), (300, 400)])
@pytest.mark.parametrize("kind,out", [(1, 0), (1, 1), (1, 2), (0, 0), (2, 1)])
@pytest.mark.parametrize("gather", [True, False])
def test_experts_of_every_size(N, K, kind, out, gather):
    say("weight grad experts of every size", N, K, kind, out, gather)
    g = gen(N + K)
    E, rows, T = len(COUNTS), sum(COUNTS), 900
    offsets = torch.tensor([0] + COUNTS, device=DEV).cumsum(0).int()
    a, a_s = exact_codes(g, T if gather else rows, K)
    index = torch.randint(0, 3 * T, (rows,), generator=g, device=DEV).int() if gather else None
    d = exact_d(g, rows, N, kind)
    want = expert_grad(d, a, a_s, offsets, index, 3, E)
    poison_lds()
    got = torch.full((E, N, K), float("nan"), dtype=TYPES[out], device=DEV)
    binding().fp8gemm_weight_grad_grouped(d, a, a_s, offsets, index=index, index_div=3, out=got, out_type=out)
    assert torch.equal(got, want.float().to(TYPES[out]))
