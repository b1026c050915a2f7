"""E4M3 codes and products with a scale per block of 128, dense and by expert,
against the 64-bit forms."""
import pytest
import torch

import fp8_ref as ref
from gpu_util import binding, say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {0: torch.float32, 1: torch.bfloat16, 2: torch.float16}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert binding().mxgemm_device_supported()
    yield


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def exact_codes(g, rows, K, block_rows=1):
    """Codes of 0, +-1/2, +-1, +-2 and scales 1/2, 1, 2: any sum of products of two
    such values over fewer than 2^15 columns is a multiple of 1/16 below 2^20, which fp32
    holds, whatever the order."""
    v = torch.tensor([0.0, 0.5, -0.5, 1.0, -1.0, 2.0, -2.0], device=DEV)
    q = ref.encode(v[torch.randint(0, 7, (rows, K), generator=g, device=DEV)].double())
    s = torch.tensor([0.5, 1.0, 2.0], device=DEV)[
        torch.randint(0, 3, (-(-rows // block_rows), -(-K // 128)), generator=g, device=DEV)]
    return q, s


# ---- quantizer ----------------------------------------------------------------


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 128), (5, 144), (127, 272), (128, 256), (129, 1040), (1, 16384), (1000, 96),
                                    (260, 4096), (4097, 112)])
def test_quantize(kind, pow2, block_rows, rows, K):
    say("fp8 quantize", kind, pow2, block_rows, rows, K)
    x = (randn(gen(rows + K), rows, K) * torch.exp2(torch.randint(-12, 4, (rows, 1), generator=gen(K), device=DEV).float())).to(
        TYPES[kind])
    q, s = binding().fp8gemm_quantize(x, block_rows, pow2)
    q_r, s_r = ref.quantize(x.float(), block_rows, pow2)
    assert torch.equal(s, s_r)
    assert torch.equal(q, q_r)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_borders(kind, block_rows):
    """Ties of codes, zeros of both signs, the smallest and largest values, blocks
    with NaNs and infinities beside blocks without."""
    say("fp8 quantize borders", kind, block_rows)
    t = TYPES[kind]
    v = ref.values().to(DEV)
    x = torch.zeros(300, 400, device=DEV, dtype=torch.float64)
    ties = torch.cat([v[:64], (v[1:] + v[:-1])[:64] / 2])
    x[0, :128], x[1, :128] = ties, -ties
    x[0:2, 5] = 448.0 if block_rows == 1 else 0.0
    x[2, :3] = torch.tensor([0.0, -0.0, 448.0], device=DEV)
    x[5, ::3] = -0.0   # blocks of zeros keep the signs too
    x = x.to(t)
    x[3, 128:256] = torch.finfo(t).smallest_subnormal if hasattr(torch.finfo(t), "smallest_subnormal") else 1e-45
    x[4, 200] = torch.finfo(t).max
    x[140, 10], x[150, 300], x[299, 399] = float("inf"), float("nan"), -float("inf")
    for pow2 in (False, True):
        q, s = binding().fp8gemm_quantize(x, block_rows, pow2)
        q_r, s_r = ref.quantize(x.float(), block_rows, pow2)
        assert torch.equal(s.nan_to_num(-1.0), s_r.nan_to_num(-1.0))
        assert torch.equal(q, q_r)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_next_to_ties(block_rows):
    """fp32 values that are a few steps from a tie of two codes, for scales of any
    mantissa and of every size."""
    say("fp8 quantize next to ties", block_rows)
    v = ref.values().to(DEV)
    ties = (v[1:] + v[:-1]) / 2
    blocks = 6 * 250
    g = gen(block_rows)
    exponent = torch.arange(250, device=DEV).repeat(6) - 125
    amax = torch.ldexp(1 + torch.rand(blocks, generator=g, device=DEV), exponent)
    s = ref.scale_of(amax, False).double()
    x = torch.zeros(blocks, 128, device=DEV)
    at = torch.randint(0, 126, (blocks, 127), generator=g, device=DEV)
    near = (ties[at] * s[:, None]).float()
    step = torch.randint(-2, 3, (blocks, 127), generator=g, device=DEV)
    for _ in range(2):
        near = torch.where(step > 0, torch.nextafter(near, near + 1e30), torch.where(step < 0, torch.nextafter(near, -near), near))
        step = step - step.sign()
    x[:, 1:] = near * torch.where(torch.rand(blocks, 127, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    x = torch.minimum(torch.maximum(x, -amax[:, None]), amax[:, None])
    x[:, 0] = amax
    if block_rows == 128:
        full = torch.zeros(blocks, 128, 128, device=DEV)
        full[:, 77] = x
        x = full.view(blocks * 128, 128)
    q, scale = binding().fp8gemm_quantize(x, block_rows)
    q_r, s_r = ref.quantize(x, block_rows)
    assert torch.equal(scale, s_r)
    assert torch.equal(q, q_r)


def test_quantize_experts():
    say("fp8 quantize experts")
    for block_rows in (1, 128):
        x = randn(gen(4), 3, 200, 336)
        q, s = binding().fp8gemm_quantize(x, block_rows)
        for e in range(3):
            q_r, s_r = ref.quantize(x[e], block_rows)
            assert torch.equal(q[e], q_r) and torch.equal(s[e], s_r)


def test_quantize_rows_past_4_gib():
    say("fp8 quantize rows past 4 GiB")
    rows, K = 2 ** 26, 80
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 1, 2 ** 25 + 3, rows - 2, rows - 1], device=DEV)
    x[at] = randn(gen(9), 5, K).to(torch.bfloat16)
    q, s = binding().fp8gemm_quantize(x)
    q_r, s_r = ref.quantize(x[at].float())
    assert torch.equal(q[at], q_r) and torch.equal(s[at], s_r)
    assert int((s != 0).sum()) == 5


# ---- products -----------------------------------------------------------------


def result_tol(y, err, act, out):
    """Error allowed to the results, with err that of the sums: bias (one rounding);
    GELU is Lipschitz with 1.13 and its evaluation off by 4e-7 of y/2 and 2^-23 of the
    result; half a step of the output type."""
    err = err + U * y.abs()
    if act:
        g = ref.gelu(y)
        err = 1.13 * err + y.abs() * 4e-7 + 2.0 ** -23 * g.abs()
        y = g
    return err + torch.finfo(out).eps / 2 * (y.abs() + err) + (2.0 ** -25 if out == torch.float16 else 2.0 ** -140)


def check(got, y, top, mass, KB, bias, act, out):
    """Against 64 bits.  A block's MFMA drops at most 2^-7 of its largest product
    (gpu_util.MFMA_STEP_KAPPA); its fma and the scales' product round to 2^-24 of a
    term, and the running sum to 2^-24 of what it holds, once a block, twice where
    the sums of several waves are joined."""
    err = top * 2.0 ** -7 + mass * U * (2 * KB + 4)
    y = y if bias is None else y + bias.double()
    tol = result_tol(y, err, act, out)
    want = ref.gelu(y) if act else y
    off = (got.double() - want).abs()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ratio = torch.where(torch.isnan(want), torch.zeros_like(off), off / tol)
    say("  error / bound %.3g" % ratio.max().item())
    assert bool((ratio <= 1).all())


def normal_codes(g, rows, K, block_rows=1, size=1.0, pow2=False):
    return ref.quantize(randn(g, rows, K) * size, block_rows, pow2)


SIZES = [(1, 1, 16), (1, 16, 128), (2, 130, 144), (3, 5, 272), (16, 16, 256), (17, 300, 1040), (16, 512, 4096), (33, 129, 528),
         (64, 256, 2048), (65, 64, 4112), (100, 1000, 96), (129, 257, 384), (256, 256, 512), (300, 700, 1168),
         (513, 384, 640), (777, 1030, 2064), (1024, 2048, 256), (40, 4100, 7168)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out", [0, 1, 2])
def test_product(M, N, K, out):
    say("fp8 product", M, N, K, out)
    g = gen(M + N + K)
    a, a_s = normal_codes(g, M, K)
    b, b_s = normal_codes(g, N, K, 128, 0.02)
    y, top, mass = ref.product(a, a_s, b, b_s)
    bn = binding()
    got = bn.fp8gemm_run(a, a_s, b, b_s, out_type=out)
    check(got, y, top, mass, a_s.shape[1], None, False, TYPES[out])
    bias = randn(g, N)
    got = bn.fp8gemm_run(a.view(torch.float8_e4m3fn), a_s, b.view(torch.float8_e4m3fn), b_s, bias=bias, act=1, out_type=out)
    check(got, y, top, mass, a_s.shape[1], bias, True, TYPES[out])


def test_product_error_on_normal_data():
    """2^-16 of the results, root mean square, as the entry point's comment has it."""
    say("fp8 product error")
    g = gen(3)
    for K in (128, 4096):
        a, a_s = normal_codes(g, 512, K)
        b, b_s = normal_codes(g, 512, K, 128)
        y, _, _ = ref.product(a, a_s, b, b_s)
        got = binding().fp8gemm_run(a, a_s, b, b_s).double()
        rms = ((got - y).square().mean() / y.square().mean()).sqrt().item()
        say("  rms 2^%.2f" % torch.tensor(rms).log2().item())
        assert rms <= 2.0 ** -15


EXACT = SIZES + [(1, 4096, 512), (8, 28672, 256), (48, 2064, 1536), (200, 4096, 400), (2048, 1000, 1024), (4096, 4096, 384),
                 (1111, 6000, 2000 // 16 * 16), (8192, 1024, 128), (16, 2000, 32768 - 16)]


@pytest.mark.parametrize("M,N,K", EXACT)
def test_product_exact(M, N, K):
    """Sums that are exact in any order: equal, from every kernel."""
    say("fp8 product exact", M, N, K)
    g = gen(M + N + K)
    a, a_s = exact_codes(g, M, K)
    b, b_s = exact_codes(g, N, K, 128)
    y = ref.dequantize(a, a_s) @ ref.dequantize(b, b_s, 128).t()
    assert torch.equal(binding().fp8gemm_run(a, a_s, b, b_s).double(), y)


@pytest.mark.parametrize("M", [5, 200, 2000])
def test_product_specials(M):
    """NaN codes, NaN and infinite scales, and zero scales reach the results of their
    rows and columns alone."""
    say("fp8 product specials", M)
    N, K = 520, 400
    g = gen(M)
    a, a_s = exact_codes(g, M, K)
    b, b_s = exact_codes(g, N, K, 128)
    a[1, 399] = 0x7F           # the last column
    a_s[2, 1] = float("nan")
    a_s[3] = 0.0
    b[7, 130] = 0xFF
    b_s[1, 3] = float("nan")   # columns 128 .. 255, the partial block
    y = ref.dequantize(a, a_s) @ ref.dequantize(b, b_s, 128).t()
    got = binding().fp8gemm_run(a, a_s, b, b_s).double()
    assert torch.equal(torch.isnan(got), torch.isnan(y))
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 200]).all() and not torch.isnan(y[0, :7]).any()
    ok = ~torch.isnan(y)
    assert torch.equal(got[ok], y[ok])
    a_s[0, 2] = float("inf")
    got = binding().fp8gemm_run(a, a_s, b, b_s)
    assert not torch.isfinite(got[0]).any()


def test_product_scale_layout():
    """Views of scales that start at any element, and out given."""
    say("fp8 product scale layout")
    g = gen(11)
    a, a_s = exact_codes(g, 70, 640)
    b, b_s = exact_codes(g, 300, 640, 128)
    hold = torch.zeros(a_s.numel() + b_s.numel() + 2, device=DEV)
    a2, b2 = hold[1:1 + a_s.numel()].view_as(a_s), hold[2 + a_s.numel():].view_as(b_s)
    a2.copy_(a_s)
    b2.copy_(b_s)
    out = torch.full((70, 300), float("nan"), device=DEV)
    got = binding().fp8gemm_run(a, a2, b, b2, out=out)
    assert got is out
    assert torch.equal(out.double(), ref.dequantize(a, a_s) @ ref.dequantize(b, b_s, 128).t())


# ---- by expert ------------------------------------------------------------------


def expert_case(g, E, tokens, k, N, K):
    a, a_s = exact_codes(g, tokens, K)
    w = [exact_codes(g, N, K, 128) for _ in range(E)]
    b, b_s = torch.stack([x[0] for x in w]), torch.stack([x[1] for x in w])
    ids = torch.rand(tokens, E, generator=g, device=DEV).topk(k, 1).indices.int()
    return a, a_s, b, b_s, ids


def expert_result(a, a_s, b, b_s, offsets, index, div, rows):
    """Rows inside the offsets in 64 bits; the others NaN here."""
    E, N, _ = b.shape
    x = ref.dequantize(a, a_s)
    y = torch.full((rows, N), float("nan"), dtype=torch.float64, device=a.device)
    for e, (lo, hi) in enumerate(ref.rows_of_experts(offsets.tolist(), rows)):
        at = torch.arange(lo, hi, device=a.device)
        if index is not None:
            at = torch.where(index[lo:hi] < 0, -1, torch.div(index[lo:hi], div, rounding_mode="floor")).long()
        good = (at >= 0) & (at < a.shape[0])
        part = x[at.clamp(0, a.shape[0] - 1)] @ ref.dequantize(b[e], b_s[e], 128).t()
        y[lo:hi] = torch.where(good[:, None], part, torch.full_like(part, float("nan")))
    return y


@pytest.mark.parametrize("E,tokens,k,N,K", [(1, 1, 1, 16, 128), (4, 3, 2, 130, 144), (8, 16, 2, 300, 1040), (64, 16, 4, 128, 512),
                                            (7, 100, 3, 257, 272), (16, 300, 4, 520, 640), (2, 1000, 2, 256, 256),
                                            (130, 40, 8, 64, 384), (16, 1024, 4, 512, 512), (5, 2000, 2, 1000, 400),
                                            (1024, 30, 2, 32, 128), (64, 1024, 4, 256, 256)])
def test_experts(E, tokens, k, N, K):
    say("fp8 experts", E, tokens, k, N, K)
    g = gen(E + tokens + N)
    a, a_s, b, b_s, ids = expert_case(g, E, tokens, k, N, K)
    bn = binding()
    offsets, order, _ = bn.expert_plan(ids, E)
    got = bn.fp8gemm_run_grouped(a, a_s, b, b_s, offsets, index=order, index_div=k)
    assert torch.equal(got.double(), expert_result(a, a_s, b, b_s, offsets, order, k, tokens * k))
    # the rows already sorted, with bias and activation
    at = (order // k).long()
    bias = randn(g, E, N)
    got = bn.fp8gemm_run_grouped(a[at], a_s[at], b, b_s, offsets, bias=bias, act=1, out_type=1)
    y = expert_result(a, a_s, b, b_s, offsets, order, k, tokens * k)
    y = y + bias.double()[ids.reshape(-1)[order.long()].long()]
    assert bool(((got.double() - ref.gelu(y)).abs() <= result_tol(y, torch.zeros_like(y), True, torch.bfloat16)).all())


@pytest.mark.parametrize("rows", [20, 300])
def test_experts_offsets_and_index(rows):
    """Offsets that start late, end early, fall or lie outside; indices outside A;
    rows that no expert has are left as they were."""
    say("fp8 experts offsets and index", rows)
    E, N, K, T = 5, 200, 272, 40
    g = gen(rows)
    a, a_s, b, b_s, _ = expert_case(g, E, T, 1, N, K)
    r = rows
    index = torch.randint(0, 2 * T, (rows,), generator=g, device=DEV).int()
    index[3], index[4], index[5] = -1, 2 * T, 2 ** 31 - 1
    for offsets in ([2, 2, 7, 9, 15, r - 4], [0] * 6, [0, 0, 0, r, r, r], [-5, 3, 1, 12, 10, r + 50], [r, r, r, r, r, r],
                    [4, 2 ** 31 - 1, 5, 6, 7, 8], [-2 ** 31, -1, 0, 1, 2, 3]):
        off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        out = torch.full((rows, N), -7.0, device=DEV)
        binding().fp8gemm_run_grouped(a, a_s, b, b_s, off, index=index, index_div=2, out=out)
        y = expert_result(a, a_s, b, b_s, off, index, 2, rows)
        inside = torch.zeros(rows, dtype=torch.bool, device=DEV)
        for lo, hi in ref.rows_of_experts(offsets, rows):
            inside[lo:hi] = True
        assert bool((out[~inside] == -7.0).all())
        assert torch.equal(out[inside].double().nan_to_num(-9.0), y[inside].nan_to_num(-9.0))


@pytest.mark.parametrize("rows", [64, 700])
def test_experts_gathered_rows_past_4_gib(rows):
    say("fp8 experts rows past 4 GiB", rows)
    K, N, E = 4096, 136, 3
    big = 2 ** 20 + 5000
    a = torch.zeros(big, K, dtype=torch.uint8, device=DEV)
    a_s = torch.zeros(big, 32, device=DEV)
    g = gen(rows)
    at = torch.randint(0, big, (rows,), generator=g, device=DEV).int()
    at[0], at[1] = big - 1, 2 ** 20 + 1
    q, s = exact_codes(g, rows, K)
    a[at.long()], a_s[at.long()] = q, s
    w = [exact_codes(g, N, K, 128) for _ in range(E)]
    b, b_s = torch.stack([x[0] for x in w]), torch.stack([x[1] for x in w])
    off = torch.tensor([0, rows // 3, rows // 2, rows], dtype=torch.int32, device=DEV)
    got = binding().fp8gemm_run_grouped(a, a_s, b, b_s, off, index=at)
    q, s = a[at.long()], a_s[at.long()]
    assert torch.equal(got.double(), expert_result(q, s, b, b_s, off, None, 1, rows))


# ---- streams, graphs, refusals ----------------------------------------------------


@pytest.mark.parametrize("M", [4, 70, 600])
def test_graph_replay(M):
    """Quantizer and products captured together; every replay against the eager calls,
    with eager work between."""
    say("graph replay fp8", M)
    bn = binding()
    g = gen(M)
    N, K, E = 384, 512, 4
    x = randn(g, M, K)
    w, w_s = bn.fp8gemm_quantize(randn(g, E, N, K) * 0.05, 128)
    off = torch.tensor([0, M // 4, M // 2, M // 2, M], dtype=torch.int32, device=DEV)

    def work():
        q, s = bn.fp8gemm_quantize(x)
        return q, s, bn.fp8gemm_run(q, s, w[0], w_s[0], out_type=1), bn.fp8gemm_run_grouped(q, s, w, w_s, off)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for i in range(4):
        x.copy_(randn(g, M, K) * (i + 1))
        graph.replay()
        got = [t.clone() for t in held]
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_side_streams():
    say("side streams fp8")
    bn = binding()
    g = gen(5)
    sets = []
    for M in (3, 90, 700, 2048):
        a, a_s = exact_codes(g, M, 1024)
        b, b_s = exact_codes(g, 640, 1024, 128)
        sets.append((a, a_s, b, b_s))
    want = [bn.fp8gemm_run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[bn.fp8gemm_run(*s, stream=st) for _ in range(5)] for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        assert all(torch.equal(w, m) for m in many)


def test_binding_refusals():
    bn = binding()
    g = gen(6)
    a, a_s = exact_codes(g, 8, 256)
    b, b_s = exact_codes(g, 300, 256, 128)
    x = randn(g, 8, 256)
    off = torch.zeros(2, dtype=torch.int32, device=DEV)
    for call in (lambda: bn.fp8gemm_quantize(x[:, :100]), lambda: bn.fp8gemm_quantize(x, 64), lambda: bn.fp8gemm_quantize(x[0]),
                 lambda: bn.fp8gemm_run(a, a_s, b[:, :128], b_s), lambda: bn.fp8gemm_run(a, a_s[:, :1], b, b_s),
                 lambda: bn.fp8gemm_run(a, a_s, b, b_s[:2]), lambda: bn.fp8gemm_run(a, a_s, b, b_s, out_type=5),
                 lambda: bn.fp8gemm_run(a, a_s, b, b_s, bias=a_s[0]), lambda: bn.fp8gemm_run(a.t(), a_s, b, b_s),
                 lambda: bn.fp8gemm_run(a, a_s, b, b_s, out=torch.empty(8, 299, device=DEV)),
                 lambda: bn.fp8gemm_run_grouped(a, a_s, b, b_s[None], off),
                 lambda: bn.fp8gemm_run_grouped(a, a_s, b[None], b_s[None], off[:1]),
                 lambda: bn.fp8gemm_run(a.cpu(), a_s, b, b_s)):
        with pytest.raises((ValueError, bn.MXGemmError)):
            call()
    for call in (lambda: bn.fp8gemm_run(a, a_s.half(), b, b_s), lambda: bn.fp8gemm_run(a.view(torch.int8), a_s, b, b_s),
                 lambda: bn.fp8gemm_quantize(x.double()), lambda: bn.fp8gemm_run_grouped(a, a_s, b[None], b_s[None], off.long())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(bn.MXGemmError):
        bn.fp8gemm_quantize(randn(g, 4, 24))
