"""int8 quantizer and products (dense and by expert) against 64-bit forms."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from gpu_util import binding, poison_lds, say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {0: torch.float32, 1: torch.bfloat16, 2: torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert binding().mxgemm_device_supported()
    yield


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


# ---- quantizer --------------------------------------------------------------


def _check_quantize(x):
    b = binding()
    rows, K = x.shape
    q = torch.full((rows, K), 77, dtype=torch.int8, device=DEV)
    s = torch.full((rows,), -5.0, device=DEV)
    b.int8gemm_quantize(x, q=q, s=s)
    torch.cuda.synchronize()
    qr, sr = ref.quantize(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), sr, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), qr)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (5, 2032), (4, 2064), (300, 1024), (17, 8192), (9, 14336), (2, 65552)])
def test_quantize(kind, rows, K):
    say("quantize", kind, rows, K)
    rng = np.random.default_rng(rows * K + kind)
    x = rng.standard_normal((rows, K), dtype=np.float32)
    x[:, ::97] *= 20.0
    _check_quantize(dev(x).to(TYPES[kind]))


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_quantize_special_rows(kind):
    say("quantize special", kind)
    K = 272
    x = np.random.default_rng(1).standard_normal((14, K)).astype(np.float32)
    x[0] = 0.0
    x[1] = -0.0
    x[2, 100] = np.nan
    x[3, 271] = np.inf
    x[4, 0] = -np.inf
    # scale 1: every half is a tie
    x[5] = np.arange(K) % 127 - 63.5
    x[5, 7] = 127.0
    # scale 2^-10, ties again
    x[6] = (np.arange(K) % 200 - 99.5) * 2.0 ** -10
    x[6, 3] = -127.0 * 2.0 ** -10
    x[7] = 0.0
    x[7, 5] = 1.0
    x[8] = 3.0
    x[9] *= np.float32(2.0 ** -120)
    x[10] *= np.float32(2.0 ** -125)   # scale held at 2^-126 (fp32; others are zero there)
    x[11] *= np.float32(2.0 ** -140)
    x[12] *= np.float32(1e4)
    x[13, :] = 1e-7
    x[13, 0] = 60000.0
    _check_quantize(dev(x).to(TYPES[kind]))


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("rows,K", [(1000, 16), (37, 64), (33, 128), (65, 112), (19, 256), (2050, 512), (2049, 1040),
                                    (2051, 2048), (2048, 4096), (700, 4096), (600, 8192), (513, 16384), (512, 8208),
                                    (3, 16400), (2, 32784), (1, 65536), (2, 131088)])
def test_quantize_row_lengths(kind, rows, K):
    """Every number of lanes per row; rows that are zero or not finite beside others."""
    say("quantize row lengths", kind, rows, K)
    x = np.random.default_rng(rows + K + kind).standard_normal((rows, K), dtype=np.float32)
    x[:, ::53] *= 9.0
    if rows > 16:
        x[3::16] = 0.0
        x[5::17, K - 1] = np.nan
        x[7::19, 0] = np.inf
        x[11::23, K // 2] = -np.inf
    _check_quantize(dev(x).to(TYPES[kind]))


@pytest.mark.parametrize("rows,K", [(1 << 18, 16384), (4100, 1 << 20), (1 << 20, 4096)])
def test_quantize_past_4_gib(rows, K):
    say("quantize past 4 GiB", rows, K)
    b = binding()
    x = torch.empty((rows, K), dtype=torch.bfloat16, device=DEV)
    some = torch.tensor([0, rows // 2 - 1, rows // 2, rows - 2, rows - 1], device=DEV)
    x[some] = torch.randn((5, K), device=DEV).to(torch.bfloat16)
    q, s = b.int8gemm_quantize(x)
    qr, sr = ref.quantize(x[some].float().cpu().numpy())
    assert np.array_equal(s[some].cpu().numpy(), sr) and np.array_equal(q[some].cpu().numpy(), qr)


# each number of lanes per row, in more workgroups than one dimension of the
# launch holds; the last is as many rows as a call can have
@pytest.mark.parametrize("rows,K", [((1 << 24) + 21, 16), ((1 << 20) + 3, 4112), ((1 << 20) + 5, 16400),
                                    ((1 << 22) + 7, 528), ((64 << 20) - 1, 272), (64 << 20, 16)])
def test_quantize_many_rows(rows, K):
    say("quantize many rows", rows, K)
    b = binding()
    x = torch.empty((rows, K), dtype=torch.bfloat16, device=DEV)
    some = torch.tensor([0, 1, (1 << 20) - 1, min(1 << 20, rows - 3), rows // 2, rows - 2, rows - 1], device=DEV)
    x[some] = torch.randn((len(some), K), device=DEV).to(torch.bfloat16)
    q, s = b.int8gemm_quantize(x)
    qr, sr = ref.quantize(x[some].float().cpu().numpy())
    assert np.array_equal(s[some].cpu().numpy(), sr) and np.array_equal(q[some].cpu().numpy(), qr)


def test_quantize_near_borders():
    """fp32 values one step to either side of every border between two codes."""
    say("quantize borders")
    rows = []
    rng = np.random.default_rng(2)
    for amax in rng.uniform(0.5, 2.0, 40).astype(np.float32):
        s = np.float32(np.float64(amax) / 127.0)
        border = ((np.arange(-127, 127) + 0.5) * np.float64(s)).astype(np.float32)
        vals = np.concatenate([border, np.nextafter(border, np.float32(np.inf)), np.nextafter(border, np.float32(-np.inf)),
                               np.full(6, amax, np.float32)])
        rows.append(np.clip(vals, -amax, amax))
    _check_quantize(dev(np.stack(rows)))


# ---- products ---------------------------------------------------------------


def _codes(rng, rows, K):
    return rng.integers(-128, 128, (rows, K), dtype=np.int64).astype(np.int8)


def _check(got, want, tol, kind, what):
    got = got.float().cpu().numpy().astype(np.float64)
    # a result of size |y| + tol is rounded by half a step of it; below the
    # type's smallest normal value the step no longer shrinks, so half of that
    # value's step is added (fp16: 2^-14 * 2^-11 = 2^-25)
    half = ref.half_step(TYPES[kind])
    bound = tol + half * (np.abs(want) + tol) + half * torch.finfo(TYPES[kind]).smallest_normal
    off = np.abs(got - want)
    worst = np.max(off / np.maximum(bound, 1e-300))
    say("  %s: error / bound %.3g" % (what, worst))
    assert np.isfinite(got).all()
    assert worst <= 1.0


def _dense(M, N, K, kind, bias, act, seed):
    rng = np.random.default_rng(seed)
    a, w = _codes(rng, M, K), _codes(rng, N, K)
    a_s = rng.uniform(0.5, 1.5, M).astype(np.float32) / 128
    b_s = rng.uniform(0.5, 1.5, N).astype(np.float32) / (128 * np.sqrt(K).astype(np.float32))
    bi = rng.standard_normal(N).astype(np.float32) if bias else None
    want, tol = ref.product(a, a_s, w, b_s, bi, act)
    b = binding()
    out = torch.full((M, N), float("nan"), dtype=TYPES[kind], device=DEV)
    poison_lds()
    b.int8gemm_run(dev(a), dev(a_s), dev(w), dev(b_s), bias=None if bi is None else dev(bi),
                   act=b.ACT_GELU if act else b.ACT_NONE, out_type=kind, out=out)
    torch.cuda.synchronize()
    _check(out, want, tol, kind, "%dx%dx%d" % (M, N, K))
    return out


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 3, 48), (1, 4096, 4096), (2, 100, 80), (5, 17, 2064), (15, 256, 1024), (16, 1000, 8192), (17, 260, 4096),
    (31, 64, 144), (32, 512, 2048), (33, 1028, 1040), (48, 300, 512), (64, 4100, 2064), (65, 129, 272), (100, 1000, 1008),
    (128, 128, 128), (129, 257, 4096), (256, 256, 64), (300, 640, 2000), (512, 512, 1024), (1000, 200, 16), (777, 1031, 528),
    (64, 5000, 96), (1, 20000, 32)])
def test_product(M, N, K):
    say("product", M, N, K)
    _dense(M, N, K, 0, False, False, M * 7 + N * 3 + K)


@pytest.mark.parametrize("M,N,K", [(1024, 2048, 1024), (2304, 2560, 256), (2049, 2300, 400)])
def test_product_larger(M, N, K):
    say("product", M, N, K)
    _dense(M, N, K, 1, True, False, 5)


def _exact64(a, a_s, w, w_s):
    """The product in float64 on the GPU (integers below 2^53: the sums are
    exact), and the tolerance of its fp32 evaluation without bias and activation."""
    y = (a.double() @ w.double().t()) * a_s.double()[:, None] * w_s.double()[None, :]
    return y, 3.01 * 2.0 ** -24 * y.abs()


# sizes that take each tile shape, with more tiles than run at once, ragged
# rows and columns and a partial last slice
@pytest.mark.parametrize("M,N,K", [
    (515, 966, 4800), (489, 2034, 5488), (931, 515, 4624), (1939, 2046, 1776), (8192, 4301, 400), (2050, 8203, 2000),
    (5000, 9001, 1104), (4097, 4099, 144)])
def test_product_many_tiles(M, N, K):
    say("product many tiles", M, N, K)
    b = binding()
    g = torch.Generator(device=DEV).manual_seed(M)
    a, w = (torch.empty((n, K), dtype=torch.int8, device=DEV).random_(-128, 128, generator=g) for n in (M, N))
    a_s, w_s = (torch.rand(n, device=DEV, generator=g) + 0.5 for n in (M, N))
    out = torch.full((M, N), float("nan"), device=DEV)
    poison_lds()
    b.int8gemm_run(a, a_s, w, w_s, out=out)
    want, tol = _exact64(a, a_s, w, w_s)
    assert ((out.double() - want).abs() <= tol + 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("E,tokens,div,N,K", [
    (40, 111, 2, 587, 3488), (40, 255, 2, 3201, 624), (2, 1966, 3, 3331, 1344), (3, 4500, 2, 6101, 2064),
    (5, 2250, 4, 4201, 1040), (2, 32, 2, 301, 8208), (30, 30, 2, 2101, 4112), (64, 225, 4, 1101, 2064)])
def test_experts_many_tiles(E, tokens, div, N, K):
    say("experts many tiles", E, tokens, div, N, K)
    b = binding()
    rows = tokens * div
    g = torch.Generator(device=DEV).manual_seed(rows)
    a = torch.empty((tokens, K), dtype=torch.int8, device=DEV).random_(-128, 128, generator=g)
    w = torch.empty((E, N, K), dtype=torch.int8, device=DEV).random_(-128, 128, generator=g)
    a_s, w_s = torch.rand(tokens, device=DEV, generator=g) + 0.5, torch.rand((E, N), device=DEV, generator=g) + 0.5
    off = _counts(np.random.default_rng(rows), E, rows, 0.7).astype(np.int32)
    index = torch.randperm(rows, device=DEV, generator=g).int()
    out = torch.full((rows, N), float("nan"), device=DEV)
    poison_lds()
    b.int8gemm_run_grouped(a, a_s, w, w_s, dev(off), index=index, index_div=div, out=out)
    src = (index // div).long()
    for e in range(E):
        mine = slice(int(off[e]), int(off[e + 1]))
        if off[e + 1] > off[e]:
            want, tol = _exact64(a[src[mine]], a_s[src[mine]], w[e], w_s[e])
            assert ((out[mine].double() - want).abs() <= tol + 2.0 ** -24 * want.abs()).all(), e
    # rows already sorted: the same without an index
    again = b.int8gemm_run_grouped(a[src], a_s[src], w, w_s, dev(off))
    assert torch.equal(out, again)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("bias,act", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,N,K", [(3, 67, 160), (16, 512, 1024), (70, 132, 272), (260, 516, 1040)])
def test_product_output_step(kind, bias, act, M, N, K):
    say("product output", kind, bias, act, M, N, K)
    _dense(M, N, K, kind, bias, act, M + N + K + kind)


@pytest.mark.parametrize("M", [1, 20, 130, 300])
@pytest.mark.parametrize("a,b", [(-128, -128), (127, -128), (-127, 127)])
def test_product_largest_sums(M, a, b):
    """Every product at its largest, at the largest K: the sum fills 32 bits."""
    say("largest sums", M, a, b)
    bd = binding()
    K = bd.INT8_MAX_K
    N = 34
    out = bd.int8gemm_run(torch.full((M, K), a, dtype=torch.int8, device=DEV), torch.ones(M, device=DEV),
                          torch.full((N, K), b, dtype=torch.int8, device=DEV), torch.ones(N, device=DEV))
    torch.cuda.synchronize()
    want = np.float32(a * b * K)
    assert (out.cpu().numpy() == want).all()


def test_product_scale_values():
    """A zero, an infinite and a NaN scale reach their row or column alone."""
    say("scale values")
    b = binding()
    rng = np.random.default_rng(3)
    for M in (5, 140):
        N, K = 40, 64
        a, w = _codes(rng, M, K), _codes(rng, N, K)
        a_s, b_s = np.ones(M, np.float32), np.ones(N, np.float32)
        a_s[2], a_s[3], b_s[7], b_s[9] = 0.0, np.nan, np.inf, np.nan
        got = b.int8gemm_run(dev(a), dev(a_s), dev(w), dev(b_s)).cpu().numpy()
        s = (a.astype(np.int64) @ w.astype(np.int64).T).astype(np.float32)
        with np.errstate(all="ignore"):
            want = (s * a_s[:, None]) * b_s[None, :]
        assert np.array_equal(got, want, equal_nan=True)


# ---- by expert --------------------------------------------------------------


def _experts(offsets, rows, N, K, kind=0, tokens=None, div=1, bias=False, act=False, seed=0, index=None):
    """Runs the experts' products into a filled buffer; (result, expected, tolerance, rows that belong to an expert)."""
    rng = np.random.default_rng(seed)
    E = len(offsets) - 1
    rows_a = rows if tokens is None else tokens
    a, w = _codes(rng, rows_a, K), _codes(rng, E * N, K).reshape(E, N, K)
    a_s = rng.uniform(0.5, 1.5, rows_a).astype(np.float32) / 128
    b_s = (rng.uniform(0.5, 1.5, (E, N)) / (128 * np.sqrt(K))).astype(np.float32)
    bi = rng.standard_normal((E, N)).astype(np.float32) if bias else None
    if tokens is not None and index is None:
        index = rng.permutation(tokens * div)[:rows].astype(np.int32)
    src = np.arange(rows) if index is None else np.where(index < 0, -1, index // div)
    src = np.where(src >= rows_a, -1, src)
    want, tol = np.full((rows, N), np.nan), np.zeros((rows, N))
    owned = np.zeros(rows, bool)
    edges = np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, rows))
    for e in range(E):
        mine = np.arange(edges[e], edges[e + 1])
        owned[mine] = True
        ok = mine[src[mine] >= 0]
        if ok.size:
            want[ok], tol[ok] = ref.product(a[src[ok]], a_s[src[ok]], w[e], b_s[e], None if bi is None else bi[e], act)
    b = binding()
    out = torch.full((rows, N), 123.0, dtype=TYPES[kind], device=DEV)
    poison_lds()
    b.int8gemm_run_grouped(dev(a), dev(a_s), dev(w), dev(b_s), dev(np.asarray(offsets, np.int32)),
                           index=None if index is None else dev(index.astype(np.int32)), index_div=div,
                           bias=None if bi is None else dev(bi), act=b.ACT_GELU if act else b.ACT_NONE, out_type=kind,
                           out=out)
    torch.cuda.synchronize()
    return out, want, tol, owned


def _check_experts(out, want, tol, owned, kind, what):
    assert (out.float().cpu().numpy()[~owned] == 123.0).all(), "rows of no expert were written"
    bad = owned & np.isnan(want).any(1)
    assert torch.isnan(out).cpu().numpy()[bad].all()
    good = owned & ~bad
    if good.any():
        _check(out[torch.from_numpy(good).to(DEV)], want[good], tol[good], kind, what)


def _counts(rng, E, rows, skew):
    p = rng.dirichlet(np.full(E, skew))
    return np.concatenate([[0], np.cumsum(rng.multinomial(rows, p))])


@pytest.mark.parametrize("E,rows,N,K,skew", [
    (1, 1, 16, 16, 1.0), (8, 5, 64, 64, 1.0), (64, 64, 128, 256, 1.0), (64, 40, 100, 272, 0.1), (5, 300, 132, 144, 1.0),
    (16, 1000, 260, 512, 0.3), (3, 700, 512, 1024, 5.0), (1024, 2000, 20, 32, 0.5), (100, 3000, 68, 80, 0.05),
    (7, 2000, 300, 208, 1.0), (2, 4096, 256, 128, 50.0), (130, 130, 33, 48, 1.0)])
def test_experts(E, rows, N, K, skew):
    say("experts", E, rows, N, K)
    off = _counts(np.random.default_rng(E + rows), E, rows, skew)
    _check_experts(*_experts(off, rows, N, K, seed=E), 0, "experts")


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("E,tokens,div,N,K", [(8, 16, 4, 128, 256), (16, 200, 2, 72, 144), (32, 1, 8, 256, 512),
                                              (4, 600, 3, 260, 272)])
def test_experts_with_index(kind, E, tokens, div, N, K):
    say("experts index", kind, E, tokens, div, N, K)
    rows = tokens * div
    off = _counts(np.random.default_rng(rows), E, rows, 1.0)
    _check_experts(*_experts(off, rows, N, K, kind, tokens=tokens, div=div, bias=True, act=kind != 0, seed=rows), kind,
                   "experts")


@pytest.mark.parametrize("rows", [7, 40, 700])
@pytest.mark.parametrize("offsets", [
    (0, 0, 0, 0), (3, 3, 5, 5), (2, 4, 4, 6), (0, 7, 7, 7), (-5, 2, 3, 1000000), (5, 2, 6, 4), (7, 7, 7, 9), (0, 1, 2, 3),
    (-2147483648, 2147483647, 0, 3)])
def test_experts_offsets(rows, offsets):
    """Empty experts, rows in front and behind left alone, offsets outside the rows and falling."""
    say("experts offsets", rows, offsets)
    _check_experts(*_experts(offsets, rows, 36, 80, seed=9), 0, "experts")


@pytest.mark.parametrize("rows", [12, 400])
def test_experts_index_outside(rows):
    say("experts index outside", rows)
    index = np.arange(rows, dtype=np.int32)
    index[[1, 5]] = -1
    index[3] = rows * 2
    index[7] = 2147483647
    index[9] = -2147483648
    index[10] = 2                                   # the same row twice
    off = (0, rows // 3, rows // 3, rows)
    out = _experts(off, rows, 44, 64, tokens=rows // 2, div=2, index=index, seed=4)
    _check_experts(*out, 0, "experts")


def test_dense_is_one_expert():
    """The sums are exact, so the dense product and one expert's agree bit for bit, whatever kernels they take."""
    b = binding()
    rng = np.random.default_rng(8)
    for M in (1, 16, 40, 100, 300, 600):
        say("dense = one expert", M)
        a, w = dev(_codes(rng, M, 528)), dev(_codes(rng, 260, 528))
        a_s, b_s = torch.rand(M, device=DEV), torch.rand(260, device=DEV)
        bias = torch.rand(260, device=DEV)
        for kind in (0, 1, 2):
            x = b.int8gemm_run(a, a_s, w, b_s, bias=bias, act=b.ACT_GELU, out_type=kind)
            off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
            y = b.int8gemm_run_grouped(a, a_s, w[None], b_s[None], off, bias=bias[None], act=b.ACT_GELU, out_type=kind)
            z = b.int8gemm_run_grouped(a, a_s, w[None].expand(70, -1, -1).contiguous(), b_s[None].expand(70, -1).contiguous(),
                                       torch.tensor([0] * 35 + [M // 2] * 20 + [M] * 16, dtype=torch.int32, device=DEV),
                                       bias=bias[None].expand(70, -1).contiguous(), act=b.ACT_GELU, out_type=kind)
            assert torch.equal(x, y) and torch.equal(x, z)


def test_weights_past_4_gib():
    say("weights past 4 GiB")
    b = binding()
    E, N, K, rows = 70, 8192, 8192, 70
    w = torch.empty((E, N, K), dtype=torch.int8, device=DEV).random_(-128, 128)
    a = torch.empty((rows, K), dtype=torch.int8, device=DEV).random_(-128, 128)
    one = torch.ones(rows, device=DEV)
    off = torch.arange(E + 1, dtype=torch.int32, device=DEV)
    got = b.int8gemm_run_grouped(a, one, w, torch.ones(E, N, device=DEV), off)
    for e in (0, 31, 32, 63, 64, 69):
        want = (a[e].double()[None] @ w[e].double().t())[0].float()
        assert torch.equal(got[e], want), e


def test_gathered_rows_past_4_gib():
    say("gathered rows past 4 GiB")
    b = binding()
    T, K, N, E = 262144 + 70, 16384, 100, 3
    a = torch.empty((T, K), dtype=torch.int8, device=DEV)
    index = torch.tensor([T - 1, 0, 262143, 262144, T, -1, 131072, T - 1], dtype=torch.int32, device=DEV)
    rows = index[[0, 1, 2, 3, 6]].long()
    a[rows] = torch.empty((5, K), dtype=torch.int8, device=DEV).random_(-128, 128)
    w = torch.empty((E, N, K), dtype=torch.int8, device=DEV).random_(-128, 128)
    off = torch.tensor([0, 3, 3, 8], dtype=torch.int32, device=DEV)
    got = b.int8gemm_run_grouped(a, torch.ones(T, device=DEV), w, torch.ones(E, N, device=DEV), off, index=index)
    for p, e in ((0, 0), (1, 0), (2, 0), (3, 2), (6, 2), (7, 2)):
        want = (a[int(index[p])].double()[None] @ w[e].double().t())[0].float()
        assert torch.equal(got[p], want), p
    assert torch.isnan(got[4:6]).all()


def test_many_gathered_rows_past_4_gib():
    """More tiles than run at once of the kernel that takes such an A."""
    say("many gathered rows past 4 GiB")
    b = binding()
    T, K, N, E, rows = 262144 + 70, 16384, 100, 3, 64 * 2048 + 17
    used = torch.tensor([T - 1, 0, 262143, 262144, 131072, 7], device=DEV)
    a = torch.empty((T, K), dtype=torch.int8, device=DEV)
    a[used] = torch.empty((len(used), K), dtype=torch.int8, device=DEV).random_(-128, 128)
    w = torch.empty((E, N, K), dtype=torch.int8, device=DEV).random_(-128, 128)
    bounds = [0, 50001, 50001, rows]
    pick = torch.arange(rows, device=DEV) * 7 // 5 % len(used)
    got = b.int8gemm_run_grouped(a, torch.ones(T, device=DEV), w, torch.ones(E, N, device=DEV),
                                 torch.tensor(bounds, dtype=torch.int32, device=DEV), index=used[pick].int())
    for e in range(E):
        want = (a[used].double() @ w[e].double().t()).float()
        assert torch.equal(got[bounds[e]:bounds[e + 1]], want[pick[bounds[e]:bounds[e + 1]]]), e


def test_output_past_4_gib():
    say("output past 4 GiB")
    b = binding()
    M, N, K = 70000, 16400, 16
    a = torch.empty((M, K), dtype=torch.int8, device=DEV).random_(-128, 128)
    w = torch.empty((N, K), dtype=torch.int8, device=DEV).random_(-128, 128)
    got = b.int8gemm_run(a, torch.ones(M, device=DEV), w, torch.ones(N, device=DEV))
    for r in (slice(0, 64), slice(32700, 32840), slice(65400, 65600), slice(M - 70, M)):
        assert torch.equal(got[r], (a[r].double() @ w.double().t()).float())


def test_two_calls_at_once():
    """Products, routing and plans of two streams side by side give what they give alone."""
    say("two calls at once")
    b = binding()
    sets = []
    for seed, T in ((1, 3000), (2, 40)):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x = torch.randn((T, 528), device=DEV, generator=g)
        w, w_s = b.int8gemm_quantize(torch.randn((8 * 700, 528), device=DEV, generator=g))
        logits = torch.randn((T, 8), device=DEV, generator=g)
        sets.append((x, w.view(8, 700, 528), w_s.view(8, 700), logits))

    def work(x, w, w_s, logits):
        ids, weights = b.expert_route(logits, 2)
        off, order, pos = b.expert_plan(ids, 8)
        q, s = b.int8gemm_quantize(x)
        y = b.int8gemm_run_grouped(q, s, w, w_s, off, index=order, index_div=2)
        return y, b.expert_combine(y, pos, weights), b.int8gemm_run(q, s, w[3], w_s[3])

    alone = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(work(*s))
        torch.cuda.synchronize()
        for x, y in zip(got, alone):
            assert all(torch.equal(u, v) for u, v in zip(x, y))


@pytest.mark.parametrize("M,N,K", [(1, 701, 272), (20, 1023, 528), (300, 517, 1040), (700, 4099, 2064), (2050, 4097, 1104)])
def test_one_expert_of_many(M, N, K):
    """Weights, scales and bias of one expert, and of a range of experts, as
    slices that start at any element: the same as copies of them."""
    say("one expert of many", M, N, K)
    b = binding()
    E = 5
    x, x_s = b.int8gemm_quantize(torch.randn((M, K), device=DEV))
    w = torch.empty((E, N, K), dtype=torch.int8, device=DEV).random_(-128, 128)
    w_s, bias = torch.rand((E, N), device=DEV) / K, torch.randn((E, N), device=DEV)
    side = torch.cuda.Stream()
    for kind in (0, 1, 2):
        kw = dict(act=b.ACT_GELU, out_type=kind)
        for e in (1, 2, 3):
            want = b.int8gemm_run(x, x_s, w[e], w_s[e].clone(), bias=bias[e].clone(), **kw)
            assert torch.equal(b.int8gemm_run(x, x_s, w[e], w_s[e], bias=bias[e], **kw), want)
        torch.cuda.synchronize()
        got = b.int8gemm_run(x, x_s, w[3], w_s[3], bias=bias[3], stream=side, **kw)
        side.synchronize()
        assert torch.equal(got, want)
        off = torch.tensor([0, M // 3, M // 3, M], dtype=torch.int32, device=DEV)
        want = b.int8gemm_run_grouped(x, x_s, w[1:4], w_s[1:4].clone(), off, bias=bias[1:4].clone(), **kw)
        assert torch.equal(b.int8gemm_run_grouped(x, x_s, w[1:4], w_s[1:4], off, bias=bias[1:4], **kw), want)
    # captured, with other values at each replay
    out = torch.empty((M, N), device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.int8gemm_run(x, x_s, w[1], w_s[1], bias=bias[1], out=out)
    for _ in range(3):
        bias.normal_()
        want = b.int8gemm_run(x, x_s, w[1], w_s[1], bias=bias[1])
        torch.cuda.synchronize()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# ---- streams, graphs, refusals ----------------------------------------------


def test_side_stream():
    """The call joins the stream it is given, and the current one without."""
    say("side stream")
    b = binding()
    rng = np.random.default_rng(11)
    x = dev(rng.standard_normal((64, 2048)).astype(np.float32))
    w, w_s = b.int8gemm_quantize(dev(rng.standard_normal((512, 2048)).astype(np.float32)))
    want = b.int8gemm_run(*b.int8gemm_quantize(x), w, w_s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for given in (True, False):
        big = torch.zeros(64 << 20, device=DEV)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            y = torch.zeros_like(x)
            for _ in range(20):
                big.add_(1.0)       # work that the call has to wait for
            y.copy_(x)
            if not given:
                got = b.int8gemm_run(*b.int8gemm_quantize(y), w, w_s)
        if given:
            q, s = b.int8gemm_quantize(y, stream=side)
            got = b.int8gemm_run(q, s, w, w_s, stream=side)
        side.synchronize()
        assert torch.equal(got, want)


def test_outputs_of_another_stream():
    """What a call on another stream allocates is not memory that the current
    stream's queued work still uses."""
    say("outputs of another stream")
    b = binding()
    x = torch.randn((512, 4096), device=DEV)
    want, _ = b.int8gemm_quantize(x)
    y, pos, w = torch.randn((64, 256), device=DEV), torch.arange(64, dtype=torch.int32, device=DEV).view(32, 2), torch.ones((32, 2), device=DEV)
    want_y, _ = b.expert_combine_backward(torch.ones((32, 256), device=DEV), y, pos, w)
    d_out = torch.ones((32, 256), device=DEV)
    side = torch.cuda.Stream()
    big = torch.zeros(64 << 20, device=DEV)
    torch.cuda.synchronize()
    for _ in range(3):
        held = [torch.empty((512, 4096), dtype=torch.int8, device=DEV), torch.empty((64, 256), device=DEV)]
        torch.cuda.synchronize()
        for _ in range(30):
            big.add_(1.0)
        for t in held:
            t.fill_(7)
        del held, t
        q, _ = b.int8gemm_quantize(x, stream=side)
        d_y, _ = b.expert_combine_backward(d_out, y, pos, w, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(q, want) and torch.equal(d_y, want_y)


@pytest.mark.parametrize("M", [1, 16, 60, 300])
def test_graph_replay(M):
    say("graph replay int8", M)
    b = binding()
    rng = np.random.default_rng(M)
    N, K, E = 516, 1040, 6
    x = dev(rng.standard_normal((M, K)).astype(np.float32)).bfloat16()
    w = dev(_codes(rng, E * N, K)).view(E, N, K)
    w_s, bias = torch.rand(E, N, device=DEV), torch.rand(E, N, device=DEV)
    off = dev(_counts(rng, E, M, 1.0).astype(np.int32))
    q, s = torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    dense, by = torch.empty((M, N), dtype=torch.bfloat16, device=DEV), torch.empty((M, N), device=DEV)

    def run():
        b.int8gemm_quantize(x, q=q, s=s)
        b.int8gemm_run(q, s, w[0], w_s[0], bias=bias[0], act=b.ACT_GELU, out_type=b.OUT_BF16, out=dense)
        b.int8gemm_run_grouped(q, s, w, w_s, off, bias=bias, out=by)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for rep in range(3):
        x.copy_(dev(rng.standard_normal((M, K)).astype(np.float32)))
        off.copy_(dev(_counts(rng, E, M, 0.5).astype(np.int32)))
        run()
        torch.cuda.synchronize()
        want = [t.clone() for t in (q, s, dense, by)]
        for t in (q, s, dense, by):
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for got, t in zip((q, s, dense, by), want):
            assert torch.equal(got, t), rep


def test_refusals():
    say("refusals")
    b = binding()
    x = torch.zeros((4, 64), device=DEV)
    q, s = b.int8gemm_quantize(x)
    with pytest.raises(ValueError):
        b.int8gemm_quantize(x.t())
    with pytest.raises(ValueError):
        b.int8gemm_quantize(x[0])
    with pytest.raises(TypeError):
        b.int8gemm_quantize(x.double())
    with pytest.raises(b.MXGemmError):
        b.int8gemm_quantize(torch.zeros((4, 24), device=DEV))
    with pytest.raises(b.MXGemmError):
        b.int8gemm_quantize(torch.zeros((0, 64), device=DEV))
    with pytest.raises(ValueError):
        b.int8gemm_quantize(x, q=q[:2])
    with pytest.raises(TypeError):
        b.int8gemm_run(q.view(torch.uint8), s, q, s)
    with pytest.raises(ValueError):
        b.int8gemm_run(q, s[:3], q, s)
    with pytest.raises(ValueError):
        b.int8gemm_run(q, s, q[:, :32].contiguous(), s)
    with pytest.raises(ValueError):
        b.int8gemm_run(q, s, q, s.cpu())
    with pytest.raises(ValueError):
        b.int8gemm_run(q, s, q, s, out_type=7)
    with pytest.raises(b.MXGemmError):
        b.int8gemm_run(q, s, q, s, act=9)
    with pytest.raises(ValueError):
        b.int8gemm_run(q, s, q, s, bias=torch.zeros(5, device=DEV))
    with pytest.raises(TypeError):
        b.int8gemm_run(q, s, q, s, out_type=b.OUT_BF16, out=torch.zeros((4, 4), device=DEV))
    big = torch.zeros((1, b.INT8_MAX_K + 16), dtype=torch.int8, device=DEV)
    with pytest.raises(b.MXGemmError):
        b.int8gemm_run(big, s[:1].clone(), big, s[:1].clone())
    odd = torch.zeros(4 * 64 + 1, dtype=torch.int8, device=DEV)[1:].view(4, 64)
    with pytest.raises(b.MXGemmError):
        b.int8gemm_run(odd, s, q, s)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        b.int8gemm_run_grouped(q, s, q[None], s[None], off.long())
    with pytest.raises(ValueError):
        b.int8gemm_run_grouped(q, s, q[None], s[None], off[:1])
    with pytest.raises(ValueError):
        b.int8gemm_run_grouped(q, s, q, s, off)
    with pytest.raises(b.MXGemmError):
        b.int8gemm_run_grouped(q, s, q[None], s[None], off, index=off.clone(), index_div=0)
