"""int8 products on the large tiles: output step, special values, experts'
rows, and the agreement of all tiles, against float64 on the GPU.

Each case names the tile that it is there for; the library's own choice says
that it takes it (test_abi_int8.py checks the same without a GPU)."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from gpu_util import binding, poison_lds, say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {0: torch.float32, 1: torch.bfloat16, 2: torch.float16}
U = 2.0 ** -24

# variants in the order of csrc/int8_choice.h; "deep" is 128 x 128 with 8 waves
TILES = ["16x16", "16x32", "32x32", "32x64", "deep", "128x128", "256x128", "256x256"]
# tile, M, N, K: ragged in every size, then whole tiles
DENSE = [("deep", 1939, 2046, 1776), ("128x128", 4097, 4099, 144), ("128x128", 2051, 4098, 400),
         ("256x128", 2050, 8203, 2000), ("256x256", 5000, 9001, 1104), ("deep", 2048, 2048, 1040),
         ("128x128", 2048, 4096, 512), ("256x128", 2048, 4096, 1152), ("256x256", 4096, 4096, 1024)]
# tile, experts, tokens, choices, N, K
EXPERTS = [("deep", 64, 225, 4, 1101, 2064), ("128x128", 40, 255, 2, 3201, 624), ("256x128", 2, 1966, 3, 3331, 1344),
           ("256x256", 3, 4500, 2, 6101, 2064), ("deep", 4, 512, 4, 1024, 1024), ("128x128", 4, 1024, 2, 4096, 256),
           ("256x128", 4, 1024, 4, 4096, 1152), ("256x256", 4, 2048, 4, 1024, 1152)]
# tile, M, N at the largest K
LARGEST = [("deep", 770, 1537), ("256x128", 2041, 4090), ("256x256", 3001, 4095)]
# tile, rows over 3 experts, N, K
OFFSETS = [("deep", 2000, 1100, 1040), ("128x128", 3000, 2100, 272), ("256x128", 2500, 2500, 1040),
           ("256x256", 4200, 2100, 1104)]


def load_choice():
    lib = ctypes.CDLL(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libint8_choice.so"))
    lib.int8_choice.argtypes = [ctypes.c_int64] * 4
    return lambda M, N, K, E=0: TILES[lib.int8_choice(M, N, K, E)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert binding().mxgemm_device_supported()
    yield


def _codes(g, *shape):
    return torch.empty(shape, dtype=torch.int8, device=DEV).random_(-128, 128, generator=g)


def _scales(g, *shape, by=1.0):
    return (torch.rand(shape, device=DEV, generator=g) + 0.5) / by


def _sums(a, w):
    return a.double() @ w.double().t()   # whole numbers below 2^53: exact


def _output(p, bias, act):
    """(result, tolerance of the fp32 evaluation) of products p in float64: three
    roundings of p, one of the sum with the bias; GELU with an erf good to
    1.5e-7 and 12 roundings of values of at most 1, its slope below 1.13."""
    y, tol = p, 3.01 * U * p.abs()
    if bias is not None:
        y = y + bias.double()
        tol = tol + 1.01 * U * y.abs()
    if act:
        gelu = 0.5 * y * torch.special.erfc(-y / math.sqrt(2.0))
        tol = 1.13 * tol + 0.5 * y.abs() * (1.5e-7 + 12 * U) + 2.01 * U * gelu.abs()
        y = gelu
    return y, tol


def _worst(got, want, tol, kind):
    """Largest error over its bound; the result's own rounding is half a step."""
    half = torch.finfo(TYPES[kind]).eps / 2
    bound = tol + half * (want.abs() + tol) + half * torch.finfo(TYPES[kind]).smallest_normal
    assert torch.isfinite(got).all()
    return float(((got.double() - want).abs() / bound).max())


@pytest.mark.parametrize("tile,M,N,K", DENSE)
def test_output_step(tile, M, N, K):
    """Bias, GELU and every type, on whole and on partial tiles."""
    say("large output step", tile, M, N, K)
    assert load_choice()(M, N, K) == tile
    b = binding()
    g = torch.Generator(device=DEV).manual_seed(M + N)
    a, w = _codes(g, M, K), _codes(g, N, K)
    a_s, w_s = _scales(g, M, by=128), _scales(g, N, by=64 * math.sqrt(K))
    bias = torch.randn(N, device=DEV, generator=g)
    p = _sums(a, w) * a_s.double()[:, None] * w_s.double()
    for bi, act in ((None, 0), (bias, 0), (None, 1), (bias, 1)):
        want, tol = _output(p, bi, act)
        for kind in (0, 1, 2):
            out = torch.full((M, N), float("nan"), dtype=TYPES[kind], device=DEV)
            poison_lds()
            b.int8gemm_run(a, a_s, w, w_s, bias=bi, act=b.ACT_GELU if act else b.ACT_NONE, out_type=kind, out=out)
            worst = _worst(out, want, tol, kind)
            say("  bias %d act %d type %d: error / bound %.3g" % (bi is not None, act, kind, worst))
            assert worst <= 1.0


@pytest.mark.parametrize("tile,E,tokens,div,N,K", EXPERTS)
def test_experts_output_step(tile, E, tokens, div, N, K):
    """By expert: gathered rows, some of them outside A, and sorted ones."""
    say("large experts", tile, E, tokens, div, N, K)
    rows = tokens * div
    assert load_choice()(rows, N, K, E) == tile
    b = binding()
    g = torch.Generator(device=DEV).manual_seed(rows + N)
    a, w = _codes(g, tokens, K), _codes(g, E, N, K)
    a_s, w_s = _scales(g, tokens, by=128), _scales(g, E, N, by=64 * math.sqrt(K))
    bias = torch.randn((E, N), device=DEV, generator=g)
    if N % 256 == 0:     # whole tiles
        edges = np.linspace(0, rows // 256, E + 1).astype(np.int64) * 256
    else:
        p = np.random.default_rng(rows).dirichlet(np.full(E, 0.7))
        edges = np.concatenate([[0], np.cumsum(np.random.default_rng(E).multinomial(rows - 5, p))])
    off = torch.tensor(edges, dtype=torch.int32, device=DEV)
    index = torch.randperm(rows, device=DEV, generator=g).int()
    bad = torch.tensor([0, 3, rows // 2, int(edges[-1]) - 1], device=DEV)
    index[bad] = torch.tensor([-1, rows, 2147483647, -2147483648], dtype=torch.int32, device=DEV)
    src = (index.long() // div).clamp(0, tokens - 1)
    good = torch.ones(rows, dtype=torch.bool, device=DEV)
    good[bad] = False
    owned = torch.arange(rows, device=DEV) < int(edges[-1])
    exact = torch.zeros((rows, N), dtype=torch.float64, device=DEV)
    each = torch.zeros((rows, N), dtype=torch.float64, device=DEV)
    for e in range(E):
        mine = slice(int(edges[e]), int(edges[e + 1]))
        exact[mine] = _sums(a[src[mine]], w[e]) * a_s[src[mine]].double()[:, None] * w_s[e].double()
        each[mine] = bias[e].double()
    for kind in (0, 1, 2):
        for bi, act in ((bias, 1), (None, 0)):
            want, tol = _output(exact, None if bi is None else each, act)
            out = torch.full((rows, N), 123.0, dtype=TYPES[kind], device=DEV)
            kw = dict(bias=bi, act=b.ACT_GELU if act else b.ACT_NONE, out_type=kind)
            poison_lds()
            b.int8gemm_run_grouped(a, a_s, w, w_s, off, index=index, index_div=div, out=out, **kw)
            assert torch.isnan(out[bad]).all() and (out[~owned] == 123.0).all()
            live = good & owned
            worst = _worst(out[live], want[live], tol[live], kind)
            say("  bias %d act %d type %d: error / bound %.3g" % (bi is not None, act, kind, worst))
            assert worst <= 1.0
            sorted_out = torch.full((rows, N), 123.0, dtype=TYPES[kind], device=DEV)
            poison_lds()
            b.int8gemm_run_grouped(a[src], a_s[src], w, w_s, off, out=sorted_out, **kw)
            assert torch.equal(sorted_out[live], out[live]) and (sorted_out[~owned] == 123.0).all()


@pytest.mark.parametrize("tile,M,N,K", DENSE)
def test_scale_values(tile, M, N, K):
    """A zero, an infinite and a NaN scale reach their row or column alone."""
    say("large scale values", tile, M, N, K)
    b = binding()
    g = torch.Generator(device=DEV).manual_seed(K)
    a, w = _codes(g, M, K), _codes(g, N, K)
    a_s, w_s = _scales(g, M), _scales(g, N)
    a_s[2], a_s[M - 1], a_s[M // 2] = 0.0, float("nan"), float("inf")
    w_s[7], w_s[N - 1], w_s[N // 2] = float("inf"), float("nan"), 0.0
    want = (_sums(a, w).float() * a_s[:, None]) * w_s    # the stated roundings, one by one
    got = b.int8gemm_run(a, a_s, w, w_s)
    assert ((got == want) | (torch.isnan(got) & torch.isnan(want))).all()


@pytest.mark.parametrize("tile,M,N", LARGEST)
@pytest.mark.parametrize("x,y", [(-128, -128), (127, -128)])
def test_largest_sums(tile, M, N, x, y):
    """Every product at its largest, at the largest K: the sum fills 32 bits."""
    say("large largest sums", tile, M, N, x, y)
    b = binding()
    K = b.INT8_MAX_K
    assert load_choice()(M, N, K) == tile
    out = b.int8gemm_run(torch.full((M, K), x, dtype=torch.int8, device=DEV), torch.ones(M, device=DEV),
                         torch.full((N, K), y, dtype=torch.int8, device=DEV), torch.ones(N, device=DEV))
    assert (out == float(np.float32(x * y * K))).all()


@pytest.mark.parametrize("tile,M,N,K", DENSE)
def test_every_tile_gives_the_same(tile, M, N, K):
    """The sums are exact, so whatever tiles two calls take, they agree bit for
    bit: the product at once, in few-row pieces, as one expert's, and over
    experts some of which have no rows."""
    say("every tile the same", tile, M, N, K)
    b = binding()
    g = torch.Generator(device=DEV).manual_seed(N)
    a, w = _codes(g, M, K), _codes(g, N, K)
    a_s, w_s, bias = _scales(g, M, by=128), _scales(g, N, by=64 * math.sqrt(K)), torch.randn(N, device=DEV, generator=g)
    E = 6
    many = [t.expand(E, *t.shape).contiguous() for t in (w, w_s, bias)]
    off = torch.tensor([0, 0, M // 3, M // 3, M - 1, M - 1, M], dtype=torch.int32, device=DEV)
    for kind in (0, 1, 2):
        kw = dict(act=b.ACT_GELU, out_type=kind)
        want = b.int8gemm_run(a, a_s, w, w_s, bias=bias, **kw)
        rows = slice(M // 2, M // 2 + 23)
        few = b.int8gemm_run(a[rows], a_s[rows], w, w_s, bias=bias, **kw)
        assert torch.equal(few, want[rows])
        one = torch.tensor([0, M], dtype=torch.int32, device=DEV)
        assert torch.equal(b.int8gemm_run_grouped(a, a_s, w[None], w_s[None], one, bias=bias[None], **kw), want)
        assert torch.equal(b.int8gemm_run_grouped(a, a_s, many[0], many[1], off, bias=many[2], **kw), want)


@pytest.mark.parametrize("tile,rows,N,K", OFFSETS)
@pytest.mark.parametrize("shape", ["front and behind", "falling", "outside", "all in the last"])
def test_offsets(tile, rows, N, K, shape):
    """Rows in front and behind left alone, offsets outside the rows and falling."""
    say("large offsets", tile, rows, N, K, shape)
    assert load_choice()(rows, N, K, 3) == tile
    b = binding()
    offsets = {"front and behind": (300, 300, 1500, 1700), "falling": (900, 200, 1300, 700),
               "outside": (-2147483648, 1200, 700, 2147483647), "all in the last": (0, 0, 0, rows)}[shape]
    g = torch.Generator(device=DEV).manual_seed(rows)
    a, w = _codes(g, rows, K), _codes(g, 3, N, K)
    a_s, w_s = _scales(g, rows), _scales(g, 3, N)
    out = torch.full((rows, N), 123.0, device=DEV)
    poison_lds()
    b.int8gemm_run_grouped(a, a_s, w, w_s, torch.tensor(offsets, dtype=torch.int32, device=DEV), out=out)
    edges = np.maximum.accumulate(np.clip(np.array(offsets, np.int64), 0, rows))
    assert (out[:edges[0]] == 123.0).all() and (out[edges[3]:] == 123.0).all()
    for e in range(3):
        mine = slice(int(edges[e]), int(edges[e + 1]))
        want = (_sums(a[mine], w[e]).float() * a_s[mine, None]) * w_s[e]
        assert torch.equal(out[mine], want), e
