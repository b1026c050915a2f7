"""E4M3 products on every tile: tile after tile with any number of blocks, output
step, experts' rows, and the agreement of all tiles; sums that are exact in any
order, so that results are compared bit for bit.

Each case names the tile that it is there for; the library's own choice says
that it takes it (test_abi_fp8.py checks the same without a GPU)."""
import ctypes
import os

import pytest
import torch

import fp8_ref as ref
from gpu_util import binding, poison_lds, say
from test_gpu_fp8 import DEV, TYPES, exact_codes, expert_result, gen, randn, result_tol

pytestmark = pytest.mark.gpu

# variants in the order of csrc/fp8_choice.h; "deep" is 128 x 128 with 8 waves
TILES = ["16x16", "16x32", "32x32", "32x64", "deep", "128x128", "256x128", "256x256", "64x128"]
# tile, M, N: more tiles than run at once, for 1 .. 6 blocks of K
BLOCKS = [("64x128", 1025, 7174), ("128x128", 2049, 7174), ("256x128", 7174, 2050), ("256x256", 2690, 8836)]
# the same over experts, the most rows with one
BLOCKS_EXPERTS = [("64x128", 385, 8640), ("64x128", 449, 8640), ("128x128", 897, 8616), ("256x128", 769, 8698),
                  ("256x256", 1795, 8499)]
# tile, M, N, K: ragged in every size, then whole tiles
DENSE = [("16x16", 9, 4000, 4000), ("16x32", 13, 14000, 1040), ("32x32", 60, 4090, 4112), ("32x64", 61, 14003, 2064),
         ("deep", 1939, 2046, 1776), ("128x128", 384, 20000, 528), ("256x128", 2050, 8203, 2000),
         ("256x256", 5000, 9001, 1104), ("64x128", 2048, 2048, 1040), ("64x128", 1001, 2046, 2064),
         ("deep", 2048, 2048, 2064), ("256x128", 2048, 4096, 1152),
         ("256x256", 4096, 4096, 1024)]
# tile, experts, tokens, choices, N, K
EXPERTS = [("64x128", 3, 500, 2, 1100, 1040), ("deep", 3, 500, 2, 2100, 2064),
           ("128x128", 64, 225, 4, 1101, 2064), ("256x128", 2, 2949, 2, 3331, 1344),
           ("256x256", 3, 4500, 2, 6101, 2064), ("64x128", 4, 512, 4, 1024, 1024), ("deep", 4, 512, 4, 1536, 2048),
           ("256x128", 4, 1024, 4, 4096, 1152),
           ("256x256", 4, 2048, 4, 1024, 1152)]
# tile, rows over 3 experts, N, K
OFFSETS = [("64x128", 2000, 1100, 1040), ("deep", 2000, 1500, 2064), ("128x128", 600, 8600, 400), ("256x128", 2500, 2500, 1040),
           ("256x256", 4200, 2100, 1104)]


def load_choice():
    lib = ctypes.CDLL(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libfp8_choice.so"))
    lib.fp8_choice.argtypes = [ctypes.c_int64] * 4
    return lambda M, N, K, E=0: TILES[lib.fp8_choice(M, N, K, E)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert binding().mxgemm_device_supported()
    yield


def values(q, s, block_rows=1):
    """The dequantized values in fp32: exact, and so are sums of products of them here."""
    return ref.dequantize(q, s, block_rows).float()


@pytest.mark.parametrize("tile,M,N", BLOCKS)
@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 6])
@pytest.mark.parametrize("short", [0, 48, 96])
def test_blocks(tile, M, N, blocks, short):
    """Every way that the copies of one tile meet those of the next, and partial
    last blocks."""
    say("fp8 large blocks", tile, M, N, blocks, short)
    K = 128 * blocks - short
    assert load_choice()(M, N, K) == tile
    g = gen(blocks + short)
    a, a_s = exact_codes(g, M, K)
    b, b_s = exact_codes(g, N, K, 128)
    poison_lds()
    got = binding().fp8gemm_run(a, a_s, b, b_s)
    assert torch.equal(got, (ref.dequantize(a, a_s) @ ref.dequantize(b, b_s, 128).t()).float())


@pytest.mark.parametrize("tile,M,N", BLOCKS_EXPERTS)
@pytest.mark.parametrize("blocks", [1, 2, 3, 5])
@pytest.mark.parametrize("short", [0, 48])
def test_blocks_experts(tile, M, N, blocks, short):
    say("fp8 large blocks by index", tile, M, N, blocks, short)
    K = 128 * blocks - short
    assert load_choice()(M, N, K, 1) == tile
    g = gen(blocks + short)
    a, a_s = exact_codes(g, M // 2, K)
    b, b_s = exact_codes(g, N, K, 128)
    index = torch.randint(0, 2 * (M // 2), (M,), generator=g, device=DEV).int()
    off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    poison_lds()
    got = binding().fp8gemm_run_grouped(a, a_s, b[None], b_s[None], off, index=index, index_div=2)
    assert torch.equal(got.double(), expert_result(a, a_s, b[None], b_s[None], off, index, 2, M))


@pytest.mark.parametrize("tile,M,N,K", DENSE)
def test_every_tile_gives_the_same(tile, M, N, K):
    """The product at once, in few-row pieces, as one expert's, and over experts some
    of which have no rows, with bias, activation and each type."""
    say("fp8 large every tile the same", tile, M, N, K)
    bn = binding()
    assert load_choice()(M, N, K) == tile
    g = gen(N)
    a, a_s = exact_codes(g, M, K)
    b, b_s = exact_codes(g, N, K, 128)
    bias = randn(g, N)
    y = ref.dequantize(a, a_s) @ ref.dequantize(b, b_s, 128).t()
    assert torch.equal(bn.fp8gemm_run(a, a_s, b, b_s), y.float())
    many = [t.expand(6, *t.shape).contiguous() for t in (b, b_s, bias)]
    off = torch.tensor([0, 0, M // 3, M // 3, M - 1, M - 1, M], dtype=torch.int32, device=DEV)
    one = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    rows = slice(M // 2, M // 2 + 23)
    for kind in (0, 1, 2):
        kw = dict(act=bn.ACT_GELU, out_type=kind)
        poison_lds()
        want = bn.fp8gemm_run(a, a_s, b, b_s, bias=bias, **kw)
        t = y + bias.double()
        tol = result_tol(t, torch.zeros_like(t), True, TYPES[kind])
        assert bool(((want.double() - ref.gelu(t)).abs() <= tol).all())
        assert torch.equal(bn.fp8gemm_run(a[rows], a_s[rows], b, b_s, bias=bias, **kw), want[rows])
        assert torch.equal(bn.fp8gemm_run_grouped(a, a_s, b[None], b_s[None], one, bias=bias[None], **kw), want)
        assert torch.equal(bn.fp8gemm_run_grouped(a, a_s, many[0], many[1], off, bias=many[2], **kw), want)
        assert torch.equal(bn.fp8gemm_run(a, a_s, b, b_s, out_type=kind), y.to(TYPES[kind]))


@pytest.mark.parametrize("tile,E,tokens,k,N,K", EXPERTS)
def test_experts(tile, E, tokens, k, N, K):
    say("fp8 large experts", tile, E, tokens, k, N, K)
    bn = binding()
    assert load_choice()(tokens * k, N, K, E) == tile
    g = gen(E + N)
    a, a_s = exact_codes(g, tokens, K)
    w = [exact_codes(g, N, K, 128) for _ in range(E)]
    b, b_s = torch.stack([x[0] for x in w]), torch.stack([x[1] for x in w])
    ids = torch.rand(tokens, E, generator=g, device=DEV).topk(k, 1).indices.int()
    offsets, order, _ = bn.expert_plan(ids, E)
    poison_lds()
    got = bn.fp8gemm_run_grouped(a, a_s, b, b_s, offsets, index=order, index_div=k, out_type=1)
    want = expert_result(a, a_s, b, b_s, offsets, order, k, tokens * k)
    assert torch.equal(got, want.float().bfloat16())
    at = (order // k).long()
    assert torch.equal(bn.fp8gemm_run_grouped(a[at], a_s[at], b, b_s, offsets).double(), want)


@pytest.mark.parametrize("tile,rows,N,K", OFFSETS)
@pytest.mark.parametrize("shape", ["front and behind", "falling", "outside", "all in the last", "none"])
def test_offsets(tile, rows, N, K, shape):
    """Rows that no expert has are left as they were; indices outside A give NaN."""
    say("fp8 large offsets", tile, rows, N, K, shape)
    assert load_choice()(rows, N, K, 3) == tile
    g = gen(rows)
    T = 500
    a, a_s = exact_codes(g, T, K)
    w = [exact_codes(g, N, K, 128) for _ in range(3)]
    b, b_s = torch.stack([x[0] for x in w]), torch.stack([x[1] for x in w])
    index = torch.randint(0, 3 * T, (rows,), generator=g, device=DEV).int()
    index[7], index[300], index[rows - 100] = -1, 3 * T, -2 ** 31
    offsets = {"front and behind": [130, 400, 401, rows - 90], "falling": [0, rows // 2, 40, rows - 5],
               "outside": [-9, 100, 2 ** 31 - 1, 5], "all in the last": [0, 0, 0, rows], "none": [rows] * 4}[shape]
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    for kind in (0, 1):
        out = torch.full((rows, N), -7.0, dtype=TYPES[kind], device=DEV)
        poison_lds()
        binding().fp8gemm_run_grouped(a, a_s, b, b_s, off, index=index, index_div=3, out=out, out_type=kind)
        want = expert_result(a, a_s, b, b_s, off, index, 3, rows).to(TYPES[kind])
        inside = torch.zeros(rows, dtype=torch.bool, device=DEV)
        for lo, hi in ref.rows_of_experts(offsets, rows):
            inside[lo:hi] = True
        assert bool((out[~inside] == -7.0).all())
        assert torch.equal(out[inside].nan_to_num(-9.0), want[inside].nan_to_num(-9.0))


@pytest.mark.parametrize("M,N", [(4096, 4096), (300, 700), (17, 260)])
def test_specials_reach_their_rows(M, N):
    """NaN codes and scales in the last block, in whole tiles too."""
    say("fp8 large specials", M, N)
    K = 400
    g = gen(M)
    a, a_s = exact_codes(g, M, K)
    b, b_s = exact_codes(g, N, K, 128)
    a[3, 399], b[5, 390] = 0x7F, 0xFF
    a_s[7, 3], b_s[1, 0] = float("nan"), float("nan")
    y = ref.dequantize(a, a_s) @ ref.dequantize(b, b_s, 128).t()
    got = binding().fp8gemm_run(a, a_s, b, b_s).double()
    assert torch.equal(torch.isnan(got), torch.isnan(y))
    ok = ~torch.isnan(y)
    assert torch.equal(got[ok], y[ok])


def test_streams_and_replays_of_large_tiles():
    say("fp8 large streams and replays")
    bn = binding()
    g = gen(5)
    sets = []
    for M, N, K in ((4096, 4096, 512), (2690, 8836, 272), (2048, 2048, 1040), (7174, 2050, 384)):
        a, a_s = exact_codes(g, M, K)
        b, b_s = exact_codes(g, N, K, 128)
        sets.append((a, a_s, b, b_s))
    want = [bn.fp8gemm_run(*s) for s in sets]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [bn.fp8gemm_run(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for h in held:
            h.zero_()
        graph.replay()
        got = [bn.fp8gemm_run(*s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, want))
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_millions_of_tiles():
    """1000 rows over 1024 experts of 2^20 x 16."""
    say("fp8 large many tiles")
    E, N, K, M = 1024, 1 << 20, 16, 1000
    assert load_choice()(M, N, K, E) == "64x128"
    g = gen(11)
    a, a_s = exact_codes(g, M, K)
    b = torch.randint(0x30, 0x40, (E, N, K), generator=g, device=DEV, dtype=torch.uint8)  # 0.5 .. 1.875
    b_s = torch.exp2(torch.randint(-2, 3, (E, N // 128, 1), generator=g, device=DEV).float())
    expert = torch.randint(0, E, (M,), generator=g, device=DEV).sort()[0]
    off = torch.searchsorted(expert, torch.arange(E + 1, device=DEV)).int()
    got = binding().fp8gemm_run_grouped(a, a_s, b, b_s, off, out_type=1)
    for p in (0, 1, 333, 500, 998, 999):
        e = int(expert[p])
        y = ref.dequantize(b[e], b_s[e], 128) @ ref.dequantize(a[p:p + 1], a_s[p:p + 1])[0]
        assert torch.equal(got[p], y.float().bfloat16())
    assert bool(torch.isfinite(got).all()) and int((got == 0).all(-1).sum()) == 0


@pytest.mark.parametrize("tile,M,N,K", [("256x128", 2 ** 20, 300, 4224), ("16x32", 16, 2 ** 20, 4224), ("256x256", 2 ** 17 + 9, 20000, 400)])
def test_operands_past_4_gib(tile, M, N, K):
    """A, B and C of more than 4 GiB."""
    say("fp8 large past 4 GiB", tile, M, N, K)
    assert load_choice()(M, N, K) == tile
    g = gen(K + N)

    def operand(rows, block_rows):
        q = torch.randint(0, 4, (rows, K), generator=g, device=DEV, dtype=torch.uint8).mul_(4).add_(0x30)   # 0.5 .. 1.5
        s = torch.exp2(torch.randint(0, 2, (-(-rows // block_rows), -(-K // 128)), generator=g, device=DEV).float())
        return q, s

    (a, a_s), (b, b_s) = operand(M, 1), operand(N, 128)
    got = binding().fp8gemm_run(a, a_s, b, b_s, out_type=1)
    # sums of multiples of 1 / 16 below 2^16: exact in fp32
    rows = torch.tensor([0, M // 2 + 1, M - 2, M - 1], device=DEV)
    for n0 in sorted({0, max(0, N // 256 * 128 - 128), (N - 1) // 128 * 128}):
        cols = slice(n0, min(n0 + 128, N))
        want = ref.dequantize(a[rows], a_s[rows]) @ ref.dequantize(b[cols], b_s[n0 // 128:n0 // 128 + 1], 128).t()
        assert torch.equal(got[rows, cols], want.float().bfloat16())
    assert bool(torch.isfinite(got).all()) and not bool((got == 0).any())
