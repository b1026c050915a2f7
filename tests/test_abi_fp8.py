"""Refusals of the fp8 and norm entry points that need no GPU (every call below
returns from argument validation, before the device is looked at), and the
64-bit forms that the GPU tests compare with."""
import os

import pytest
import torch

import fp8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x1000
OK, EINVAL, EALIGN = 0, 1, 2
NAMES = ("fp8gemm_quantize", "fp8gemm_run", "fp8gemm_run_grouped", "fp8gemm_weight_grad", "fp8gemm_weight_grad_grouped",
         "rmsnorm_quantize", "rmsnorm_backward")


@pytest.fixture(scope="module")
def lib():
    from block_scaled_precision_mxgemm_amd import mxgemm

    return mxgemm.raw_library()


def test_exports(lib):
    header = open(os.path.join(ROOT, "include", "mxgemm.h")).read()
    for name in NAMES + ("fp8gemm_weight_grad_workspace", "rmsnorm_backward_workspace"):
        assert hasattr(lib, name), name
        assert name + "(" in header


def test_package_names():
    import block_scaled_precision_mxgemm_amd as pkg

    for name in NAMES + ("QUANT_NONE", "QUANT_INT8", "QUANT_FP8", "QUANT_FP8_POW2", "QUANT_MXFP8"):
        assert getattr(pkg, name) is not None


@pytest.mark.parametrize("change,want", [
    (dict(X=None), EINVAL), (dict(Q=None), EINVAL), (dict(S=None), EINVAL), (dict(kind=3), EINVAL), (dict(E=0), EINVAL),
    (dict(E=1025), EINVAL), (dict(rows=0), EINVAL), (dict(K=24), EINVAL), (dict(K=0), EINVAL), (dict(K=(1 << 20) + 16), EINVAL),
    (dict(br=64), EINVAL), (dict(br=0), EINVAL), (dict(pow2=2), EINVAL), (dict(rows=(64 << 20) + 1), EINVAL),
    (dict(rows=32 << 20, E=3), EINVAL), (dict(rows=(1 << 20) + 1, br=128), EINVAL), (dict(rows=64 << 20, S=A + 2), EALIGN),
    (dict(X=A + 8), EALIGN), (dict(Q=A + 4), EALIGN), (dict(S=A + 1), EALIGN)])
def test_quantize(lib, change, want):
    p = dict(X=A, kind=0, E=1, rows=4, K=64, br=1, pow2=0, Q=A, S=A) | change
    assert lib.fp8gemm_quantize(p["X"], p["kind"], p["E"], p["rows"], p["K"], p["br"], p["pow2"], p["Q"], p["S"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(A=None), EINVAL), (dict(SA=None), EINVAL), (dict(B=None), EINVAL), (dict(SB=None), EINVAL), (dict(C=None), EINVAL),
    (dict(M=0), EINVAL), (dict(N=-1), EINVAL), (dict(K=40), EINVAL), (dict(K=(1 << 20) + 16), EINVAL), (dict(act=2), EINVAL),
    (dict(out=3), EINVAL), (dict(A=A + 8), EALIGN), (dict(B=A + 1), EALIGN), (dict(C=A + 4), EALIGN), (dict(SA=A + 2), EALIGN),
    (dict(SB=A + 1), EALIGN), (dict(bias=A + 4), EALIGN)])
def test_run(lib, change, want):
    p = dict(A=A, SA=A, B=A, SB=A, C=A, M=4, N=4, K=64, bias=None, act=0, out=0) | change
    assert lib.fp8gemm_run(p["A"], p["SA"], p["B"], p["SB"], p["C"], p["M"], p["N"], p["K"], p["bias"], p["act"], p["out"],
                           None) == want


EXPERTS = [(dict(off=None), EINVAL), (dict(rows=0), EINVAL), (dict(rows=(64 << 20) + 1, rowsA=64 << 20), EINVAL),
           (dict(rowsA=0), EINVAL), (dict(rowsA=7), EINVAL), (dict(E=0), EINVAL), (dict(E=1025), EINVAL),
           (dict(index=A, div=0), EINVAL), (dict(K=8), EINVAL), (dict(N=0), EINVAL), (dict(off=A + 2), EALIGN),
           (dict(index=A + 1), EALIGN), (dict(SA=A + 2), EALIGN)]


@pytest.mark.parametrize("change,want", EXPERTS)
def test_run_grouped(lib, change, want):
    p = dict(A=A, SA=A, rowsA=8, rows=8, N=4, K=64, E=2, off=A, index=None, div=1) | change
    assert lib.fp8gemm_run_grouped(p["A"], p["SA"], p["rowsA"], A, A, A, p["rows"], p["N"], p["K"], p["E"], p["off"],
                                   p["index"], p["div"], None, 0, 0, None) == want


@pytest.mark.parametrize("change,want", EXPERTS + [(dict(kind=3), EINVAL), (dict(out=-1), EINVAL), (dict(dC=None), EINVAL),
                                                   (dict(dW=None), EINVAL), (dict(dC=A + 8), EALIGN), (dict(dW=A + 4), EALIGN)])
def test_weight_grad_grouped(lib, change, want):
    p = dict(dC=A, kind=1, rows=8, N=4, A=A, SA=A, rowsA=8, K=64, E=2, off=A, index=None, div=1, dW=A, out=0) | change
    assert lib.fp8gemm_weight_grad_grouped(p["dC"], p["kind"], p["rows"], p["N"], p["A"], p["SA"], p["rowsA"], p["K"], p["E"],
                                           p["off"], p["index"], p["div"], p["dW"], p["out"], A, None) == want


@pytest.mark.parametrize("change,want", [
    (dict(dC=None), EINVAL), (dict(A=None), EINVAL), (dict(SA=None), EINVAL), (dict(dW=None), EINVAL), (dict(kind=-1), EINVAL),
    (dict(out=3), EINVAL), (dict(M=0), EINVAL), (dict(M=(64 << 20) + 1), EINVAL), (dict(N=0), EINVAL), (dict(K=24), EINVAL),
    (dict(dC=A + 2), EALIGN), (dict(A=A + 8), EALIGN), (dict(SA=A + 1), EALIGN), (dict(dW=A + 8), EALIGN),
    (dict(ws=A + 4), EALIGN)])
def test_weight_grad(lib, change, want):
    p = dict(dC=A, kind=1, M=8, N=4, A=A, SA=A, K=64, dW=A, out=0, ws=A) | change
    assert lib.fp8gemm_weight_grad(p["dC"], p["kind"], p["M"], p["N"], p["A"], p["SA"], p["K"], p["dW"], p["out"], p["ws"],
                                   None) == want


def test_workspaces(lib):
    assert lib.fp8gemm_weight_grad_workspace(0, 4, 64, 1) == -1
    assert lib.fp8gemm_weight_grad_workspace(8, 4, 24, 1) == -1
    assert lib.fp8gemm_weight_grad_workspace(8, 4, 64, 1025) == -1
    assert lib.fp8gemm_weight_grad_workspace(8, 4, 64, 1) >= 0
    assert lib.fp8gemm_weight_grad_workspace(64 << 20, 1 << 20, 1 << 20, 1) >= 0
    assert lib.rmsnorm_backward_workspace(0, 64) == -1
    assert lib.rmsnorm_backward_workspace(4, 24) == -1
    assert lib.rmsnorm_backward_workspace(4, 64) >= 0
    assert lib.rmsnorm_backward_workspace(1000, 4096) > 0


@pytest.mark.parametrize("change,want", [
    (dict(X=None), EINVAL), (dict(W=None), EINVAL), (dict(kind=3), EINVAL), (dict(wkind=-1), EINVAL), (dict(rows=0), EINVAL),
    (dict(rows=(64 << 20) + 1), EINVAL), (dict(K=24), EINVAL), (dict(K=48, quant=4), EINVAL), (dict(eps=-1.0), EINVAL),
    (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL), (dict(R=None), EINVAL), (dict(H=None), EINVAL),
    (dict(quant=5), EINVAL), (dict(quant=-1), EINVAL), (dict(Q=None), EINVAL), (dict(S=None), EINVAL), (dict(quant=0), EINVAL),
    (dict(quant=0, Q=None, S=None, Y=None), EINVAL), (dict(X=A + 8), EALIGN), (dict(R=A + 8), EALIGN), (dict(W=A + 4), EALIGN),
    (dict(H=A + 8), EALIGN), (dict(Y=A + 2), EALIGN), (dict(Q=A + 4), EALIGN), (dict(S=A + 2), EALIGN), (dict(rstd=A + 2), EALIGN)])
def test_norm(lib, change, want):
    p = dict(X=A, R=A, kind=1, W=A, wkind=0, rows=4, K=64, eps=1e-6, H=A, Y=A, quant=2, Q=A, S=A, rstd=A) | change
    assert lib.rmsnorm_quantize(p["X"], p["R"], p["kind"], p["W"], p["wkind"], p["rows"], p["K"], p["eps"], p["H"], p["Y"],
                                p["quant"], p["Q"], p["S"], p["rstd"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(dY=None), EINVAL), (dict(H=None), EINVAL), (dict(W=None), EINVAL), (dict(rstd=None), EINVAL), (dict(dX=None), EINVAL),
    (dict(dW=None), EINVAL), (dict(ws=None), EINVAL), (dict(kind=4), EINVAL), (dict(wkind=3), EINVAL), (dict(rows=0), EINVAL),
    (dict(K=20), EINVAL), (dict(dY=A + 8), EALIGN), (dict(H=A + 8), EALIGN), (dict(dH=A + 8), EALIGN), (dict(W=A + 8), EALIGN),
    (dict(rstd=A + 2), EALIGN), (dict(dX=A + 8), EALIGN), (dict(dW=A + 8), EALIGN), (dict(ws=A + 8), EALIGN)])
def test_norm_backward(lib, change, want):
    p = dict(dY=A, H=A, dH=None, kind=1, W=A, wkind=0, rstd=A, rows=1000, K=4096, dX=A, dW=A, ws=A) | change
    assert lib.rmsnorm_backward(p["dY"], p["H"], p["dH"], p["kind"], p["W"], p["wkind"], p["rstd"], p["rows"], p["K"], p["dX"],
                                p["dW"], p["ws"], None) == want


def test_binding_refuses_host_tensors():
    from block_scaled_precision_mxgemm_amd import mxgemm as mx

    x, w = torch.zeros((4, 64)), torch.zeros(64)
    q, s, i = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 1)), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: mx.fp8gemm_quantize(x), lambda: mx.fp8gemm_run(q, s, q, s[:1]),
                 lambda: mx.fp8gemm_run_grouped(q, s, q[None], s[None, :1], i), lambda: mx.fp8gemm_weight_grad(x, q, s),
                 lambda: mx.fp8gemm_weight_grad_grouped(x, q, s, i), lambda: mx.rmsnorm_quantize(x, w),
                 lambda: mx.rmsnorm_backward(x, x, w, w[:4])):
        with pytest.raises(ValueError, match="must be a GPU tensor"):
            call()


# ---- the forms that the GPU tests compare with --------------------------------


def test_reference_codes():
    """Every value has its code, every middle of two the even one."""
    v = ref.values()
    codes = torch.arange(127, dtype=torch.uint8)
    assert v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[126] == 448.0
    assert torch.equal(ref.encode(v), codes) and torch.equal(ref.encode(-v), codes | 128)
    middle = (v[1:] + v[:-1]) / 2
    low = codes[:126]
    even = torch.where(low % 2 == 0, low, low + 1)
    assert torch.equal(ref.encode(middle), even)
    assert torch.equal(ref.encode(middle * (1 - 1e-12)), low) and torch.equal(ref.encode(middle * (1 + 1e-12)), low + 1)
    assert ref.encode(torch.tensor([1e9], dtype=torch.float64))[0] == 126
    x = torch.linspace(-460, 460, 20001)
    assert torch.equal(ref.encode(x.double()), x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    assert torch.equal(ref.decode(codes), v) and torch.isnan(ref.decode(torch.tensor([127, 255], dtype=torch.uint8))).all()


def test_reference_scales():
    x = torch.zeros(2, 160)
    x[0, 0], x[0, 130], x[1, 3] = 448.0, 1.0, float("inf")
    q, s = ref.quantize(x)
    assert s[0, 0] == 1.0 and s[0, 1] == torch.tensor(1.0) / 448.0 and torch.isnan(s[1, 0]) and s[1, 1] == 0
    assert q[0, 0] == 126 and q[0, 130] == 126 and not q[1].any()
    _, s = ref.quantize(x[:1], pow2=True)
    assert s[0, 0] == 1.0 and s[0, 1] == 2.0 ** -8   # 1 / 448 lies between 2^-9 and 2^-8
    _, s = ref.quantize(torch.full((1, 16), 2.0 ** -140))
    assert s[0, 0] == 2.0 ** -126


def test_reference_norm_gradient_against_differences():
    """Central differences with h = 1e-6: h^2 times a third derivative below 100,
    rounding 1e-15 / h."""
    g = torch.Generator().manual_seed(0)
    x, w, dy, dh = (torch.randn(n, generator=g, dtype=torch.float64) for n in ((3, 16), (16,), (3, 16), (3, 16)))

    def loss(x, w):
        return (ref.norm(x, w, 1e-3)[1] * dy).sum() + (x * dh).sum()

    dx, dw = ref.norm_backward(dy, x, w, 1e-3, dh)
    step = 1e-6
    for i in range(3):
        for j in range(16):
            d = torch.zeros_like(x)
            d[i, j] = step
            assert dx[i, j].item() == pytest.approx(((loss(x + d, w) - loss(x - d, w)) / (2 * step)).item(), abs=1e-7)
    for j in range(16):
        d = torch.zeros_like(w)
        d[j] = step
        assert dw[j].item() == pytest.approx(((loss(x, w + d) - loss(x, w - d)) / (2 * step)).item(), abs=1e-7)


def test_reference_weight_gradient_against_differences():
    """The product is linear in the weights: differences of any size, rounding alone."""
    g = torch.Generator().manual_seed(1)
    q, s = ref.quantize(torch.randn(5, 32, generator=g), pow2=True)
    x = ref.dequantize(q, s)
    w, d = torch.randn(4, 32, generator=g, dtype=torch.float64), torch.randn(5, 4, generator=g).double()
    dw, _ = ref.bf16_grad(d, x)
    for n in range(4):
        for k in range(32):
            e = torch.zeros_like(w)
            e[n, k] = 1.0
            assert dw[n, k].item() == pytest.approx(((x @ (w + e).t() * d).sum() - (x @ (w - e).t() * d).sum()).item() / 2, abs=1e-12)


def test_reference_expert_ranges():
    assert ref.rows_of_experts([-3, 2, 1, 99, 5], 8) == [(0, 2), (2, 2), (2, 8), (8, 8)]


# ---- which tile the GPU tests' sizes take ---------------------------------------


def test_large_tile_cases_take_their_tiles():
    import test_gpu_fp8_large as large

    chosen = large.load_choice()
    for tile, M, N, K in large.DENSE:
        assert chosen(M, N, K) == tile
    for tile, E, tokens, k, N, K in large.EXPERTS:
        assert chosen(tokens * k, N, K, E) == tile
    for tile, rows, N, K in large.OFFSETS:
        assert chosen(rows, N, K, 3) == tile
    for cases, E in ((large.BLOCKS, 0), (large.BLOCKS_EXPERTS, 1)):
        for tile, M, N in cases:
            assert all(chosen(M, N, 128 * n - short, E) == tile for n in range(1, 7) for short in (0, 48, 96))
    assert {c[0] for c in large.DENSE} == set(large.TILES)


def test_gradient_cases_take_every_form():
    """Large tiles, small ones, and rows in parts, with dY in one and two terms."""
    import ctypes

    import test_gpu_fp8_grad as grad

    lib = ctypes.CDLL(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libfp8_choice.so"))
    lib.fp8_grad_choice.argtypes = [ctypes.c_int64] * 4 + [ctypes.c_int]
    for terms in (1, 2):
        taken = {lib.fp8_grad_choice(M, N, K, 1, terms) for M, N, K in grad.SIZES}
        assert {0, 1} <= taken and len(taken) >= 4
        taken = {lib.fp8_grad_choice(t * k, N, K, E, terms) for E, t, k, N, K in grad.EXPERTS}
        assert {0, 1} <= taken and len(taken) >= 3
