"""Refusals of the int8 and expert entry points that need no GPU: every call
below returns from argument validation, before the device is looked at."""
import ctypes
import os

import pytest
import torch

import experts_ref as ref
import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x1000
OK, EINVAL, EALIGN = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from block_scaled_precision_mxgemm_amd import mxgemm

    return mxgemm.raw_library()


def test_exports(lib):
    for name in ("int8gemm_quantize", "int8gemm_run", "int8gemm_run_grouped", "expert_route", "expert_route_backward",
                 "expert_plan", "expert_plan_workspace", "expert_combine", "expert_combine_backward"):
        assert hasattr(lib, name), name
        assert name + "(" in open(os.path.join(ROOT, "include", "mxgemm.h")).read()


def test_alignment_status_names_both_kinds(lib):
    """Data is aligned to 16 bytes, but a scale or an index to its element: the text does not call that data."""
    text = lib.mxgemm_status_string(EALIGN)
    assert b"16 bytes" in text and b"element" in text


def test_package_names():
    import block_scaled_precision_mxgemm_amd as pkg

    for name in ("int8gemm_quantize", "int8gemm_run", "int8gemm_run_grouped", "expert_route", "expert_route_backward",
                 "expert_plan", "expert_combine", "expert_combine_backward", "SCORE_SOFTMAX", "SCORE_SIGMOID", "INT8_MAX_K"):
        assert getattr(pkg, name) is not None


@pytest.mark.parametrize("change,want", [
    (dict(X=None), EINVAL), (dict(Q=None), EINVAL), (dict(S=None), EINVAL), (dict(kind=3), EINVAL), (dict(rows=0), EINVAL),
    (dict(K=0), EINVAL), (dict(K=24), EINVAL), (dict(K=(1 << 20) + 16), EINVAL), (dict(X=A + 4), EALIGN),
    (dict(Q=A + 8), EALIGN), (dict(S=A + 2), EALIGN)])
def test_quantize(lib, change, want):
    p = dict(X=A, kind=0, rows=4, K=64, Q=A, S=A) | change
    assert lib.int8gemm_quantize(p["X"], p["kind"], p["rows"], p["K"], p["Q"], p["S"], None) == want


@pytest.mark.parametrize("rows,want", [((1 << 20) + 1, EALIGN), (64 << 20, EALIGN), ((64 << 20) + 1, EINVAL)])
def test_quantize_rows(lib, rows, want):
    """As many rows as the experts' products have (a misaligned S ends the call behind that check)."""
    assert lib.int8gemm_quantize(A, 0, rows, 64, A, A + 2, None) == want


@pytest.mark.parametrize("change,want", [
    (dict(A=None), EINVAL), (dict(SA=None), EINVAL), (dict(B=None), EINVAL), (dict(SB=None), EINVAL), (dict(C=None), EINVAL),
    (dict(M=0), EINVAL), (dict(N=-1), EINVAL), (dict(K=40), EINVAL), (dict(K=131072), EINVAL), (dict(act=2), EINVAL),
    (dict(out=3), EINVAL), (dict(A=A + 8), EALIGN), (dict(B=A + 1), EALIGN), (dict(C=A + 4), EALIGN), (dict(SA=A + 2), EALIGN),
    (dict(SB=A + 4), EALIGN), (dict(bias=A + 4), EALIGN)])
def test_run(lib, change, want):
    p = dict(A=A, SA=A, B=A, SB=A, C=A, M=4, N=4, K=64, bias=None, act=0, out=0) | change
    assert lib.int8gemm_run(p["A"], p["SA"], p["B"], p["SB"], p["C"], p["M"], p["N"], p["K"], p["bias"], p["act"], p["out"],
                            None) == want


@pytest.mark.parametrize("change,want", [
    (dict(off=None), EINVAL), (dict(rows=0), EINVAL), (dict(rows=(64 << 20) + 1, rowsA=64 << 20), EINVAL), (dict(rowsA=0), EINVAL),
    (dict(rowsA=7), EINVAL), (dict(E=0), EINVAL), (dict(E=1025), EINVAL), (dict(index=A, div=0), EINVAL), (dict(K=8), EINVAL),
    (dict(off=A + 2), EALIGN), (dict(index=A + 1), EALIGN), (dict(SB=A + 8), EALIGN)])
def test_run_grouped(lib, change, want):
    p = dict(A=A, SA=A, rowsA=8, B=A, SB=A, C=A, rows=8, N=4, K=64, E=2, off=A, index=None, div=1) | change
    assert lib.int8gemm_run_grouped(p["A"], p["SA"], p["rowsA"], p["B"], p["SB"], p["C"], p["rows"], p["N"], p["K"], p["E"],
                                    p["off"], p["index"], p["div"], None, 0, 0, None) == want


@pytest.mark.parametrize("change,want", [
    (dict(l=None), EINVAL), (dict(ids=None), EINVAL), (dict(w=None), EINVAL), (dict(kind=-1), EINVAL), (dict(T=0), EINVAL),
    (dict(E=0, k=1), EINVAL), (dict(E=1025), EINVAL), (dict(k=0), EINVAL), (dict(k=17), EINVAL), (dict(E=128, k=65), EINVAL),
    (dict(score=2), EINVAL), (dict(groups=3), EINVAL), (dict(groups=0), EINVAL), (dict(E=130, groups=65), EINVAL),
    (dict(groups=4, top=5), EINVAL), (dict(groups=4, top=0), EINVAL), (dict(group_top=3), EINVAL), (dict(renorm=2), EINVAL),
    (dict(groups=8, top=1, k=3), EINVAL), (dict(l=A + 2), EALIGN), (dict(bias=A + 1), EALIGN), (dict(ids=A + 2), EALIGN),
    (dict(w=A + 3), EALIGN), (dict(kind=1, l=A + 1), EALIGN)])
def test_route(lib, change, want):
    p = dict(l=A, kind=0, T=4, E=16, k=2, score=0, bias=None, groups=1, top=1, group_top=1, renorm=1, ids=A, w=A) | change
    assert lib.expert_route(p["l"], p["kind"], p["T"], p["E"], p["k"], p["score"], p["bias"], p["groups"], p["top"],
                            p["group_top"], p["renorm"], 1.0, p["ids"], p["w"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(l=None), EINVAL), (dict(ids=None), EINVAL), (dict(dw=None), EINVAL), (dict(dl=None), EINVAL), (dict(kind=3), EINVAL),
    (dict(k=17), EINVAL), (dict(score=-1), EINVAL), (dict(renorm=-1), EINVAL), (dict(ids=A + 1), EALIGN), (dict(dl=A + 2), EALIGN)])
def test_route_backward(lib, change, want):
    p = dict(l=A, kind=0, T=4, E=16, ids=A, dw=A, k=2, score=0, renorm=1, dl=A) | change
    assert lib.expert_route_backward(p["l"], p["kind"], p["T"], p["E"], p["ids"], p["dw"], p["k"], p["score"], p["renorm"], 1.0,
                                     p["dl"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(ids=None), EINVAL), (dict(off=None), EINVAL), (dict(order=None), EINVAL), (dict(pos=None), EINVAL), (dict(T=0), EINVAL),
    (dict(T=(1 << 20) + 1), EINVAL), (dict(k=65), EINVAL), (dict(E=0), EINVAL), (dict(E=1025), EINVAL), (dict(ids=A + 1), EALIGN),
    (dict(pos=A + 2), EALIGN), (dict(ws=A + 2), EALIGN)])
def test_plan(lib, change, want):
    p = dict(ids=A, T=4, k=2, E=8, off=A, order=A, pos=A, ws=A) | change
    assert lib.expert_plan(p["ids"], p["T"], p["k"], p["E"], p["off"], p["order"], p["pos"], p["ws"], None) == want


def test_plan_workspace(lib):
    assert lib.expert_plan_workspace(0, 1, 8) == -1
    assert lib.expert_plan_workspace(8, 65, 8) == -1
    assert lib.expert_plan_workspace(8, 2, 1025) == -1
    assert lib.expert_plan_workspace(1, 1, 1) >= 0
    need = lib.expert_plan_workspace(1 << 20, 64, 1024)
    assert need >= 0
    if need:
        assert lib.expert_plan(A, 1 << 20, 64, 1024, A, A, A, None, None) == EINVAL


@pytest.mark.parametrize("change,want", [
    (dict(Y=None), EINVAL), (dict(pos=None), EINVAL), (dict(w=None), EINVAL), (dict(out=None), EINVAL), (dict(yt=3), EINVAL),
    (dict(ot=-1), EINVAL), (dict(rows=0), EINVAL), (dict(N=0), EINVAL), (dict(T=0), EINVAL), (dict(k=0), EINVAL),
    (dict(k=65), EINVAL), (dict(Y=A + 8), EALIGN), (dict(out=A + 4), EALIGN), (dict(pos=A + 2), EALIGN), (dict(w=A + 1), EALIGN)])
def test_combine(lib, change, want):
    p = dict(Y=A, yt=0, rows=8, N=64, pos=A, w=A, T=4, k=2, out=A, ot=0) | change
    assert lib.expert_combine(p["Y"], p["yt"], p["rows"], p["N"], p["pos"], p["w"], p["T"], p["k"], p["out"], p["ot"],
                              None) == want
    assert lib.expert_combine_backward(p["out"], p["ot"], p["Y"], p["yt"], p["rows"], p["N"], p["pos"], p["w"], p["T"], p["k"],
                                       A, A, None) == want


def test_combine_backward_outputs(lib):
    for dy, dw, want in ((None, A, EINVAL), (A, None, EINVAL), (A + 8, A, EALIGN), (A, A + 2, EALIGN)):
        assert lib.expert_combine_backward(A, 0, A, 0, 8, 64, A, A, 4, 2, dy, dw, None) == want


def test_binding_refuses_host_tensors():
    from block_scaled_precision_mxgemm_amd import mxgemm as mx

    x = torch.zeros((4, 64))
    q, s, i = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4), torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: mx.int8gemm_quantize(x), lambda: mx.int8gemm_run(q, s, q, s), lambda: mx.expert_route(x, 2),
                 lambda: mx.int8gemm_run_grouped(q, s, q[None], s[None], i[0]), lambda: mx.expert_plan(i, 8),
                 lambda: mx.expert_route_backward(x, i, x[:, :2]), lambda: mx.expert_combine(x, i, x[:, :2]),
                 lambda: mx.expert_combine_backward(x, x, i, x[:, :2])):
        with pytest.raises(ValueError, match="must be a GPU tensor"):
            call()


def test_large_tile_cases_take_their_tiles():
    """The GPU tests of the large tiles are at sizes that take them."""
    import test_gpu_int8_large as large

    chosen = large.load_choice()
    for tile, M, N, K in large.DENSE:
        assert chosen(M, N, K) == tile
    for tile, E, tokens, div, N, K in large.EXPERTS:
        assert chosen(tokens * div, N, K, E) == tile
    for tile, M, N in large.LARGEST:
        assert chosen(M, N, 131056) == tile
    for tile, rows, N, K in large.OFFSETS:
        assert chosen(rows, N, K, 3) == tile


def test_many_tiles_cases_take_every_tile():
    """The GPU tests of more tiles than run at once reach all of them."""
    import test_gpu_int8 as gpu
    import test_gpu_int8_large as large

    chosen = large.load_choice()
    cases = [m.args[1] for f in (gpu.test_product_many_tiles, gpu.test_experts_many_tiles) for m in f.pytestmark
             if m.name == "parametrize"]
    taken = {chosen(*c) for c in cases[0]} | {chosen(c[1] * c[2], c[3], c[4], c[0]) for c in cases[1]}
    assert taken == set(large.TILES)


# ---- the 64-bit forms that the GPU tests compare with -----------------------


def test_reference_quantizer():
    q, s = ref.quantize(np.array([[127.0, -0.5, 0.5, 1.5] * 4, [0.0] * 16, [np.nan] + [1.0] * 15], np.float32))
    assert s[0] == 1.0 and s[1] == 0.0 and np.isnan(s[2])
    assert list(q[0, :4]) == [127, 0, 0, 2] and not q[1:].any()


def test_reference_router():
    x = np.array([[0.0, 1.0, 1.0, -np.inf, 3.0, -1.0]])
    ids, w = ref.route(x, 4, "softmax")
    assert list(ids[0]) == [4, 1, 2, 0]
    assert w.sum() == pytest.approx(1.0)
    ids, w = ref.route(x, 3, "sigmoid", bias=np.array([9.0, 0, 0, 99.0, 0, 0]), renormalize=False, scale=2.0)
    assert list(ids[0]) == [0, 4, 1] and w[0, 0] == pytest.approx(1.0)
    ids, _ = ref.route(x, 3, "softmax", groups=3, top_groups=1)
    assert list(ids[0]) == [4, 5, -1]
    ids, w = ref.route(np.full((1, 4), -np.inf), 2, "softmax")
    assert (ids == -1).all() and (w == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_reference_gradient_against_differences(score, renormalize):
    """Central differences of the weights, the choice held: the step h = 1e-5
    costs h^2 times a third derivative below 10, rounding 1e-16 / h."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 12))
    ids, _ = ref.route(x, 4, score)
    dw = rng.standard_normal((3, 4))
    got, _ = ref.route_backward(x, ids, dw, score, renormalize, 1.7)
    h = 1e-5
    for t in range(3):
        for e in range(12):
            f = []
            for d in (h, -h):
                y = x[t].copy()
                y[e] += d
                f.append((ref.chosen_weights(y, list(ids[t]), score, renormalize, 1.7) * dw[t]).sum())
            assert got[t, e] == pytest.approx((f[0] - f[1]) / (2 * h), abs=1e-8)


def test_reference_plan():
    off, order, pos = ref.plan(np.array([[2, 0], [-1, 2], [0, 7]]), 3)
    assert list(off) == [0, 2, 2, 4] and list(order) == [1, 4, 0, 3, -1, -1]
    assert pos.tolist() == [[2, 0], [-1, 3], [1, -1]]
