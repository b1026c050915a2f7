"""Routing to experts, its plan and gradient, the combination of the experts'
outputs, and a layer of int8 experts made of them, against 64-bit forms."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from gpu_util import binding, say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {0: torch.float32, 1: torch.bfloat16, 2: torch.float16}
SCORES = {"softmax": 0, "sigmoid": 1}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert binding().mxgemm_device_supported()
    yield


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


# ---- routing ----------------------------------------------------------------


def _weight_tol(x, ids, k):
    """Relative error allowed to a weight, for an evaluation in fp32: with d the
    largest distance of a chosen logit from the row's largest finite one, each
    exponential is off by at most 3 |d| + 2 roundings (the difference, the
    change of base, the exponential itself), the sum of k of them by 3 k more
    (a term's error times its size is largest at |d| = 1) and the division, the
    scale and the result by 6."""
    x = x.astype(np.float64)   # the distance of two fp32 values can pass fp32's range
    finite = np.where(np.isfinite(x), x, -np.inf)
    top = finite.max(-1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    d = np.abs(np.take_along_axis(np.where(np.isfinite(x), x, 0.0), np.maximum(ids, 0), 1) - top)
    return (3 * d + 3 * x.shape[1] ** 0.5 + 3 * k + 8) * U


def _check_route(x, k, score, kind=0, **kw):
    b = binding()
    t = dev(x).to(TYPES[kind])
    x = t.float().cpu().numpy()
    bias = kw.get("bias")
    ids = torch.full((len(x), k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((len(x), k), -7.0, device=DEV)
    b.expert_route(t, k, SCORES[score], ids=ids, weights=w, **dict(kw, bias=None if bias is None else dev(bias)))
    torch.cuda.synchronize()
    ids_r, w_r = ref.route(x, k, score, **kw)
    assert np.array_equal(ids.cpu().numpy(), ids_r)
    got = w.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(w_r))
    tol = _weight_tol(x, ids_r, k) * np.abs(w_r) + 2.0 ** -149
    off = np.where(np.isnan(w_r), 0.0, np.abs(got - w_r))
    say("  error / bound %.3g" % np.max(np.where(np.isnan(w_r), 0.0, off / tol)))
    assert (np.where(np.isnan(w_r), True, off <= tol)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 4), (2, 8, 2), (3, 5, 5), (17, 63, 6), (33, 65, 8), (100, 128, 8),
                                   (7, 192, 6), (50, 256, 8), (5, 257, 16), (9, 512, 10), (4, 1000, 64), (6, 1024, 33),
                                   (300, 16, 1), (1025, 60, 4), (64, 96, 3)])
def test_route(score, T, E, k):
    say("route", score, T, E, k)
    x = np.random.default_rng(T + E + k).standard_normal((T, E)).astype(np.float32) * 2
    _check_route(x, k, score)


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_types_and_ties(kind, score, renormalize):
    """16-bit logits tie often: the lower expert comes first."""
    say("route types", kind, score, renormalize)
    x = np.random.default_rng(kind).standard_normal((200, 200)).astype(np.float32)
    _check_route(x, 8, score, kind, renormalize=renormalize, scale=2.5)
    _check_route(np.round(x), 16, score, kind, renormalize=renormalize)
    _check_route(np.zeros((3, 130), np.float32), 70 - 6, score, kind, renormalize=renormalize)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,k", [(8, 2, 1, 4), (64, 8, 3, 6), (128, 4, 2, 8), (60, 5, 5, 7), (256, 8, 4, 16),
                                                   (64, 64, 9, 9), (512, 16, 2, 5), (1024, 64, 7, 20), (6, 3, 2, 4)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_groups(score, E, groups, top_groups, k, group_top, with_bias):
    say("route groups", score, E, groups, top_groups, k, group_top, with_bias)
    rng = np.random.default_rng(E + groups + k)
    x = rng.standard_normal((70, E)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if with_bias else None
    _check_route(x, k, score, groups=groups, top_groups=top_groups, group_top=group_top, bias=bias, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups_with_one_expert_left(score):
    """The score of a group whose other experts are all out is that of the one
    left, against groups with two and with none."""
    say("route groups with one expert left", score)
    x = np.full((4, 16), -np.inf, np.float32)
    x[0, [1, 5, 6, 9]] = [3.0, 1.0, 0.5, 0.0]        # 3 against 1 + 0.5, by its score: s(3) or the pair
    x[1, [0, 4, 5, 8, 9, 12]] = [0.2, 0.1, 0.0, 0.1, 0.1, 9.0]
    x[2, [7, 15]] = [-4.0, -5.0]
    x[3, :4] = 0.0
    for top_groups in (1, 2, 3):
        _check_route(x, 3, score, groups=4, top_groups=top_groups, group_top=2)
        _check_route(x, 3, score, groups=4, top_groups=top_groups, group_top=2, bias=np.linspace(0, 0.3, 16).astype(np.float32))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_extreme_logits(score, renormalize):
    say("route extremes", score, renormalize)
    rng = np.random.default_rng(5)
    E = 70
    x = rng.standard_normal((16, E)).astype(np.float32)
    low = np.finfo(np.float32).min
    x[0] = -np.inf                       # no expert at all
    x[1] = -np.inf
    x[1, 66] = 0.5                       # one
    x[2, 3:] = -np.inf                   # three
    x[3] = low                           # the type's lowest value is a number
    x[4, 10:] = low
    x[5, 8] = np.nan
    x[6, 8] = np.inf
    x[7] = np.nan
    x[8, ::2] = np.nan
    x[9] = rng.standard_normal(E) * 1000
    x[10] = -200.0 - rng.random(E)       # sigmoids that underflow fp32
    x[11] = 50.0 + rng.random(E)         # and that round to one
    x[12, ::2] = -np.inf
    x[13, 69] = np.nan
    x[13, :68] = -np.inf
    x[14] = 3e38 * rng.standard_normal(E).clip(-1, 1)
    _check_route(x, 6, score, renormalize=renormalize)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    bias[4] = -np.inf
    _check_route(x, 6, score, renormalize=renormalize, bias=bias)
    _check_route(x, 6, score, renormalize=renormalize, bias=bias, groups=7, top_groups=2, group_top=2)
    bias[5] = np.nan
    _check_route(x[:12], 6, score, renormalize=renormalize, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_close_scores(score):
    """Biased scores a few 64-bit steps of their 32-bit spacing apart: the order
    is the real one."""
    say("route close scores", score)
    rng = np.random.default_rng(6)
    T, E = 256, 64
    x = rng.standard_normal((T, E)).astype(np.float32)
    # the bias that makes every score of row 0 nearly equal
    s = ref.scores(x[0].astype(np.float64), score)
    bias = (0.75 - s).astype(np.float32)
    x[1:] = x[0] + (rng.standard_normal((T - 1, E)) * 2e-7).astype(np.float32)
    _check_route(x, 8, score, bias=bias)
    _check_route(x, 8, score, bias=bias, groups=8, top_groups=3, group_top=2)


def test_route_logits_past_4_gib():
    """The last of 2^20 tokens over 1024 experts, against calls of those tokens alone."""
    say("route past 4 GiB")
    b = binding()
    T, E, k = 1 << 20, 1024, 3
    x = torch.empty((T, E), device=DEV)
    rows = torch.tensor([0, 1, 524287, 524288, T - 2, T - 1], device=DEV)
    x.fill_(0.5)
    x[rows] = torch.randn((6, E), device=DEV)
    bias = torch.randn(E, device=DEV) * 0.1
    for kw in ({}, {"score": b.SCORE_SIGMOID, "bias": bias, "groups": 8, "top_groups": 2, "group_top": 2}):
        ids, w = b.expert_route(x, k, **kw)
        some, few = b.expert_route(x[rows].contiguous(), k, **kw)
        assert torch.equal(ids[rows], some) and torch.equal(w[rows], few)
    dw = torch.randn((T, k), device=DEV)
    d = torch.full((T, E), 7.0, device=DEV)
    for renormalize in (True, False):
        b.expert_route_backward(x, ids, dw, renormalize=renormalize, d_logits=d)
        want = b.expert_route_backward(x[rows].contiguous(), ids[rows].contiguous(), dw[rows].contiguous(),
                                       renormalize=renormalize)
        assert torch.equal(d[rows], want)


# ---- gradient ---------------------------------------------------------------


def _check_backward(x, ids, dw, score, kind=0, renormalize=True, scale=1.0):
    b = binding()
    t = dev(x).to(TYPES[kind])
    x = t.float().cpu().numpy()
    out = torch.full(x.shape, 99.0, dtype=TYPES[kind], device=DEV)
    b.expert_route_backward(t, dev(ids), dev(dw), SCORES[score], renormalize=renormalize, scale=scale, d_logits=out)
    torch.cuda.synchronize()
    want, mag = ref.route_backward(x, ids, dw, score, renormalize, scale)
    # each term is a product of scores (see _weight_tol; twice, and the sum of
    # all E of a softmax) and a sum over the k choices
    d = (x.max(-1, keepdims=True) - x.min(-1, keepdims=True))
    tol = (6 * d + 6 * x.shape[1] ** 0.5 + 6 * ids.shape[1] + 24) * U * mag
    tol = tol + ref.half_step(TYPES[kind]) * (np.abs(want) + tol) + torch.finfo(TYPES[kind]).smallest_normal * ref.half_step(TYPES[kind])
    off = np.abs(out.float().cpu().numpy().astype(np.float64) - want)
    say("  error / bound %.3g" % np.max(off / np.maximum(tol, 1e-300)))
    assert (off <= tol).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 4), (5, 8, 2), (33, 65, 8), (129, 128, 8), (7, 256, 6), (3, 1024, 64),
                                   (6, 500, 10), (40, 61, 3)])
def test_route_backward(score, renormalize, kind, T, E, k):
    say("route backward", score, renormalize, kind, T, E, k)
    rng = np.random.default_rng(T + E + k)
    x = rng.standard_normal((T, E)).astype(np.float32)
    ids, _ = ref.route(x, k, score)
    _check_backward(x, ids, rng.standard_normal((T, k)).astype(np.float32), score, kind, renormalize, 1.25)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward_missing_choices(score, renormalize):
    """Slots without an expert, ids outside the experts, masked logits, and a row with no choice at all."""
    say("route backward missing", score, renormalize)
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 20)).astype(np.float32)
    ids = np.stack([rng.permutation(20)[:4] for _ in range(6)]).astype(np.int32)
    ids[1] = -1
    ids[2, 2:] = -1
    ids[3, 0] = 20
    ids[4, 1] = 2147483647
    ids[4, 2] = -2147483648
    _check_backward(x, ids, rng.standard_normal((6, 4)).astype(np.float32), score, 0, renormalize)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_route_backward_of_one_choice(score, kind):
    """A renormalized weight of one choice is constant: its gradient is zero, exactly."""
    say("route backward of one choice", score, kind)
    b = binding()
    for T, E in ((149, 95), (33, 8), (20, 300)):
        x = (torch.randn((T, E), device=DEV) * 3).to(TYPES[kind])
        ids, w = b.expert_route(x, 1, SCORES[score])
        assert ((w - 1).abs() <= 2.0 ** -23).all()  # p times 1 / p: two roundings
        dw = torch.randn((T, 1), device=DEV)
        assert (b.expert_route_backward(x, ids, dw, SCORES[score]) == 0).all()
        ids = torch.cat([torch.full_like(ids, -1), ids, torch.full_like(ids, -1)], 1)
        assert (b.expert_route_backward(x, ids, dw.expand(T, 3).contiguous(), SCORES[score], scale=2.5) == 0).all()
        dw[0] = float("nan")
        got = b.expert_route_backward(x, ids[:, 1:2].contiguous(), dw, SCORES[score])
        assert torch.isnan(got[0, ids[0, 1].long()]) and (got[1:] == 0).all()


def _check_dominated(x, ids, dw, renormalize, kind, scale=1.0, score="softmax"):
    """The gradient where one logit, of expert a, leads: with D_e the sum of
    expert e's dw and s the softmax (where weights are renormalized: the chosen
    scores p over their sum), dl_e = scale s_e sum_f s_f (D_e - D_f) has no terms
    that cancel (sigmoid: times 1 - p_e).  Allowed are the roundings of _check_backward, of the size of
    s_e (|D_e - D_a| + sum_f s_f |D_f - D_a|): what is left of dl_a when a has
    nearly all of the sum, and not s_a |D_a|."""
    b = binding()
    t = dev(x).to(TYPES[kind])
    x = t.float().cpu().numpy().astype(np.float64)
    out = torch.full(x.shape, 99.0, dtype=TYPES[kind], device=DEV)
    b.expert_route_backward(t, dev(ids), dev(dw), SCORES[score], renormalize=renormalize, scale=scale, d_logits=out)
    got = out.double().cpu().numpy()
    for r in range(len(x)):
        D, p = np.zeros(x.shape[1]), np.exp(x[r] - x[r].max()) if score == "softmax" else 1 / (1 + np.exp(-x[r]))
        slope = 1 / (1 + np.exp(x[r])) if score == "sigmoid" else 1.0
        np.add.at(D, ids[r], dw[r].astype(np.float64) * scale)
        if renormalize:
            named = np.zeros(x.shape[1], bool)
            named[ids[r]] = True
            p = np.where(named, p / p[named].max(), 0.0)
        p = p / p.sum()
        a = int(np.argmax(p))
        want = slope * p * ((D[:, None] - D[None, :]) * p).sum(1)
        mag = slope * p * (np.abs(D - D[a]) + (p * np.abs(D - D[a])).sum())
        tol = (6 * (x[r].max() - x[r].min()) + 6 * x.shape[1] ** 0.5 + 6 * ids.shape[1] + 24) * U * mag
        tol = tol + ref.half_step(TYPES[kind]) * (np.abs(want) + tol + torch.finfo(TYPES[kind]).smallest_normal) + 2.0 ** -126 * np.abs(D).max()
        worst = np.max(np.abs(got[r] - want) / np.maximum(tol, 1e-300))
        say("  lead %.3g: error / bound %.3g" % (np.sort(x[r])[-1] - np.sort(x[r])[-2], worst))
        assert worst <= 1.0


LEADS = [0.0, 0.5, 4.0, 8.0, 12.0, 14.0, 16.0, 17.0, 18.0, 20.0, 22.0, 25.0, 40.0, 70.0]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("E", [8, 100, 200, 300, 1000])
def test_route_backward_of_a_leading_choice(kind, E):
    """Softmax weights that are not renormalized, one of them close to one."""
    say("route backward of a leading choice", kind, E)
    rng = np.random.default_rng(E)
    x = (0.5 * rng.standard_normal((len(LEADS), E))).astype(np.float32)
    a = rng.integers(0, E, len(LEADS))
    others = np.stack([rng.permutation(np.delete(np.arange(E), e)) for e in a])
    for r, lead in enumerate(LEADS):
        x[r, a[r]] = np.sort(x[r])[-1] + lead
    for k in (1, 3, 7):
        ids = np.concatenate([a[:, None], others[:, :k - 1]], 1).astype(np.int32)
        for dw in (np.ones(ids.shape), rng.standard_normal(ids.shape)):
            _check_dominated(x, ids, dw.astype(np.float32), False, kind, 2.5)
        # a leading expert that is not among the chosen
        _check_dominated(x, others[:, :k].astype(np.int32), np.ones((len(x), k), np.float32), False, kind)
    # the same expert twice: whole numbers, whose sums are exact
    ids = np.concatenate([a[:, None], others[:, :2], a[:, None], others[:, 1:2]], 1).astype(np.int32)
    _check_dominated(x, ids, np.array([3, -2, 1, 4, 5], np.float32)[None].repeat(len(x), 0), False, kind)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 100, 300])
def test_route_backward_of_a_leading_renormalized_choice(score, E):
    """Renormalized weights, one of them so close to one that 64 bits do not hold the rest."""
    say("route backward of a leading renormalized choice", score, E)
    rng = np.random.default_rng(E)
    x = (0.5 * rng.standard_normal((len(LEADS), E))).astype(np.float32)
    ids = np.stack([rng.permutation(E)[:7] for _ in LEADS]).astype(np.int32)
    for r, lead in enumerate(LEADS):
        x[r, ids[r, r % 7]] = np.sort(x[r])[-1] + lead
        if score == "sigmoid":
            x[r] -= x[r].max()
    for k in (2, 7):
        for r in range(len(LEADS)):
            # the leading choice among the k
            mine = np.roll(ids[r:r + 1], -(r % 7), 1)[:, :k].copy()
            mine = np.roll(mine, r % k, 1)
            for dw in (np.arange(k)[None] + 1.0, rng.standard_normal((1, k))):
                _check_dominated(x[r:r + 1], mine, dw.astype(np.float32), True, 0, 1.5, score)


@pytest.mark.parametrize("E", [8, 130, 600])
def test_route_backward_of_rows_with_nan(E):
    """Weights that are not renormalized: a NaN logit makes its row's gradient NaN
    wherever there is a score; masked experts have none, nor has a row without any."""
    say("route backward of rows with NaN", E)
    b = binding()
    x = torch.randn((6, E), device=DEV)
    x[:, ::3] = -float("inf")
    ids = torch.tensor([[1, 2, 4]] * 6, dtype=torch.int32, device=DEV)
    ids[4] = -1
    x[1, 1], x[3, E - 1 if (E - 1) % 3 else E - 2] = float("nan"), float("nan")
    x[4] = -float("inf")
    got = b.expert_route_backward(x, ids, torch.randn((6, 3), device=DEV), renormalize=False)
    assert (got[:, ::3] == 0).all() and (got[4] == 0).all()
    there = torch.arange(E, device=DEV) % 3 != 0
    for row in (1, 3):
        assert torch.isnan(got[row, there]).all()
    assert (torch.isfinite(got[[0, 2, 5]]) & ((got[[0, 2, 5]] != 0) == there)).all()


def test_route_backward_against_differences():
    """The kernel's gradient against differences of the kernel's own weights.
    A step of 2^-6 costs h^2/6 times a third derivative below 2 per unit of dw
    (4e-5 * 4 choices * |dw| <= 4), rounding 2^-23 / h per weight."""
    say("route backward differences")
    b = binding()
    rng = np.random.default_rng(12)
    T, E, k, h = 4, 10, 4, 2.0 ** -6
    for score in (0, 1):
        for renormalize in (True, False):
            x = rng.standard_normal((T, E)).astype(np.float32)
            # choices that a step does not change: the chosen logits well above the rest
            x[:, :k] += np.array([9, 7, 5, 3], np.float32)
            x[:, k:] -= 3
            dw = rng.standard_normal((T, k)).astype(np.float32)
            ids, _ = b.expert_route(dev(x), k, score, renormalize=renormalize)
            got = b.expert_route_backward(dev(x), ids, dev(dw), score, renormalize=renormalize).cpu().numpy()
            for e in range(E):
                f = []
                for d in (h, -h):
                    y = x.copy()
                    y[:, e] += np.float32(d)
                    i2, w = b.expert_route(dev(y), k, score, renormalize=renormalize)
                    assert torch.equal(i2, ids)
                    f.append((w.double().cpu().numpy() * dw).sum(1))
                assert np.abs((f[0] - f[1]) / (2 * h) - got[:, e]).max() <= 4e-5 * 4 * 4 + 16 * 2.0 ** -23 / h


# ---- plan -------------------------------------------------------------------


def _check_plan(ids, E):
    b = binding()
    n = ids.size
    outs = [torch.full((m,), -9, dtype=torch.int32, device=DEV) for m in (E + 1, n)]
    pos = torch.full(ids.shape, -9, dtype=torch.int32, device=DEV)
    b.expert_plan(dev(ids), E, offsets=outs[0], order=outs[1], position=pos)
    torch.cuda.synchronize()
    for got, want in zip((*outs, pos), ref.plan(ids, E)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 4, 64), (3, 2, 5), (16, 4, 64), (63, 1, 7), (64, 1, 1024), (65, 3, 16),
                                   (500, 8, 256), (1025, 2, 63), (4096, 4, 16), (5000, 7, 1000), (20000, 8, 128),
                                   (70001, 3, 1), (40000, 8, 1024)])
def test_plan(T, k, E):
    say("plan", T, k, E)
    rng = np.random.default_rng(T + E)
    _check_plan(rng.integers(0, E, (T, k)).astype(np.int32), E)
    # skewed, with slots without an expert
    ids = np.minimum((E + 2) * rng.random((T, k)) ** 3, E + 1).astype(np.int32) - 1
    _check_plan(ids, E)


@pytest.mark.parametrize("n", [5, 5000, 200000])
def test_plan_edges(n):
    say("plan edges", n)
    _check_plan(np.full((n, 1), 3, np.int32), 9)
    _check_plan(np.full((n, 1), -1, np.int32), 9)
    ids = np.full((n, 1), 9, np.int32)
    ids[n // 2] = 8
    ids[0] = -2147483648
    ids[n - 1] = 2147483647
    _check_plan(ids, 9)


@pytest.mark.parametrize("E", [1, 1024])
def test_plan_most_slots(E):
    """As many slots as a call can have."""
    say("plan most slots", E)
    b = binding()
    T, k = 1 << 20, 64
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV).random_(-1, E + 1)
    off, order, pos = b.expert_plan(ids, E)
    flat = torch.where((ids < 0) | (ids >= E), E, ids).flatten().to(torch.int16)
    by, slot = torch.sort(flat, stable=True)
    counts = torch.bincount(flat.int(), minlength=E + 1)
    live = int(counts[:E].sum())
    assert torch.equal(off.long(), torch.cat([counts.new_zeros(1), counts[:E].cumsum(0)]))
    assert torch.equal(order[:live], slot[:live].int()) and (order[live:] == -1).all()
    p = pos.flatten()
    assert (p[slot[live:]] == -1).all()
    assert torch.equal(p[slot[:live]], torch.arange(live, dtype=torch.int32, device=DEV))


# ---- combination ------------------------------------------------------------


def _combine_case(T, k, N, y_kind, o_kind, seed, missing=False, rows=None):
    rng = np.random.default_rng(seed)
    rows = T * k if rows is None else rows
    y = dev(rng.standard_normal((rows, N)).astype(np.float32)).to(TYPES[y_kind])
    pos = rng.permutation(rows)[:T * k].reshape(T, k).astype(np.int32)
    if missing:
        pos[rng.random((T, k)) < 0.4] = -1
        pos[0] = -1
        pos[-1, 0] = rows
        pos[-1, -1] = 2147483647
    w = rng.standard_normal((T, k)).astype(np.float32)
    d = dev(rng.standard_normal((T, N)).astype(np.float32)).to(TYPES[o_kind])
    return y, pos, w, d


def _check_combine(T, k, N, y_kind, o_kind, seed, **kw):
    b = binding()
    y, pos, w, d = _combine_case(T, k, N, y_kind, o_kind, seed, **kw)
    rows = y.shape[0]
    yf, df = y.double().cpu().numpy(), d.double().cpu().numpy()
    live = (pos >= 0) & (pos < rows)
    at = np.where(live, pos, 0)
    wl = np.where(live, w, 0.0).astype(np.float64)
    out = torch.full((T, N), 99.0, dtype=TYPES[o_kind], device=DEV)
    b.expert_combine(y, dev(pos), dev(w), out_type=o_kind, out=out)
    torch.cuda.synchronize()
    want = (wl[..., None] * yf[at]).sum(1)
    # k products and sums in fp32: k roundings of at most the sum of magnitudes
    tol = (k + 1) * U * (np.abs(wl[..., None] * yf[at])).sum(1)
    tol = tol + ref.half_step(TYPES[o_kind]) * (np.abs(want) + tol) + 2.0 ** -25
    off = np.abs(out.double().cpu().numpy() - want)
    assert (off <= tol).all()
    # gradients
    d_y = torch.full((rows, N), 99.0, dtype=TYPES[y_kind], device=DEV)
    d_w = torch.full((T, k), 99.0, device=DEV)
    b.expert_combine_backward(d, y, dev(pos), dev(w), d_y=d_y, d_weights=d_w)
    torch.cuda.synchronize()
    got = d_y.double().cpu().numpy()
    named = np.zeros(rows, bool)
    for t in range(T):
        for j in range(k):
            if live[t, j]:
                named[pos[t, j]] = True
                g = wl[t, j] * df[t]
                h = (ref.half_step(TYPES[y_kind]) + 1.01 * U) * np.abs(g) + 2.0 ** -25
                assert (np.abs(got[pos[t, j]] - g) <= h).all()
    assert (got[~named] == 99.0).all()
    prod = df[:, None, :] * yf[at] * live[..., None]
    # a sum of N products in any order: at most N roundings of the sum of magnitudes
    assert (np.abs(d_w.double().cpu().numpy() - prod.sum(-1)) <= (N + 1) * U * np.abs(prod).sum(-1)).all()
    assert (d_w.cpu().numpy()[~live] == 0).all()


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 4, 4096), (3, 2, 7), (5, 8, 520), (17, 6, 1000), (64, 1, 8), (9, 64, 33),
                                   (130, 3, 2056), (2, 2, 16384), (1, 1, 40000)])
@pytest.mark.parametrize("missing", [False, True])
def test_combine(T, k, N, missing):
    say("combine", T, k, N, missing)
    _check_combine(T, k, N, 1, 1, T + N, missing=missing)


@pytest.mark.parametrize("y_kind", [0, 1, 2])
@pytest.mark.parametrize("o_kind", [0, 1, 2])
@pytest.mark.parametrize("N", [264, 100, 31])
def test_combine_types(y_kind, o_kind, N):
    say("combine types", y_kind, o_kind, N)
    _check_combine(20, 4, N, y_kind, o_kind, N + y_kind, rows=95)


def test_combine_skips_what_no_slot_names():
    """NaN and infinities in rows that no slot names, and a zero weight of a named one."""
    say("combine unnamed rows")
    b = binding()
    y = torch.full((6, 64), float("nan"), device=DEV)
    y[2], y[4] = 1.0, 3.0
    pos = dev(np.array([[2, -1], [4, 99]], np.int32))
    out = b.expert_combine(y, pos, torch.tensor([[0.5, 7.0], [2.0, float("nan")]], device=DEV))
    assert torch.equal(out[:, 0].cpu(), torch.tensor([0.5, 6.0]))
    d_y, d_w = b.expert_combine_backward(torch.ones(2, 64, device=DEV), y, pos, torch.ones(2, 2, device=DEV))
    assert torch.equal(d_w.cpu(), torch.tensor([[64.0, 0.0], [192.0, 0.0]]))
    assert d_y[[0, 1, 3, 5]].abs().max() == 0


def test_combine_rows_past_4_gib():
    say("combine past 4 GiB")
    b = binding()
    rows, N = 140000, 16384
    y = torch.empty((rows, N), dtype=torch.bfloat16, device=DEV)
    y[-1], y[70000], y[3] = 2.0, 3.0, 5.0
    pos = dev(np.array([[rows - 1, 70000, 3]], np.int32))
    w = torch.tensor([[1.0, 10.0, 100.0]], device=DEV)
    assert (b.expert_combine(y, pos, w) == 532.0).all()
    d_y, d_w = b.expert_combine_backward(torch.ones((1, N), dtype=torch.bfloat16, device=DEV), y, pos, w, d_y=y)
    assert torch.equal(d_w.cpu(), torch.tensor([[2.0 * N, 3.0 * N, 5.0 * N]]))
    assert (d_y[-1] == 1).all() and (d_y[70000] == 10).all() and (d_y[3] == 100).all()


@pytest.mark.parametrize("T,k,N", [(700, 3, 1041), (257, 8, 513), (2049, 1, 520), (1001, 2, 128), (77, 5, 129), (333, 7, 61),
                                   (1500, 1, 16), (2, 64, 127)])
def test_combine_row_lengths(T, k, N):
    say("combine row lengths", T, k, N)
    _check_combine(T, k, N, 1, 1, T + N, missing=True)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("T,k,N", [(6300, 8, 1027), (40, 64, 30000), (16500, 8, 1027), (40, 64, 60000)])
def test_combine_backward_of_large_rows(kind, T, k, N):
    """Rows of 100 MB and of more than 256 MB together, a few of them without a slot."""
    say("combine backward large", kind, T, k, N)
    b = binding()
    rows = T * k + 5
    slot = torch.randperm(rows, device=DEV)[:T * k]
    pos = slot.int().view(T, k)
    pos[1, 1] = -1
    y = torch.randint(-2, 3, (rows, N), device=DEV).to(TYPES[kind])
    d = torch.randint(-1, 2, (T, N), device=DEV).to(TYPES[kind])
    w = torch.randint(-3, 4, (T, k), device=DEV).float()
    d_y, d_w = b.expert_combine_backward(d, y, pos, w)
    want_y = torch.zeros_like(y)
    # whole numbers: sums below 2^24, products of at most 3
    for j in range(k):
        live = pos[:, j] >= 0
        at = pos[live, j].long()
        want_y[at] = (w[live, j, None] * d[live].float()).to(TYPES[kind])
        want_w = torch.zeros(T, device=DEV)
        want_w[live] = (y[at].float() * d[live].float()).sum(1)
        assert torch.equal(d_w[:, j], want_w), j
    assert torch.equal(d_y, want_y)


@pytest.mark.parametrize("y_kind,o_kind", [(0, 0), (1, 1), (2, 0), (0, 2)])
@pytest.mark.parametrize("T,k,N", [(300, 4, 100), (3000, 2, 1041), (64, 8, 7168), (700, 3, 4096), (9000, 4, 3848)])
def test_combine_backward_in_place(y_kind, o_kind, T, k, N):
    """dY in Y's memory, for every number of lanes per row and for rows that pass the caches."""
    say("combine backward in place", y_kind, o_kind, T, k, N)
    b = binding()
    rows = T * k + 3
    pos = torch.randperm(rows, device=DEV)[:T * k].int().view(T, k)
    pos[T // 2, 1] = -1
    y = torch.randn((rows, N), device=DEV).to(TYPES[y_kind])
    d = torch.randn((T, N), device=DEV).to(TYPES[o_kind])
    w = torch.randn((T, k), device=DEV)
    want_y, want_w = b.expert_combine_backward(d, y, pos, w, d_y=y.clone())
    got_y, got_w = b.expert_combine_backward(d, y, pos, w, d_y=y)
    assert got_y.data_ptr() == y.data_ptr()
    assert torch.equal(got_y, want_y) and torch.equal(got_w, want_w)


def test_combine_most_slots():
    """As many slots as a call can have: 2^20 tokens of 64 choices."""
    say("combine most slots")
    b = binding()
    T, k = 1 << 20, 64
    n = T * k
    slot = torch.arange(n, dtype=torch.int32, device=DEV)
    pos = (n - 1 - slot).view(T, k)
    y = (slot % 5 - 2).to(torch.bfloat16)[:, None]
    w = (slot % 3 - 1).float().view(T, k)
    d = (torch.arange(T, device=DEV) % 7 - 3).to(torch.bfloat16)[:, None]
    at = y[:, 0].flip(0).view(T, k).float()  # y of a slot's row
    # small whole numbers: every sum is exact
    assert torch.equal(b.expert_combine(y, pos, w, out_type=b.OUT_F32)[:, 0], (at * w).sum(1))
    d_y, d_w = b.expert_combine_backward(d, y, pos, w)
    assert torch.equal(d_w, at * d.float())
    assert torch.equal(d_y[:, 0].flip(0).view(T, k), (w * d.float()).to(torch.bfloat16))


# ---- together ---------------------------------------------------------------


def _layer(b, x, router, up, up_s, up_b, down, down_s, down_b, k, ids=None):
    """One layer of int8 experts over the rows of x, as a program calls it."""
    if ids is None:
        ids, w = b.expert_route(x.float() @ router, k, b.SCORE_SIGMOID, scale=1.25)
    else:
        ids, w = ids
    off, order, pos = b.expert_plan(ids, up.shape[0])
    q, s = b.int8gemm_quantize(x)
    h = b.int8gemm_run_grouped(q, s, up, up_s, off, index=order, index_div=k, bias=up_b, act=b.ACT_GELU, out_type=b.OUT_BF16)
    q, s = b.int8gemm_quantize(h)
    y = b.int8gemm_run_grouped(q, s, down, down_s, off, bias=down_b, out_type=b.OUT_BF16)
    return ids, w, h, y, pos, b.expert_combine(y, pos, w)


def _layer_operands(rng, T, D, H, E):
    b = binding()
    x = dev(rng.standard_normal((T, D)).astype(np.float32)).bfloat16()
    router = dev((rng.standard_normal((D, E)) / np.sqrt(D)).astype(np.float32))
    up, up_s = b.int8gemm_quantize(dev((rng.standard_normal((E * H, D)) / np.sqrt(D)).astype(np.float32)))
    down, down_s = b.int8gemm_quantize(dev((rng.standard_normal((E * D, H)) / np.sqrt(H)).astype(np.float32)))
    up_b, down_b = (dev(rng.standard_normal((E, n)).astype(np.float32)) for n in (H, D))
    return x, router, up.view(E, H, D), up_s.view(E, H), up_b, down.view(E, D, H), down_s.view(E, D), down_b


@pytest.mark.parametrize("T,D,H,E,k", [(1, 256, 512, 8, 2), (16, 512, 272, 64, 4), (100, 256, 528, 5, 2), (700, 272, 1040, 16, 3)])
def test_layer(T, D, H, E, k):
    """Each step's output against its 64-bit form on the step's own input."""
    say("layer", T, D, H, E, k)
    b = binding()
    rng = np.random.default_rng(T)
    ops = _layer_operands(rng, T, D, H, E)
    ids, w, h, y, pos, out = _layer(b, *ops, k)
    torch.cuda.synchronize()
    x, router, up, up_s, up_b, down, down_s, down_b = ops
    ids_r, _ = ref.route((x.float() @ router).cpu().numpy(), k, "sigmoid", scale=1.25)
    assert np.array_equal(ids.cpu().numpy(), ids_r)
    off, order, pos_r = ref.plan(ids_r, E)
    assert np.array_equal(pos.cpu().numpy(), pos_r)
    for src, rows, weight, scale, bias, act, got in (
            (x, order // k, up, up_s, up_b, True, h), (h, np.arange(T * k), down, down_s, down_b, False, y)):
        q, s = ref.quantize(src.float().cpu().numpy())
        for e in range(E):
            mine = slice(off[e], off[e + 1])
            if off[e + 1] > off[e]:
                want, tol = ref.product(q[rows[mine]], s[rows[mine]], weight[e].cpu().numpy(), scale[e].cpu().numpy(),
                                        bias[e].cpu().numpy(), act)
                bound = tol + ref.half_step(torch.bfloat16) * (np.abs(want) + tol)
                assert (np.abs(got[mine].double().cpu().numpy() - want) <= bound).all()
    yf, wf = y.double().cpu().numpy(), w.double().cpu().numpy()
    want = (wf[..., None] * yf[pos_r]).sum(1)
    tol = (k + 1) * U * np.abs(wf[..., None] * yf[pos_r]).sum(1)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol + ref.half_step(torch.bfloat16) * (np.abs(want) + tol)).all()


def test_layer_of_many_tokens():
    """More than 2^20 slots: every step of the layer takes them, and tokens that
    repeat the first 64 come out as those."""
    say("layer of many tokens")
    b = binding()
    T, k = 131073, 8
    ops = _layer_operands(np.random.default_rng(5), 64, 64, 32, 16)
    x = ops[0].repeat(T // 64 + 1, 1)[:T].contiguous()
    chosen = b.expert_route(ops[0].float() @ ops[1], k, b.SCORE_SIGMOID)
    many = tuple(c.repeat(T // 64 + 1, 1)[:T].contiguous() for c in chosen)
    out = _layer(b, x, *ops[1:], k, ids=many)[-1]
    few = _layer(b, *ops, k, ids=chosen)[-1]
    assert torch.equal(out, few.repeat(T // 64 + 1, 1)[:T])


def test_layer_with_dropped_slots():
    """A padded batch: the padding rows' logits are all -inf, so they take no expert and come out as zero."""
    say("layer with padding")
    b = binding()
    rng = np.random.default_rng(4)
    T, D, H, E, k = 40, 256, 256, 8, 2
    ops = _layer_operands(rng, T, D, H, E)
    logits = ops[0].float() @ ops[1]
    logits[25:] = -float("inf")
    chosen = b.expert_route(logits, k)
    out = _layer(b, *ops, k, ids=chosen)[-1]
    alone = _layer(b, ops[0][:25].contiguous(), *ops[1:], k, ids=tuple(t[:25].contiguous() for t in chosen))[-1]
    assert (out[25:] == 0).all()
    assert torch.equal(out[:25], alone)


def test_layer_graph_replay():
    """The layer captured once follows its inputs, with eager runs of other sizes between the replays."""
    say("layer graph replay")
    b = binding()
    rng = np.random.default_rng(9)
    T, D, H, E, k = 24, 256, 272, 16, 2
    ops = _layer_operands(rng, T, D, H, E)
    other = _layer_operands(rng, 300, D, H, E)
    _layer(b, *ops, k)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = _layer(b, *ops, k)
    for rep in range(3):
        ops[0].copy_(dev(rng.standard_normal((T, D)).astype(np.float32)))
        _layer(b, *other, k)
        want = _layer(b, *ops, k)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for got, w in zip(res, want):
            assert torch.equal(got, w), rep


@pytest.mark.parametrize("T", [8, 6000])
def test_router_graph_replay(T):
    """Routing, plan, combination and the gradients in one captured graph; two graphs side by side."""
    say("router graph replay", T)
    b = binding()
    rng = np.random.default_rng(T)
    E, k, N = 96, 4, 264

    def make():
        x = torch.empty((T, E), device=DEV)
        y = dev(rng.standard_normal((T * k, N)).astype(np.float32))
        d = dev(rng.standard_normal((T, N)).astype(np.float32))
        d_y = torch.zeros_like(y)

        def run():
            ids, w = b.expert_route(x, k, b.SCORE_SOFTMAX)
            plan = b.expert_plan(ids, E)
            out = b.expert_combine(y, plan[2], w)
            _, d_w = b.expert_combine_backward(d, y, plan[2], w, d_y=d_y)
            return (ids, w, *plan, out, d_y, d_w, b.expert_route_backward(x, ids, d_w, b.SCORE_SOFTMAX))

        return x, run

    sets = []
    for _ in range(2):
        x, run = make()
        x.normal_()
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = run()
        sets.append((x, run, g, res))
    streams = [torch.cuda.Stream() for _ in sets]
    for rep in range(3):
        want = []
        for x, run, _, _ in sets:
            x.normal_()
            want.append([t.clone() for t in run()])
        torch.cuda.synchronize()
        for (_, _, g, _), s in zip(sets, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, _, res), wanted in zip(sets, want):
            for got, w in zip(res, wanted):
                assert torch.equal(got, w), rep


def test_refusals():
    say("refusals")
    b = binding()
    x = torch.zeros((4, 16), device=DEV)
    with pytest.raises(ValueError):
        b.expert_route(x, 17)
    with pytest.raises(ValueError):
        b.expert_route(x, 0)
    with pytest.raises(ValueError):
        b.expert_route(x[:, ::2], 2)
    with pytest.raises(TypeError):
        b.expert_route(x.double(), 2)
    with pytest.raises(ValueError):
        b.expert_route(x, 2, bias=torch.zeros(15, device=DEV))
    with pytest.raises(b.MXGemmError):
        b.expert_route(x, 2, score=5)
    with pytest.raises(b.MXGemmError):
        b.expert_route(x, 4, groups=8, top_groups=1)
    with pytest.raises(b.MXGemmError):
        b.expert_route(x[:0], 2)
    with pytest.raises(b.MXGemmError):
        b.expert_route(torch.zeros((2, 1040), device=DEV), 2)
    ids, w = b.expert_route(x, 2)
    with pytest.raises(TypeError):
        b.expert_plan(ids.long(), 16)
    with pytest.raises(b.MXGemmError):
        b.expert_plan(ids, 1025)
    with pytest.raises(b.MXGemmError):
        b.expert_plan(ids[:0], 16)
    with pytest.raises(ValueError):
        b.expert_route_backward(x, ids[:2].contiguous(), w)
    with pytest.raises(ValueError):
        b.expert_route_backward(x, ids, w[:, :1].contiguous())
    y = torch.zeros((8, 32), device=DEV)
    with pytest.raises(ValueError):
        b.expert_combine(y, ids, w[:2])
    with pytest.raises(ValueError):
        b.expert_combine(y, ids, w, out_type=4)
    with pytest.raises(TypeError):
        b.expert_combine(y, ids.float(), w)
    with pytest.raises(ValueError):
        b.expert_combine_backward(torch.zeros((4, 31), device=DEV), y, ids, w)
    with pytest.raises(TypeError):
        b.expert_combine_backward(torch.zeros((4, 32), device=DEV), y, ids, w, d_y=y.bfloat16())
