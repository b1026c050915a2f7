"""The root-mean-square norm with a residual and an 8-bit output, and its
gradients, against the 64-bit forms."""
import pytest
import torch

import fp8_ref as ref
from gpu_util import binding, say
from test_gpu_fp8 import DEV, TYPES, U, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert binding().mxgemm_device_supported()
    yield


def sum_error(K):
    """Relative error of a sum of K squares in fp32: a lane adds at most max(128, K / 64)
    of them in a row, and 6 + 16 partial sums are joined."""
    return (max(128, K / 64) + 24) * U


def rel_y(K):
    """Of y: half the sum's, the division, root and reciprocal (4), two products."""
    return 0.5 * sum_error(K) + 6 * U


def step_of(t):
    """Distance of E4M3 values around t (64 bits)."""
    e = torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -10))).clamp_min(-6.0)
    return torch.exp2(e - 3)


def check_codes(quant, q, s, y, K):
    """Codes and scales of y (64 bits), which the call has up to rel_y."""
    bn = binding()
    rows = y.shape[0]
    e = rel_y(K)
    if quant == bn.QUANT_INT8:
        amax = y.abs().amax(-1)
        want = torch.where(amax > 0, (amax / 127).clamp_min(2.0 ** -126), amax)
        assert bool(((s.double() - want).abs() <= (e + 2 * U) * want).all())
        off = (q.double() * s.double()[:, None] - y).abs()
        assert bool((off <= s.double()[:, None] * 0.5 * (1 + 1e-6) + e * y.abs()).all())
        return
    if quant == bn.QUANT_MXFP8:
        amax = y.abs().view(rows, K // 32, 32).amax(-1)
        lo, hi = (torch.floor(torch.log2((amax * f).clamp_min(2.0 ** -300))).clamp(-119, 135) - 8 for f in (1 - 2 * e, 1 + 2 * e))
        got = s.double() - 127
        assert bool(((got == lo) | (got == hi)).all())
        scale = torch.exp2(got).repeat_interleave(32, -1)
    else:
        amax = ref.block_amax(y, 1)
        if quant == bn.QUANT_FP8:
            want = torch.where(amax > 0, (amax / 448).clamp_min(2.0 ** -126), amax)
            assert bool(((s.double() - want).abs() <= (e + 2 * U) * want).all())
        else:
            lo, hi = (ref.scale_of((amax * f).float(), True).double() for f in (1 - 2 * e, 1 + 2 * e))
            assert bool(((s.double() == lo) | (s.double() == hi)).all())
        scale = ref.expand(s.double(), rows, K, 1)
    zero = scale == 0
    t = y / torch.where(zero, 1.0, scale)
    off = (ref.decode(q) - t.clamp(-448, 448)).abs()
    # half a step of the values at t, or of those just above it where rounding of y led there
    tol = torch.maximum(step_of(t), step_of(t * (1 + 4 * e))) / 2 + (e + 3 * U) * t.abs()
    assert bool((torch.where(zero, ref.decode(q).abs(), (off - tol).clamp_min(0)) == 0).all())


SIZES = [(1, 32), (3, 64), (5, 96), (7, 512), (2, 544), (33, 1024), (1, 4096), (16, 2080), (4, 8192), (3, 14336), (300, 608),
         (2, 32768), (1, 65568), (2, 131072), (4099, 128)]


@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("quant", [0, 1, 2, 3, 4])
def test_norm(rows, K, kind, quant):
    say("norm", rows, K, kind, quant)
    bn = binding()
    g = gen(rows + K + quant)
    t = TYPES[kind]
    x = (randn(g, rows, K) * torch.exp2(torch.randint(-6, 4, (rows, 1), generator=g, device=DEV).float())).to(t)
    r = randn(g, rows, K).to(t) if (rows + quant) % 2 else None
    w = (1 + 0.2 * randn(g, K)).to(TYPES[(kind + quant) % 3])
    q, s, h, y, rstd = bn.rmsnorm_quantize(x, w, residual=r, quant=quant, eps=1e-5, with_y=quant % 2 == 0)
    if r is None:
        assert h is x
    else:
        assert torch.equal(h, (x.float() + r.float()).to(t))
    rstd_r, y_r = ref.norm(h, w, 1e-5)
    assert bool(((rstd.double() - rstd_r).abs() <= rstd_r * (0.5 * sum_error(K) + 4 * U)).all())
    if quant == 0:
        assert q is None and s is None
    else:
        check_codes(quant, q, s, y_r, K)
    if y is not None:
        tol = y_r.abs() * (rel_y(K) + torch.finfo(t).eps / 2 * (1 + 1e-3)) + (2.0 ** -25 if kind == 2 else 2.0 ** -140)
        assert bool(((y.double() - y_r).abs() <= tol).all())


@pytest.mark.parametrize("quant", [1, 2, 3, 4])
def test_norm_odd_length(quant):
    """K a multiple of 16 alone (not of 32 or 128)."""
    say("norm odd length", quant)
    bn = binding()
    for K in (16, 48, 144, 2064, 16400):
        if quant == bn.QUANT_MXFP8:
            with pytest.raises(bn.MXGemmError):
                bn.rmsnorm_quantize(randn(gen(K), 5, K), torch.ones(K, device=DEV), quant=quant)
            continue
        for kind in (0, 1):
            x = randn(gen(K), 5, K).to(TYPES[kind])
            q, s, _, _, _ = bn.rmsnorm_quantize(x, torch.ones(K, device=DEV), quant=quant)
            check_codes(quant, q, s, ref.norm(x, torch.ones(K, device=DEV), 1e-6)[1], K)


@pytest.mark.parametrize("quant", [1, 2, 3, 4])
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_norm_specials(quant, kind):
    """Rows of zeros (eps 0: NaN), of one value, with a NaN or an infinity, and blocks whose weights
    are zero; the other rows are as without them."""
    say("norm specials", quant, kind)
    bn = binding()
    K = 384
    x = randn(gen(quant), 8, K).to(TYPES[kind])
    w = torch.ones(K, device=DEV)
    w[128:256] = 0.0
    eps = 2.0 ** -20                    # of which root and reciprocal are exact
    want = bn.rmsnorm_quantize(x, w, quant=quant, eps=eps)
    z = x.clone()
    z[1] = 0
    z[2, 5] = float("nan")
    z[3, 300] = float("inf")
    z[4] = 0
    z[4, 17] = 1.0
    q, s, _, _, rstd = bn.rmsnorm_quantize(z, w, quant=quant, eps=eps)
    for i in (0, 5, 6, 7):
        assert torch.equal(q[i], want[0][i]) and torch.equal(s[i], want[1][i])
    assert not (q[1:4] if quant == 1 else q[1:4] & 127).any() and rstd[1] == 1024.0 and torch.isnan(rstd[2]) and rstd[3] == 0.0
    nan = torch.isnan(s) if quant != bn.QUANT_MXFP8 else s == 255
    assert nan[2].all() and not nan[1].any() and not nan[4].any()
    assert bool(nan[3]) if quant == 1 else bool(nan[3, 300 // (32 if quant == 4 else 128)]) and not bool(nan[3, 0])   # inf * 0 in its block alone
    assert int((q[4] if quant == 1 else q[4] & 127).ne(0).sum()) == 1
    _, s, _, _, rstd = bn.rmsnorm_quantize(z, w, quant=quant, eps=0.0)
    assert rstd[1] == float("inf")
    nan = torch.isnan(s) if quant != bn.QUANT_MXFP8 else s == 255
    assert nan[1].all()


def test_norm_in_place():
    """h may be the residual or x."""
    say("norm in place")
    bn = binding()
    for K in (256, 4096, 70000 // 32 * 32):
        x, r = randn(gen(1), 9, K).bfloat16(), randn(gen(2), 9, K).bfloat16()
        w = randn(gen(3), K).bfloat16()
        want = bn.rmsnorm_quantize(x, w, residual=r)
        for which in (0, 1):
            x2, r2 = x.clone(), r.clone()
            got = bn.rmsnorm_quantize(x2, w, residual=r2, h=(x2, r2)[which])
            assert got[2].data_ptr() == (x2, r2)[which].data_ptr()
            for p, q in zip(want, got):
                assert (p is None and q is None) or torch.equal(p, q)


def check_dx(dx, dy, h, w, rstd, dh=None):
    """In fp32: c is a sum of K products (as the squares of the forward pass, with 3
    more roundings a term) times 1 / K; dx has 6 more; half a step of its type."""
    r = rstd.double()[:, None]
    hat, p = h.double() * r, dy.double() * w.double()
    c = (p * hat).mean(-1, keepdim=True)
    want = r * (p - hat * c)
    err = r * (p.abs() * 6 * U + hat.abs() * ((p * hat).abs().mean(-1, keepdim=True) * (sum_error(h.shape[1]) + 3 * U) + c.abs() * 6 * U))
    if dh is not None:
        want = want + dh.double()
        err = err + U * want.abs()
    tol = err + torch.finfo(h.dtype).eps / 2 * (want.abs() + err) + (2.0 ** -25 if h.dtype == torch.float16 else 2.0 ** -140)
    off = (dx.double() - want).abs()
    say("  dx error / bound %.3g" % (off / tol).max().item())
    assert bool((off <= tol).all())


def test_norm_rows_past_4_gib():
    say("norm rows past 4 GiB")
    bn = binding()
    rows, K = 2 ** 23 + 5, 288
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 2 ** 22 + 1, rows - 1], device=DEV)
    x[at] = randn(gen(9), 3, K).bfloat16()
    w = torch.ones(K, device=DEV)
    q, s, _, _, rstd = bn.rmsnorm_quantize(x, w)
    p = bn.rmsnorm_quantize(x[at], w)
    assert torch.equal(q[at], p[0]) and torch.equal(s[at], p[1]) and torch.equal(rstd[at], p[4])
    assert int((s != 0).any(-1).sum()) == 3
    d_x, d_w = bn.rmsnorm_backward(x, x, w, rstd)
    check_dx(d_x[at], x[at], x[at], w, rstd[at])
    assert int((d_x != 0).any(-1).sum()) == 3
    # three terms that are not zero: 4 roundings a term, 2 of their sum
    term = x[at].double() * (x[at].double() * rstd[at].double()[:, None])
    assert bool(((d_w.double() - term.sum(0)).abs() <= 6 * U * term.abs().sum(0)).all())


BACK = [(64, 2048), (65, 2048), (64, 16), (63, 2064), (1, 16), (3, 64), (5, 96), (7, 528), (33, 1024), (1, 4096), (17, 2064), (300, 608), (4, 8192), (3, 14336), (2, 32768),
        (2, 65552), (1, 131072), (5000, 128), (2049, 4096), (257, 8208),
        (1, 49152), (1, 49168), (2, 24576), (3, 16384), (8, 6144), (9, 5456), (24, 2048), (25, 2048), (64, 768), (65, 752), (2, 48)]


@pytest.mark.parametrize("rows,K", BACK)
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_backward(rows, K, kind):
    """Errors in fp32: c is a sum of K products (as the squares above, with 3 more
    roundings a term) times 1 / K; dx has 6 more; dw a sum over the rows, 4 a term."""
    say("norm backward", rows, K, kind)
    bn = binding()
    g = gen(rows + K)
    t = TYPES[kind]
    h, dy = randn(g, rows, K).to(t), randn(g, rows, K).to(t)
    dh = randn(g, rows, K).to(t) if rows % 2 else None
    w = (1 + 0.2 * randn(g, K)).to(TYPES[(kind + rows) % 3])
    rstd, _ = ref.norm(h, w, 1e-6)
    rstd = rstd.float()
    dx, dw = bn.rmsnorm_backward(dy, h, w, rstd, d_h=dh)
    check_dx(dx, dy, h, w, rstd, dh)
    hat = h.double() * rstd.double()[:, None]
    term = dy.double() * hat
    off, tol = (dw.double() - term.sum(0)).abs(), term.abs().sum(0) * (rows + 4) * U
    say("  dw error / bound %.3g" % (off / tol).max().item())
    assert bool((off <= tol).all())


def test_backward_in_place():
    say("norm backward in place")
    bn = binding()
    for rows, K in ((40, 512), (40, 4096), (40, 70000 // 16 * 16), (3000, 512)):
        g = gen(K)
        h, dy, dh = (randn(g, rows, K).bfloat16() for _ in range(3))
        w = randn(g, K)
        rstd = ref.norm(h, w, 1e-6)[0].float()
        want = bn.rmsnorm_backward(dy, h, w, rstd, d_h=dh)
        h2 = dh.clone()
        got = bn.rmsnorm_backward(dy, h, w, rstd, d_h=h2, d_x=h2)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_backward_specials():
    """A NaN stays in its row of dx and its column of dw, an infinite rstd in its row."""
    say("norm backward specials")
    bn = binding()
    g = gen(1)
    h, dy, w = randn(g, 20, 256), randn(g, 20, 256), randn(g, 256)
    rstd = ref.norm(h, w, 1e-6)[0].float()
    want = bn.rmsnorm_backward(dy, h, w, rstd)
    dy[3, 7] = float("nan")
    dx, dw = bn.rmsnorm_backward(dy, h, w, rstd)
    assert torch.isnan(dx[3]).all() and torch.isnan(dw[7])
    assert torch.equal(dx[:3], want[0][:3]) and torch.equal(dx[4:], want[0][4:])
    assert torch.equal(dw[:7], want[1][:7]) and torch.equal(dw[8:], want[1][8:])


def test_graph_replay_and_streams():
    say("graph replay norm")
    bn = binding()
    g = gen(3)
    x, r = randn(g, 500, 1024).bfloat16(), randn(g, 500, 1024).bfloat16()
    w = randn(g, 1024).bfloat16()
    dy = randn(g, 500, 1024).bfloat16()

    def work(stream=None):
        q, s, h, y, rstd = bn.rmsnorm_quantize(x, w, residual=r, with_y=True, stream=stream)
        return (q, s, h, y, rstd) + bn.rmsnorm_backward(dy, h, w, rstd, d_h=y, stream=stream)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for _ in range(4):
        x.copy_(randn(g, 500, 1024))
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


def test_binding_refusals():
    bn = binding()
    x, w = randn(gen(1), 4, 64), torch.ones(64, device=DEV)
    q = torch.empty(4, 64, dtype=torch.uint8, device=DEV)
    for call in (lambda: bn.rmsnorm_quantize(x, w[:32]), lambda: bn.rmsnorm_quantize(x, w, residual=x[:2]),
                 lambda: bn.rmsnorm_quantize(x, w, quant=7), lambda: bn.rmsnorm_quantize(x, w, h=x.clone()),
                 lambda: bn.rmsnorm_quantize(x, w, quant=0, q=q), lambda: bn.rmsnorm_quantize(x.t(), w),
                 lambda: bn.rmsnorm_quantize(x, w, eps=-1.0), lambda: bn.rmsnorm_backward(x, x, w, w[:3]),
                 lambda: bn.rmsnorm_backward(x[:2], x, w, w[:4]), lambda: bn.rmsnorm_backward(x, x, w, w[:4], d_h=x[:1])):
        with pytest.raises((ValueError, bn.MXGemmError)):
            call()
    for call in (lambda: bn.rmsnorm_quantize(x, w.double()), lambda: bn.rmsnorm_quantize(x, w, residual=x.half()),
                 lambda: bn.rmsnorm_quantize(x, w, quant=1, q=q), lambda: bn.rmsnorm_backward(x.half(), x, w, w[:4])):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("rows,K", [(64, 256), (33, 4096), (9, 8192), (6, 8208), (5, 14336), (4, 16384), (5, 16416), (3, 131072)])
@pytest.mark.parametrize("kind", [1, 2])
def test_rstd_and_y_are_rounded_once(rows, K, kind):
    """16-bit rows: the sum of the squares is exact in 64 bits up to 2^-52 a term of it,
    so rstd is the fp32 value next to the real one (2^-40 of a step apart at most), and
    so is y: its product with the rest of rstd has 2^-47."""
    say("norm rounded once", rows, K, kind)
    g = gen(K)
    x, w = randn(g, rows, K).to(TYPES[kind]), randn(g, K).to(TYPES[kind]).float()
    _, _, _, y, rstd = binding().rmsnorm_quantize(x, w, quant=0)
    real, _ = ref.norm(x, w, 1e-6)
    assert bool(((rstd.double() - real).abs() <= real * (U * (1 + 2.0 ** -16))).all())
    # fp32 rows, so that y is seen as it is
    _, _, _, y, rstd = binding().rmsnorm_quantize(x.float(), w, quant=0)
    want = x.double() * ref.norm(x.float(), w, 1e-6)[0][:, None] * w.double()
    assert bool(((y.double() - want).abs() <= want.abs() * (U * (1 + 2.0 ** -16)) + 2.0 ** -149).all())
