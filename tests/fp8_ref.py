"""The E4M3 products with a scale per block of 128, their weights' gradients and
the norm with an 8-bit output, from their definitions: fp32 where a rule is
stated in fp32 (scales and codes), else 64 bits.  Torch on any device."""
import torch

BLOCK = 128


def values():
    """The 127 finite E4M3 values of codes 0x00 .. 0x7E: bias 7, 3 mantissa bits."""
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(v, dtype=torch.float64)


def decode(q):
    """Codes (uint8) to 64 bits; 0x7F and 0xFF are NaN."""
    v = torch.cat([values(), torch.tensor([float("nan")], dtype=torch.float64)]).to(q.device)
    x = v[(q & 127).long()]
    return torch.where(q >= 128, -x, x)


def encode(t):
    """Codes of 64-bit values: the nearest E4M3 value, ties to the even code, saturated."""
    v = values().to(t.device)
    size = t.abs().clamp_max(448.0)
    middle = (v[1:] + v[:-1]) / 2
    code = torch.searchsorted(middle, size)            # first middle >= size
    tie = (code < 126) & (middle[code.clamp_max(125)] == size)
    code = torch.where(tie & (code % 2 == 1), code + 1, code)
    sign = torch.signbit(t).to(torch.uint8) * 128
    return code.to(torch.uint8) | sign


def expand(s, rows, K, block_rows):
    return s.repeat_interleave(block_rows, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :K]


def block_amax(x, block_rows):
    rows, K = x.shape
    full = torch.zeros(-(-rows // block_rows) * block_rows, -(-K // BLOCK) * BLOCK, dtype=x.dtype, device=x.device)
    full[:rows, :K] = x.abs()
    return full.view(full.shape[0] // block_rows, block_rows, -1, BLOCK).amax((1, 3))


def divide(a, b):
    """The fp32 quotient: 64 bits rounded to 24 once more are the nearest, as 53 >= 2 * 24 + 2."""
    return (a.double() / b.double()).float()


def scale_of(amax, pow2):
    """fp32 amax -> fp32 scale."""
    s = divide(amax, torch.full_like(amax, 448.0)).clamp_min(2.0 ** -126)
    if pow2:
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    return torch.where(amax == 0, torch.zeros_like(s), s)


def quantize(x, block_rows=1, pow2=False):
    """fp32 rows x K -> (codes, scales)."""
    rows, K = x.shape
    bad = block_amax((~torch.isfinite(x)).float(), block_rows) > 0
    amax = block_amax(torch.where(torch.isfinite(x), x, torch.zeros_like(x)), block_rows)
    s = scale_of(amax, pow2)
    by = expand(torch.where((s > 0) & ~bad, s, torch.ones_like(s)), rows, K, block_rows)
    t = divide(torch.where(torch.isfinite(x), x, torch.zeros_like(x)), by)
    q = encode(t.double())
    q = torch.where(expand(bad.to(torch.uint8), rows, K, block_rows) != 0, torch.zeros_like(q), q)
    return q, torch.where(bad, torch.full_like(s, float("nan")), s)


def dequantize(q, s, block_rows=1):
    rows, K = q.shape
    return decode(q) * expand(s.double(), rows, K, block_rows)


def product(a_q, a_s, b_q, b_s):
    """(sum, and what its error is measured by): the sum in 64 bits; sum over blocks
    of the largest product a block can have (with its scales); sum of |products|."""
    a, b = dequantize(a_q, a_s), dequantize(b_q, b_s, BLOCK)
    top_a, top_b = block_amax(a, 1), block_amax(b, 1)
    return a @ b.t(), top_a @ top_b.t(), a.abs() @ b.abs().t()


def gelu(y):
    return y * torch.special.ndtr(y)


def bf16_grad(d, x):
    """dW and sum |terms|, x rounded to bf16."""
    x = x.to(torch.bfloat16).double()
    return d.double().t() @ x, d.double().abs().t() @ x.abs()


def norm(h, w, eps):
    """(rstd, y) of rows h."""
    h, w = h.double(), w.double()
    rstd = 1.0 / torch.sqrt((h * h).mean(-1) + eps)
    return rstd, h * rstd[:, None] * w


def norm_backward(dy, h, w, eps, dh=None):
    """Gradients by the formula (64 bits), rstd from h."""
    dy, h, w = dy.double(), h.double(), w.double()
    rstd, _ = norm(h, w, eps)
    hat = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - hat * (g * hat).mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
    return dx, (dy * hat).sum(0)


def rows_of_experts(offsets, rows):
    """offsets kept inside 0 .. rows and never falling, as ranges per expert."""
    out, top = [], max(0, min(int(offsets[0]), rows))
    for o in offsets[1:]:
        hi = max(top, min(int(o), rows))
        out.append((top, hi))
        top = hi
    return out
