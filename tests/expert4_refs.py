"""The 4-bit operators and the layer of few tokens in 64 bits on the CPU, from their definitions (tests only)."""
import torch

from tests import expert_refs as refs

CODES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def exponent(top, most):
    """e of the smallest 2^e with top <= most * 2^e, at least -126; 0 where top is 0."""
    m, e = torch.frexp(top)
    mm, me = torch.frexp(torch.tensor(float(most), dtype=torch.float64))
    s = (e - me + (m > mm).to(e.dtype)).clamp(min=-126)
    return torch.where(top > 0, s, torch.zeros_like(s))


def two(e):
    return torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e)


def e2m1(v):
    """Nearest code's magnitude with the sign of v (|v| <= 6): of two as near, the even code."""
    d = (v.abs().unsqueeze(-1) - CODES).abs()
    d[..., 1::2] += 1e-12     # an odd code loses a tie; bf16 and fp32 inputs over a power of two are no nearer to one
    return torch.where(v < 0, -1.0, 1.0).double() * CODES[d.argmin(-1)]


def blocks(v, width=256, size=32):
    p = torch.zeros(*v.shape[:-1], refs.pad(v.shape[-1], width), dtype=torch.float64)
    p[..., : v.shape[-1]] = v
    return p.unflatten(-1, (-1, size))


def layout(e):
    """Exponents [.., rows, Cp/32] as scale bytes [.., Cp/256, rows, 8]."""
    return (e + 127).to(torch.uint8).unflatten(-1, (-1, 8)).transpose(-2, -3).contiguous()


def quantize(v):
    """float64 [.., rows, c] -> (values over the scales [.., rows, Cp], scale bytes as they are kept)."""
    p = blocks(v)
    e = exponent(p.abs().amax(-1), 6)
    return e2m1(p / two(e).unsqueeze(-1)).flatten(-2), layout(e)


def codes(b):
    """float64 [.., Cp] of the packed values."""
    q = b.q.cpu().view(torch.uint8)
    v = torch.stack((q & 15, q >> 4), -1).flatten(-2).long()
    return torch.cat([CODES, -CODES])[v]


def scales(b):
    """float64 [.., rows, Cp/32]; NaN where marked."""
    return b.scale.cpu().double().transpose(-2, -3).flatten(-2)


def values(b):
    return (codes(b).unflatten(-1, (-1, 32)) * scales(b).unsqueeze(-1)).flatten(-2)[..., : b.cols]


def cut(x, sx, w, sw):
    """What the instruction may cut off a sum of 8-bit x [r, k] by w [n, k]: in each eight consecutive products seven
    lose less than 2^-13 of the largest 2^(exponent of x + exponent of w); a subnormal's exponent is -6 (x) and 0 (w),
    above its value."""
    def top(v, s, low):
        p = torch.zeros(v.shape[0], refs.pad(v.shape[1], 8), dtype=torch.float64)
        p[:, : v.shape[1]] = torch.maximum(v.abs(), low * s)
        return p.unflatten(-1, (-1, 8)).amax(-1)
    return 7 * 2.0 ** -13 * top(x, sx, 2.0 ** -6) @ top(w, sw, 1.0 if sw is not None else 0.0).t()


def added(x, w, more=8):
    """fp32 additions of the products' groups of eight, of the instructions' results and of `more` partial sums, each
    off by at most 2^-23 of the sum of magnitudes."""
    return (refs.pad(x.shape[1], 256) // 8 + more) * 2.0 ** -23 * (x.abs() @ w.abs().t())


def rounded(y, off):
    """Bound of a result rounded to bf16 once (half a step: 2^-8 of the value) that was off by `off` before."""
    return 2.0 ** -8 * y.abs() + (1 + 2.0 ** -8) * off


def spread(s, size, cols):
    return s.repeat_interleave(size, -1)[..., :cols]


def quantize8(v):
    """e4m3 with a scale per 1 x 32: (values [r, c], scale of each [r, c])."""
    p = blocks(v, 32)
    s = two(exponent(p.abs().amax(-1), 448)).unsqueeze(-1)
    q = refs.e4m3(p / s) * s
    return q.flatten(-2)[:, : v.shape[1]], spread(s.squeeze(-1), 32, v.shape[1])
