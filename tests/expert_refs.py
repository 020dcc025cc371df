"""The expert-layer operators in 64 bits on the CPU, from their definitions (tests only)."""
import torch

BLK = 128


def pad(n, m=BLK):
    return -(-n // m) * m


# ---- router -------------------------------------------------------------------

def scores(x, kind):
    if kind == "sigmoid":
        return torch.where(x == -torch.inf, torch.zeros_like(x), 1 / (1 + torch.exp(-x)))
    top = x.amax(-1, keepdim=True)
    e = torch.where(x == -torch.inf, torch.zeros_like(x), torch.exp(x - torch.where(top == -torch.inf, 0.0, top)))
    return e / e.sum(-1, keepdim=True).clamp(min=1e-300)


def select(x, bias, kind, k, n_group, topk_group, group_top):
    """Indices int64 [T][k]: expert by expert, group by group, ties to the lower one."""
    s = scores(x, kind)
    choice = s if bias is None else s + bias
    key = x.clone() if bias is None else choice.clone()
    T, E = x.shape
    if n_group > 1:
        best = choice.view(T, n_group, -1).sort(dim=-1, descending=True).values[..., :group_top].sum(-1)
        for t in range(T):
            keep = sorted(range(n_group), key=lambda q: (-best[t, q].item(), q))[:topk_group]
            for q in range(n_group):
                if q not in keep:
                    key[t, q * (E // n_group):(q + 1) * (E // n_group)] = -torch.inf
    return torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :k]


def gate_weights(x, idx, kind, renorm, scale):
    s = scores(x, kind).gather(1, idx)
    return scale * (s / (s.sum(-1, keepdim=True) + 1e-20) if renorm else s)


# ---- blocks -------------------------------------------------------------------

def e4m3(v):
    """Nearest e4m3 value (|v| <= 448), ties to even, in float64."""
    m, e = torch.frexp(v.abs().clamp(min=2.0 ** -6))   # v = m 2^e, 0.5 <= m < 1: steps of 2^(e - 4)
    step = torch.ldexp(torch.ones_like(v), e - 4)
    return torch.round(v / step) * step


def block_exponent(top):
    """e of the smallest 2^e with top <= 448 * 2^e, at least -126; 0 where top is 0."""
    m, e = torch.frexp(top)
    s = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126)
    return torch.where(top > 0, s, torch.zeros_like(s))


def quantize(v, rows=1):
    """float64 [.., n, c] in blocks of rows x 128: (e4m3 values [.., n, padded c], scale bytes [.., n/rows, S])."""
    n, c = v.shape[-2:]
    p = torch.zeros(*v.shape[:-2], pad(n, rows), pad(c), dtype=torch.float64)
    p[..., :n, :c] = v
    p = p.unflatten(-1, (-1, BLK)).unflatten(-3, (-1, rows))
    e = block_exponent(p.abs().amax(-1).amax(-2))
    q = e4m3(p / torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e)[..., None, :, None])
    q = q.flatten(-2).flatten(-3, -2)[..., :n, :]
    bytes_ = torch.full((*e.shape[:-1], pad(e.shape[-1], 4)), 127, dtype=torch.uint8)
    bytes_[..., : e.shape[-1]] = (e + 127).to(torch.uint8)
    return q, bytes_


def values(b, n, rows=1):
    """float64 [.., n, cols] that Blocks stand for."""
    q, s = b.q.cpu().double()[..., : b.cols], b.scale.cpu().double()
    if rows > 1:
        s = s.repeat_interleave(rows, -2)[..., :n, :]
    return q * s.repeat_interleave(BLK, -1)[..., : b.cols]


# ---- products -----------------------------------------------------------------

def block_max(v):
    """Largest magnitude of every 1 x 128 block of float64 [n, c]."""
    p = torch.zeros(v.shape[0], pad(v.shape[1]), dtype=torch.float64)
    p[:, : v.shape[1]] = v.abs()
    return p.unflatten(-1, (-1, BLK)).amax(-1)


def product(x, w):
    """x [r, k] times w [n, k] transposed, and the bound of the kernel's error.

    bf16 rounds by at most 2^-8 |y|.  The 8-bit matrix instruction aligns the 128 products of a step to the
    largest and drops what falls below its accumulator: each product loses at most 2^-17 of the largest, so a step
    is off by at most 2^-10 max|x| max|w| of the block.  The fp32 additions of the K/128 steps and of four partial
    sums add 2^-24 of a partial sum each, at most (K/128 + 4) 2^-24 sum|x w|."""
    y = x @ w.t()
    steps = pad(x.shape[1]) // BLK
    off = 2.0 ** -10 * block_max(x) @ block_max(w).t() + (steps + 4) * 2.0 ** -24 * (x.abs() @ w.abs().t())
    return y, 2.0 ** -8 * y.abs() + (1 + 2.0 ** -8) * off


def outer(dy, x):
    """dy [r, n] transposed times x [r, k], and the bound: bf16 rounding, and fp32 sums of r exact products in the
    matrix instruction (each addition off by at most 2^-23 of the sum of magnitudes so far)."""
    y = dy.t() @ x
    off = (dy.shape[0] + 8) * 2.0 ** -23 * (dy.abs().t() @ x.abs())
    return y, 2.0 ** -8 * y.abs() + (1 + 2.0 ** -8) * off


def swiglu(y):
    f = y.shape[1] // 2
    g, u = y[:, :f], y[:, f:]
    return g / (1 + torch.exp(-g)) * u


def swiglu_grad(y, da):
    f = y.shape[1] // 2
    g, u = y[:, :f], y[:, f:]
    s = 1 / (1 + torch.exp(-g))
    return torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1)
