"""The 4-bit operators and the layer of few tokens at the ends of their contract: the most channels, every operand of a
backward pass, the inputs that only a conversion instruction sees."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import expert4_refs as refs4
from tests import expert_refs as refs
from tests.test_gpu_experts4 import BF, call_with_act, instances, normal, read, same4, u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import load_balance_planning_amd as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def small(mp):
    layer = mp.Layer(mp.make_config(8, 8, 1, 1, 1, 8, 0))
    yield layer
    layer.close()


# ---- the most channels ------------------------------------------------------------

def test_products_of_the_most_channels(mp):
    """2^20 channels, and up to 2048 instances, of which 30 are there: they are of the first 8 of 1024 experts, and only
    those have matrices."""
    rows, E, B, n, k, used, count = 6148, 1024, 1024, 1 << 20, 256, 8, 30
    print("products4 of %d channels, %d experts" % (n, E), flush=True)
    layer = mp.Layer(mp.make_config(rows, E, 1, 4, 1, 8, B), cooc=False)
    dev = layer.device
    rng = np.random.RandomState(0)
    loads = rng.multinomial(rows, rng.dirichlet(np.full(count, 0.5)))
    plan, off, spans = instances(mp, layer, loads, rng.randint(0, used, count))
    x = layer.quantize4(normal(1, rows, k).to(dev))
    w = torch.randn(used, n, k, device=dev, dtype=BF, generator=torch.Generator(device=dev).manual_seed(2)) * 2 ** -4
    wb = layer.quantize_weights4(w)
    del w
    y = torch.full((rows, n), 7.0, dtype=BF, device=dev)
    p = lambda t: t.data_ptr()
    mp.moex4_matmul(layer.handle, plan.struct(), p(off), 4, p(x.q), p(x.scale), p(wb.q), p(wb.scale), n, k, p(y),
                    torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert layer.status() == 0
    at = torch.cat([torch.arange(300), torch.from_numpy(rng.randint(0, n, 400)), torch.arange(n - 300, n)])
    q, s = wb.q.view(torch.uint8)[:, at.to(dev)], wb.scale.view(torch.uint8)[:, :, at.to(dev)].contiguous()
    wv = refs4.values(mp.Blocks4(q.contiguous(), s.view(torch.float8_e8m0fnu), k))
    xv, got, seen = refs4.values(x), y[:, at.to(dev)].cpu().double(), 0
    for e, a, z in spans:
        want = xv[a:z] @ wv[e].t()
        assert ((got[a:z] - want).abs() <= refs4.rounded(want, refs4.added(xv[a:z], wv[e]))).all()
        seen += z - a
    assert seen == rows
    layer.close()


def test_more_tiles_than_the_limit_are_refused(mp):
    """2^26 rows by 2^20 channels: refused on the host, whatever the memory."""
    layer = mp.Layer(mp.make_config(1 << 21, 32, 32, 1, 1, 8, 0), cooc=False, topk_val=False)
    plan, off, _ = instances(mp, layer, [8], [0])
    s, p, some = plan.struct(), off.data_ptr(), torch.zeros(64, dtype=torch.uint8, device=layer.device).data_ptr()
    for bits in (4, 8):
        assert mp.lib().moex4_matmul(layer.handle, ctypes.byref(s), p, bits, some, some, some, some, 1 << 20, 256, some,
                                     None) == mp.MOE_ERR_UNSUPPORTED
    layer.close()


# ---- inputs that only a conversion instruction sees --------------------------------

def every_value(e, most):
    """Blocks of 32 whose scale is 2^e: the largest, most * 2^e, then bf16 values of both signs, all there are from it
    down to 2^-7 of it (bf16's subnormals among them), and some below."""
    top = torch.tensor(most * 2.0 ** e, dtype=torch.float64)
    bits = torch.arange(1, 0x7f80, dtype=torch.int32).to(torch.int16).view(BF).double()
    v = bits[(bits <= top) & (bits >= top * 2.0 ** -7)]
    v = torch.cat([v, bits[bits < top * 2.0 ** -7][-300::7], torch.zeros(1, dtype=torch.float64)])
    v = torch.cat([v, -v])
    v = torch.cat([v, torch.zeros(-len(v) % 31, dtype=torch.float64)]).view(-1, 31)
    return torch.cat([top.expand(len(v), 1), v], 1).to(BF)


def borders():
    """The rows of the row quantizer's border test: largest magnitudes on both sides of 6 * 2^e, the type's extremes,
    halves between two codes, signed zeros."""
    rows = []
    for e in (-126, -120, -20, 0, 3, 100, 124):
        for top in (6, 5.96875, 6.03125, 7, 4, 1.0):
            r = torch.linspace(-1, 1, 32) * top * 2.0 ** e
            r[0] = top * 2.0 ** e
            rows.append(r)
    halves = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    rows += [torch.cat([halves, -halves, halves * (1 + 2.0 ** -7), halves * (1 - 2.0 ** -8)]).clamp(max=6.0),
             torch.full((32,), torch.finfo(BF).max), torch.full((32,), -torch.finfo(BF).tiny), torch.full((32,), 9.2e-41),
             torch.zeros(32), -torch.zeros(32)]
    return torch.stack(rows).to(BF)


@pytest.mark.parametrize("e", [None, -126, -125, -121, -60, 0, 77, 125])
def test_matrices_at_the_borders(mp, small, e):
    """Matrices divide in the conversion itself, rows in fp32 before it: the same codes and scales, in both layouts."""
    x = borders() if e is None else every_value(e, 6.0)
    n = len(x)
    print("matrices at the borders, exponent %s, %d blocks" % (e, n), flush=True)
    q, s = refs4.quantize(x.double())
    same4(small.quantize4(x.to(small.device)), q, s)
    w = x.unsqueeze(0).to(small.device)
    plain, both = small.quantize_weights4(w), small.quantize_weights4(w, transposed=True)
    same4(plain, q.unsqueeze(0), s.unsqueeze(0))
    same4(both[0], q.unsqueeze(0), s.unsqueeze(0))
    same4(both[1], *refs4.quantize(x.double().t().unsqueeze(0).contiguous()))
    turned = small.quantize_weights4(w.transpose(1, 2).contiguous(), transposed=True)
    same4(turned[1], q.unsqueeze(0), s.unsqueeze(0))


def one_layer(mp, T, H, f):
    layer = mp.Layer(mp.make_config(T, 1, 1, 1, 1, H, 0), cooc=False)
    dev = layer.device
    return layer, torch.zeros(T, 1, dtype=torch.int32, device=dev), torch.ones(T, 1, device=dev)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("e", [None, -126, -125, -121, -60, 0, 77, 118])
def test_few_tokens_rows_at_the_borders(mp, bits, e):
    """The rounding of the hidden rows, seen through activations that are 32 times the rounded values: a gate of 32 from
    a block of its own (its sigmoid is 1 in fp32), and every other value by itself as `up`."""
    x = borders() if e is None else every_value(e, 448.0)
    x[x.double().abs() >= 2.0 ** 127] = 0    # 32 times the value has to be in range, by a matrix of 2^-6
    T, blocks = 64, -(-len(x) // 64)
    f = 32 * blocks
    H = f + 32
    print("rows at the borders, exponent %s, %d blocks, %d bits" % (e, len(x), bits), flush=True)
    hidden = torch.zeros(T, H, dtype=BF)
    hidden[:, :f] = torch.cat([x, torch.zeros(T * blocks - len(x), 32, dtype=BF)]).view(T, f)
    hidden[:, f] = 32
    layer, idx, weight = one_layer(mp, T, H, f)
    for small_one in (0, 6):     # the matrices' values that pass `up` on: 1, and 2^-6 for the largest
        w1 = torch.zeros(1, 2 * f, H)
        w1[0, :f, f] = 1
        w1[0, f:, :f].fill_diagonal_(2.0 ** -small_one)
        quant = layer.quantize_weights4 if bits == 4 else layer.quantize_weights
        q1, q2 = quant(w1.to(BF).to(layer.device)), quant(torch.zeros(1, H, f, dtype=BF, device=layer.device))
        _, act, _ = call_with_act(mp, layer, hidden.to(layer.device), idx, weight, q1, q2, f)
        v, _ = refs4.quantize8(hidden.double())
        want, _ = refs4.quantize8(32 * 2.0 ** -small_one * v[:, :f])
        fits = (want.abs() < 2.0 ** 127).view(T, -1, 32).all(-1, keepdim=True).expand(-1, -1, 32).reshape(T, f)
        assert fits.any() and torch.equal(torch.where(fits, act, 0.0), torch.where(fits, want, 0.0))
        # nothing but the row's own rounding where the activation's scale leaves the value as it was
        same = fits & ((32 * 2.0 ** -small_one * v[:, :f]) == want)
        assert (same | ~fits).all() or small_one
    assert layer.status() == 0
    layer.close()


# ---- scales at the ends of their range ----------------------------------------------

def with_scales(mp, b, rows, regions, codes_to):
    """Matrices whose scale bytes, by 128 columns, are drawn from regions[i] = (rows' begin, end, bytes), with the values
    of other columns zero in those rows; under bytes from 250 on values stay below 2, so that they are in bf16's range."""
    E, g = b.q.shape[0], torch.Generator().manual_seed(1)
    four = isinstance(b, mp.Blocks4)
    q = b.q.cpu().view(torch.uint8).clone()
    per = 64 if four else 128                         # bytes of 128 columns
    if four:
        flat = torch.full((E, rows, 8 * b.scale.shape[1]), 127, dtype=torch.uint8)
    else:
        flat = torch.full(tuple(b.scale.shape), 127, dtype=torch.uint8)
    for begin, end, col, choices in regions:
        part = torch.zeros_like(q[:, begin:end])
        kept = q[:, begin:end, per * col: per * (col + 1)]
        if max(choices) >= 250:
            kept = kept & codes_to
        part[..., per * col: per * (col + 1)] = kept
        q[:, begin:end] = part
        pick = torch.tensor(choices, dtype=torch.uint8)
        if four:
            flat[:, begin:end, 4 * col: 4 * col + 4] = pick[torch.randint(len(choices), (E, end - begin, 4), generator=g)]
        else:
            assert begin % 128 == 0 and (end % 128 == 0 or end == rows)
            lead = slice(begin // 128, -(-end // 128))
            flat[:, lead, col] = pick[torch.randint(len(choices), flat[:, lead, col].shape, generator=g)]
    s = flat.unflatten(-1, (-1, 8)).transpose(-2, -3).contiguous() if four else flat
    dev = b.q.device
    return type(b)(q.to(dev).view(b.q.dtype), s.to(dev).view(torch.float8_e8m0fnu), b.cols)


def in_bf16(v):
    """Values as the first product takes them."""
    return v.to(BF).double()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("extreme", ["gate", "up", "w2"])
def test_few_tokens_at_the_ends_of_the_scales(mp, bits, extreme):
    """Scale bytes 0, 1, 2, 253 and 254 of either matrix, with operands on the other side that bring the sums back: a
    third of the channels each sum over columns under small, middling and large scales.

    The first product takes values as bf16, whose smallest step is 2^-133: what 8-bit values lose to that is in the
    reference too (to nearest even).  Else the bounds are those of the layer's other tests."""
    T, E, k, H, f = 9, 4, 2, 384, 384
    print("scales at the ends: %s, %d bits" % (extreme, bits), flush=True)
    layer = mp.Layer(mp.make_config(T, E, k, 1, 1, H, 0), cooc=False)
    dev = layer.device
    g = torch.Generator().manual_seed(5)
    idx = torch.rand(T, E, generator=g).argsort(-1)[:, :k].to(torch.int32).to(dev)
    weight = torch.rand(T, k, generator=g).to(dev)
    quant = layer.quantize_weights4 if bits == 4 else layer.quantize_weights
    q1, q2 = quant(normal(6, E, 2 * f, H).to(dev)), quant(normal(7, E, H, f).to(dev))
    # e2m1 codes below 2 and e4m3 values below 2 (their exponents keep less than the bias)
    low = 0xbb if bits == 4 else 0xbf
    low_bytes, high_bytes = [0, 1, 2], [253, 254]
    hidden = normal(8, T, H)
    middle = [127 - 2] if bits == 4 else [127 - 8]
    small_up = lambda b: [b - 4] if bits == 4 else [b - 10]
    if extreme == "w2":
        # activations of 2^100, 1 and 2^-100: by `up`, from the middle columns
        r1 = [(0, f, 1, middle)] + [(f + 128 * i, f + 128 * (i + 1), 1, small_up(127 + s)) for i, s in enumerate((100, 0, -100))]
        r2 = [(0, 128, 0, low_bytes), (128, 256, 1, middle), (256, 384, 2, high_bytes)]
        q1, q2 = with_scales(mp, q1, 2 * f, r1, low), with_scales(mp, q2, H, r2, low)
    else:
        hidden = hidden.double()
        hidden[:, :128] *= 2.0 ** (118 if bits == 4 else 112)
        hidden[:, 256:] *= 2.0 ** -126
        hidden = hidden.to(BF)
        at = 0 if extreme == "gate" else f
        r1 = [(at, at + 128, 0, low_bytes), (at + 128, at + 256, 1, middle), (at + 256, at + 384, 2, high_bytes),
              (f - at, f - at + f, 1, middle)]
        q1 = with_scales(mp, q1, 2 * f, r1, low)
    out, act, s = call_with_act(mp, layer, hidden.to(dev), idx, weight, q1, q2, f)
    assert layer.status() == 0
    x, _ = refs4.quantize8(hidden.double())
    (w1v, _), (w2v, s2) = read(q1, 2 * f), read(q2, H)
    w1v, x = in_bf16(w1v), in_bf16(x)
    assert torch.isfinite(w1v).all() and torch.isfinite(x).all()
    idx_, weight_ = idx.cpu().long(), weight.cpu().double()
    want, off = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(idx_[t, j])
            y, dy = w1v[e] @ x[t], refs4.added(x[t:t + 1], w1v[e])[0]
            assert (y.abs() > 8 * dy).double().mean() > 0.9     # (the sums are there)
            a = refs.swiglu(y[None])[0]
            silu = y[:f] / (1 + torch.exp(-y[:f]))
            da = 1.1 * dy[:f] * (y[f:].abs() + dy[f:]) + silu.abs() * dy[f:] + 2.0 ** -19 * a.abs()
            got, each = act[t * k + j], s[t * k + j]
            step = torch.maximum(2.0 ** -4 * (a.abs() + da), 2.0 ** -10 * each)
            err = (got - a).abs()
            assert torch.isfinite(got).all() and (err <= step + da).all(), float((err / (step + da)).max())
            top = refs4.blocks(got, 32).abs().amax(-1)
            assert (top <= 448 * refs4.blocks(each, 32).amax(-1)).all()
            w, got2, each2 = weight_[t, j], got[None], each[None]
            # eight products of zeros have nothing to cut off
            live = (w2v[e].view(H, -1, 8) != 0).any(-1).repeat_interleave(8, -1)
            want[t] += w * (w2v[e] @ got)
            off[t] += w * (refs4.added(got2, w2v[e]) + refs4.cut(got2, each2, w2v[e], s2[e] * live)
                           + (k + 16) * 2.0 ** -23 * (got2.abs() @ w2v[e].abs().t()))[0]
    err = (out.double() - want).abs()
    assert torch.isfinite(want).all() and (err <= refs4.rounded(want, off)).all(), float((err - refs4.rounded(want, off)).max())
    assert (want != 0).double().mean() > 0.9
    layer.close()


# ---- the gated activation to its stated bound ---------------------------------------

def test_the_gated_activation_is_within_its_bound(mp, small):
    """silu(gate) * up within 2^-20 of its value: pairs whose exact value lies just past a border between two codes, by
    2^-20 of it at the least, get the code of their side.

    What the kernel's steps lose, in units of 2^-24: exponential and reciprocal 2 each, five roundings 1 each, 9 in all,
    2^-20.8."""
    bits = torch.arange(0, 0x8000, dtype=torch.int32).to(torch.int16).view(BF)
    g = bits[(bits.float() >= 2.0 ** -30) & (bits.float() <= 88.5)].double()
    g = torch.cat([g, -g])
    silu = g / (1 + torch.exp(-g))
    close = []
    for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        u = (border / silu).to(BF)
        v = silu * u.double()
        gap = ((v - border) / border).abs()
        ok = (gap > 2.0 ** -20) & torch.isfinite(u) & (u.abs() > 1e-37)
        near = gap[ok].argsort()[:400]
        close.append(torch.stack([g[ok][near], u.double()[ok][near]], 1))
        print("border %g: nearest 2^%.1f, 20th 2^%.1f" % (border, gap[ok].min().log2(), gap[ok].sort().values[20].log2()), flush=True)
    pairs = torch.cat(close)
    pairs = torch.cat([pairs, pairs[: -len(pairs) % 31]]).view(-1, 31, 2)
    top = torch.tensor([8.0, 0.703125], dtype=torch.float64).expand(len(pairs), 1, 2)   # 5.62: the scale is 1
    pairs = torch.cat([top, pairs], 1)
    y = torch.cat([pairs[..., 0], pairs[..., 1]], 1).to(BF)
    assert torch.equal(y.double(), torch.cat([pairs[..., 0], pairs[..., 1]], 1))
    b = small.swiglu4(y.to(small.device))
    torch.cuda.synchronize()
    q, s = refs4.quantize(refs.swiglu(y.double()))
    assert torch.equal(u8(b.scale), s) and (s[0, :, 0] == 127).all()
    assert torch.equal(refs4.codes(b), q)


# ---- the largest sizes ---------------------------------------------------------------

@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,E,k,H,f", [(64, 32, 32, 8, 1 << 20), (64, 4, 2, 1 << 20, 24)])
def test_the_widest_layers_of_few_tokens(mp, T, E, k, H, f, bits):
    """2^31 bytes of activations, and rows of 2^20: tokens of a full call as by themselves.  (The shares of the second
    product are others then: fp32 sums in another order, bf16's half step each way, and activations whose fp32 value
    lies at a border of e4m3.)"""
    print("experts T=%d E=%d k=%d H=%d f=%d bits=%d" % (T, E, k, H, f, bits), flush=True)
    layer, one = (mp.Layer(mp.make_config(t, E, k, 1, 1, H, 0), cooc=False) for t in (T, 1))
    dev = layer.device
    g = torch.Generator(device=dev).manual_seed(1)
    n = lambda *s, by: torch.randn(*s, generator=g, device=dev, dtype=BF) * by
    quant = layer.quantize_weights4 if bits == 4 else layer.quantize_weights
    w1 = quant(n(E, 2 * f, H, by=H ** -0.5))
    w2 = quant(n(E, H, f, by=f ** -0.5))
    hidden = n(T, H, by=1.0)
    idx = torch.rand(T, E, generator=g, device=dev).argsort(-1)[:, :k].to(torch.int32)
    weight = torch.rand(T, k, generator=g, device=dev)
    out = layer.experts(hidden, weight, w1, w2, topk_idx=idx).float()
    assert torch.isfinite(out).all() and (out != 0).float().mean() > 0.9
    for t in (0, T // 2, T - 1):
        alone = one.experts(hidden[t:t + 1], weight[t:t + 1], w1, w2, topk_idx=idx[t:t + 1]).float()
        assert torch.allclose(alone[0], out[t], rtol=2.0 ** -7, atol=2e-3 * float(out[t].abs().max())), t
    assert layer.status() == 0 and one.status() == 0
    layer.close()
    one.close()


def test_the_widest_rows_and_matrices(mp, small):
    """2^24 columns, and matrices of 2^24 rows: each block as elsewhere."""
    dev, cols = small.device, 1 << 24
    x = torch.randn(2, cols, device=dev, dtype=BF, generator=torch.Generator(device=dev).manual_seed(1))
    rows, lines = small.quantize4(x), small.quantize4(x.view(-1, 256))
    assert torch.equal(u8(rows.q).view(-1, 128), u8(lines.q))
    assert torch.equal(u8(rows.scale).transpose(0, 1).reshape(-1, 8), u8(lines.scale)[0])
    assert torch.equal(small.values4(rows).view(-1, 256), small.values4(lines))
    wide = small.swiglu4(torch.cat([x[:1], x[1:]], 1))      # one row: gate, then up
    parts = small.swiglu4(torch.cat([x[0].view(-1, 256), x[1].view(-1, 256)], 1))
    assert torch.equal(u8(wide.q).view(-1, 128), u8(parts.q))
    assert torch.equal(u8(wide.scale).view(-1, 8), u8(parts.scale)[0])
    del lines, parts, wide
    one, turned = small.quantize_weights4(x[:1].t().contiguous().view(1, cols, 1), transposed=True)
    alone, row = small.quantize4(x[0].view(cols, 1)), small.quantize4(x[:1])
    assert torch.equal(u8(one.q)[0], u8(alone.q)) and torch.equal(u8(one.scale)[0], u8(alone.scale))
    assert torch.equal(u8(turned.q)[0], u8(row.q)) and torch.equal(u8(turned.scale)[0], u8(row.scale))
