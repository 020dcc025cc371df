"""4-bit quantization, its values, the gated activation and the experts' products in 4 bits, and the layer of few
tokens, against tests/expert4_refs.py (64 bits, CPU)."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import expert4_refs as refs4
from tests import expert_refs as refs

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


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


def normal(seed, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(BF)


def u8(t):
    return t.cpu().view(torch.uint8)


def same4(got, q, s):
    torch.cuda.synchronize()
    assert torch.equal(u8(got.scale), s)
    assert torch.equal(refs4.codes(got), q)


# ---- quantization ---------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 256), (257, 130), (33, 264), (64, 1000), (9, 2688), (1, 16384),
                                       (2048, 8), (70, 520), (2, 9), (7, 1001), (17, 2047), (1, 15), (4, 17), (3, 257)])
def test_rows(mp, small, rows, cols):
    print("quantize4 rows %d x %d" % (rows, cols), flush=True)
    x = normal(rows + cols, rows, cols)
    x[0] *= 1e-30
    if rows > 2:
        x[1] = 0
        x[2] *= 1e30
    b = small.quantize4(x.to(small.device))
    same4(b, *refs4.quantize(x.double()))
    v = small.values4(b).cpu()
    assert v.shape == (rows, cols) and torch.equal(v.double(), refs4.values(b))


def test_rows_at_the_borders(mp, small):
    """Largest magnitudes on both sides of 6 * 2^e, the type's extremes, halves between two codes, signed zeros."""
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
    x = torch.stack(rows).to(BF)
    b = small.quantize4(x.to(small.device))
    same4(b, *refs4.quantize(x.double()))
    want = refs4.values(b)
    # bf16's subnormals end at 2^-133: 0.5 * 2^-126 is one of them.  bf16's largest, 255/256 of 2^128, is 3.98 of its
    # block's scales 2^126, and so the code 4: 2^128, past bf16's range, is infinite.
    assert (want == 2.0 ** 128).any()
    assert torch.equal(small.values4(b).cpu().double(), torch.where(want == 2.0 ** 128, torch.inf, want))


@pytest.mark.parametrize("value", [torch.inf, -torch.inf, torch.nan])
def test_marked_blocks(mp, small, value):
    """A block with an infinity or a NaN is marked, kept as zeros, and every sum over it is NaN; others are as without."""
    x = normal(1, 8, 300)
    clean = small.quantize4(x.to(small.device))
    x[3, 200] = value
    b = small.quantize4(x.to(small.device))
    s, c = refs4.scales(b), refs4.scales(clean)
    assert torch.isnan(s[3, 6]) and int((s != c).sum()) == 1
    q, qc = refs4.codes(b), refs4.codes(clean)
    assert (q[3, 192:224] == 0).all()
    qc[3, 192:224] = 0
    assert torch.equal(q, qc)
    v = small.values4(b).cpu()
    assert torch.isnan(v[3, 192:224]).all() and int(torch.isnan(v).sum()) == 32
    w = small.quantize_weights4(normal(2, 8, 16, 300).to(small.device))
    plan, off, _ = instances(mp, small, [8], [0])
    y = small.matmul4(b, w, plan=plan, inst_offset=off).cpu()
    assert torch.isnan(y[3]).all() and torch.isfinite(y[[0, 1, 2, 4, 5, 6, 7]]).all()
    w = normal(2, 8, 16, 300)
    w[0, 5, 100] = value
    wb, wt = small.quantize_weights4(w.to(small.device), transposed=True)
    assert torch.isnan(refs4.scales(wb)[0, 5, 3]) and int(torch.isnan(refs4.scales(wb)).sum()) == 1
    assert torch.isnan(refs4.scales(wt)[0, 100, 0]) and int(torch.isnan(refs4.scales(wt)).sum()) == 1
    for rows in (clean, small.quantize(normal(1, 8, 300).to(small.device))):
        y = small.matmul4(rows, wb, plan=plan, inst_offset=off).cpu()
        assert torch.isnan(y[:, 5]).all() and int(torch.isnan(y).sum()) == 8
    x8 = small.quantize(x.to(small.device))
    y = small.matmul4(x8, small.quantize_weights4(normal(2, 8, 16, 300).to(small.device)), plan=plan, inst_offset=off)
    y = y.cpu()
    assert torch.isnan(y[3]).all() and int(torch.isnan(y).sum()) == 16


@pytest.mark.parametrize("E,n,k", [(1, 1, 1), (2, 128, 128), (3, 130, 200), (2, 760, 1000), (5, 64, 384), (1, 257, 129),
                                   (2, 512, 640), (2, 33, 1001), (1, 500, 7), (3, 129, 255), (2, 9, 1), (1, 3, 2399),
                                   (1, 384, 300), (1, 300, 384)])
def test_matrices(mp, small, E, n, k):
    print("quantize4 matrices %d x %d x %d" % (E, n, k), flush=True)
    w = normal(E + n + k, E, n, k, scale=0.02)
    w[0, : min(n, 128), : min(k, 128)] = 0
    if n > 200:
        w[0, 200] *= 1e20
    b, t = small.quantize_weights4(w.to(small.device), transposed=True)
    same4(b, *refs4.quantize(w.double()))
    same4(t, *refs4.quantize(w.double().transpose(1, 2).contiguous()))
    assert t.cols == n and b.cols == k
    alone = small.quantize_weights4(w.to(small.device))
    assert torch.equal(u8(alone.q), u8(b.q)) and torch.equal(u8(alone.scale), u8(b.scale))
    for blocks in (b, t):
        assert torch.equal(small.values4(blocks).cpu().double(), refs4.values(blocks))


@pytest.mark.parametrize("rows,f", [(1, 1), (3, 20), (130, 128), (5, 384), (33, 1000), (64, 2688), (7, 77), (1024, 136),
                                    (2, 5), (9, 131), (17, 63)])
def test_gated_activation(mp, small, rows, f):
    """The value in fp32 is within 2^-19 of the exact one (expf and its argument, a division, two products): the scale is
    that of a largest magnitude so near, and each value within half a step of e2m1 (1/5 of it at the most, 0.25 scales
    below 2 of them, so 0.25 scales or a fifth)."""
    print("swiglu4 %d x %d" % (rows, f), flush=True)
    y = normal(rows + f, rows, 2 * f, scale=2.0)
    y[0, 0], y[0, f] = -60.0, 3.0
    if rows > 2:
        y[1] = 0
    b = small.swiglu4(y.to(small.device))
    want = refs.swiglu(y.double())
    got, s = refs4.values(b), refs4.scales(b)
    top = refs4.blocks(want).abs().amax(-1)
    lo, hi = (refs4.two(refs4.exponent(top * (1 + d), 6)) for d in (-2.0 ** -19, 2.0 ** -19))
    assert ((s == lo) | (s == hi)).all()
    each = refs4.spread(s, 32, f)
    ratio = want.abs() / each
    half = torch.where(ratio < 2, 0.25, torch.where(ratio < 4, 0.5, 1.0)) * each
    assert ((got - want).abs() <= half * (1 + 2.0 ** -10) + 2.0 ** -18 * want.abs()).all()
    assert (refs4.codes(b)[:, f:] == 0).all()


def test_gated_activation_far_out(mp, small):
    """Gates to the ends of their range, a block each.  Below -88.72 the sigmoid is 0 (its exponential leaves fp32); the
    bounds are those above."""
    pairs = [(-88.5, 60), (-88.0, 60), (-87.0, 120), (-60.0, 3), (-20.25, 0), (-1e-3, 0), (-1e-30, 30), (0.0, 0), (1e-30, 0),
             (5.0, 100), (20.0, 0), (88.0, -90), (88.5, 0), (100.0, 0), (128.0, 0), (200.0, 0), (1e4, 0), (3e38, -1),
             (-89.0, 0), (-100.0, 120), (-200.0, 0), (-1e10, 0), (-3.3e38, 0)]
    g = torch.tensor([p[0] for p in pairs]).to(BF)[:, None].expand(-1, 32)
    u = (2.0 ** torch.tensor([float(p[1]) for p in pairs])).to(BF)[:, None].expand(-1, 32)
    y = torch.cat([g, u], 1).contiguous()
    b = small.swiglu4(y.to(small.device))
    want = torch.where(g.double() < -88.72, 0.0, refs.swiglu(y.double()))
    got, s = refs4.values(b), refs4.scales(b)
    each = refs4.spread(s, 32, 32)
    ratio = want.abs() / each
    half = torch.where(ratio < 2, 0.25, torch.where(ratio < 4, 0.5, 1.0)) * each
    assert ((got - want).abs() <= half * (1 + 2.0 ** -10) + 2.0 ** -18 * want.abs()).all()
    assert ((want == 0) | (ratio > 2.99)).all() and (got[want == 0] == 0).all()
    odd = y.clone()
    inf = float("inf")
    odd[0, 3], odd[1, 5], odd[2, 40], odd[3, 0], odd[4, 33] = inf, -inf, float("nan"), float("nan"), -inf
    marked = (u8(small.swiglu4(odd.to(small.device)).scale)[0, :, 0] == 255).nonzero().flatten().tolist()
    assert marked == [0, 1, 2, 3, 4]


def test_unaligned_rows(mp, small):
    """bf16 inputs and results that start 2 bytes past a 16-byte boundary."""
    x = normal(4, 20, 264)
    buf = torch.empty(20 * 264 + 1, dtype=BF, device=small.device)
    view = buf[1:].view(20, 264).copy_(x)
    b = small.quantize4(view)
    same4(b, *refs4.quantize(x.double()))
    a, c = small.swiglu4(view), small.swiglu4(x.to(small.device))
    assert torch.equal(u8(a.q), u8(c.q)) and torch.equal(u8(a.scale), u8(c.scale))
    same4(small.quantize_weights4(buf[1:].view(1, 20, 264)), *[t.unsqueeze(0) for t in refs4.quantize(x.double())])
    out = torch.empty(20 * 264 + 1, dtype=BF, device=small.device)
    assert torch.equal(small.values4(b, out=out[1:].view(20, 264)).cpu().double(), refs4.values(b))


def test_no_rows(mp, small):
    dev = small.device
    b = small.quantize4(torch.empty(0, 200, dtype=BF, device=dev))
    assert b.q.shape == (0, 128) and b.scale.shape == (1, 0, 8)
    assert small.swiglu4(torch.empty(0, 200, dtype=BF, device=dev)).q.shape == (0, 128)
    w, wt = small.quantize_weights4(torch.empty(0, 4, 200, dtype=BF, device=dev), transposed=True)
    assert w.q.shape == (0, 4, 128) and wt.q.shape == (0, 200, 128)
    assert small.values4(b).shape == (0, 200) and small.values4(w).shape == (0, 4, 200)
    torch.cuda.synchronize()
    assert small.status() == 0


# ---- products -------------------------------------------------------------------

def instances(mp, layer, loads, experts):
    """A plan of the given instance loads and experts: (PlanBuffers, inst_offset, spans)."""
    cap, dev = int(layer.sizes.inst_cap), layer.device
    off = np.concatenate([[0], np.cumsum(loads)])
    fill = lambda v, n: torch.tensor(list(v) + [-1] * (n - len(v)), dtype=torch.int32, device=dev)
    plan = mp.PlanBuffers(torch.tensor([len(loads)], dtype=torch.int32, device=dev), fill(experts, cap), None, None,
                          None, None, None, None)
    return plan, fill(off.tolist(), cap + 1), [(int(e), int(a), int(b)) for e, a, b in zip(experts, off[:-1], off[1:])]


def layer_for(mp, rows, E, B=0):
    R = 4 if E > 1024 else 1  # at most 1024 experts and replica slots a rank
    return mp.Layer(mp.make_config(rows, E, 1, R, 1, 8, B), cooc=False)


def check_products(mp, loads, experts, E, n, k, B=0, seed=0):
    """Rows in 4 and in 8 bits, and the input gradient with the transposed matrices, of one set of instances."""
    rows = int(sum(loads))
    print("products4 loads=%s.. E=%d n=%d k=%d" % (list(loads)[:8], E, n, k), flush=True)
    layer = layer_for(mp, rows, E, B)
    dev = layer.device
    plan, off, spans = instances(mp, layer, loads, experts)
    x, w = normal(seed + 1, rows, k), normal(seed + 2, E, n, k, scale=0.05)
    dy = normal(seed + 3, rows, n, scale=1e-3)
    x[rows // 2] *= 300  # rows, and blocks of a row, of different scales
    x[:, k // 2:] *= 0.01
    x4, x8, d8 = layer.quantize4(x.to(dev)), layer.quantize(x.to(dev)), layer.quantize(dy.to(dev))
    wb, wt = layer.quantize_weights4(w.to(dev), transposed=True)
    kw = dict(plan=plan, inst_offset=off)
    got = {}
    for name, a, b, cols in (("x4", x4, wb, n), ("x8", x8, wb, n), ("dx", d8, wt, k)):
        y = torch.full((rows, cols), 7.0, dtype=BF, device=dev)
        layer.matmul4(a, b, out=y, **kw)
        got[name] = y.cpu().double()
        assert torch.equal(layer.matmul4(a, b, **kw).cpu(), y.cpu())
    torch.cuda.synchronize()
    assert layer.status() == 0
    x4v, x8v, d8v, wv, wtv = refs4.values(x4), refs.values(x8, rows), refs.values(d8, rows), refs4.values(wb), refs4.values(wt)
    sx, sd = (refs4.spread(b.scale.cpu().double(), 128, b.cols) for b in (x8, d8))
    sw, st = refs4.spread(refs4.scales(wb), 32, k), refs4.spread(refs4.scales(wt), 32, n)
    for e in range(E):
        at = torch.cat([torch.arange(a, b) for f, a, b in spans if f == e] + [torch.arange(0)]).long()
        for name, a, b, more in (("x4", x4v, wv, None), ("x8", x8v, wv, (sx, sw)), ("dx", d8v, wtv, (sd, st))):
            want, off_ = a[at] @ b[e].t(), refs4.added(a[at], b[e])
            if more:
                off_ = off_ + refs4.cut(a[at], more[0][at], b[e], more[1][e])
            err, off_ = (got[name][at] - want).abs(), refs4.rounded(want, off_)
            assert (err <= off_).all(), "%s expert %d: %d of %d outside, worst excess %g" % (
                name, e, int((err > off_).sum()), err.numel(), float((err - off_).max()))
    layer.close()


CASES = [
    ([1], [0], 1, 1, 1, 0),
    ([1], [0], 1, 128, 128, 0),
    ([5, 0, 17, 1], [0, 1, 2, 3], 4, 130, 200, 0),
    ([0, 0, 33, 0], [0, 1, 2, 3], 4, 64, 128, 0),
    ([16, 15, 17, 64, 63, 65, 128, 127], list(range(8)), 8, 100, 72, 0),
    ([129, 256, 257, 3], [0, 1, 2, 3], 4, 384, 640, 0),
    ([40, 9, 70, 30, 22, 0], [0, 1, 2, 0, 2, 2], 3, 200, 136, 3),     # replicas of experts 0 and 2
    ([300, 2, 90], [0, 1, 2], 3, 257, 1000, 0),
    ([2] * 60 + [0] * 4, list(range(64)), 64, 72, 264, 0),
    ([700], [0], 1, 520, 312, 0),
    ([511, 513], [0, 1], 2, 256, 512, 0),
    ([31, 64, 1], [2, 0, 1], 3, 33, 17, 0),                           # instances out of expert order
    ([257, 300], [0, 1], 2, 300, 1300, 0),                            # an odd number of lines of 256
]


@pytest.mark.parametrize("loads,experts,E,n,k,B", CASES)
def test_products(mp, loads, experts, E, n, k, B):
    check_products(mp, loads, experts, E, n, k, B, seed=n + k)


def test_products_of_many_instances(mp):
    """A plan of 2048 experts and 1000 replicas, most of them empty."""
    rng = np.random.RandomState(0)
    E, B = 2048, 1000
    loads = rng.multinomial(900, rng.dirichlet(np.full(E + B, 0.1)))
    check_products(mp, loads, np.concatenate([np.arange(E), rng.permutation(E)[:B]]), E, 24, 40, B)


@pytest.mark.parametrize("n,k", [(24, 40), (520, 40)])
def test_tiles_of_many_instances(mp, n, k):
    """The same with 70000 rows: tiles whose lists of instances are the longest."""
    rng = np.random.RandomState(1)
    E, B = 2048, 1000
    loads = rng.multinomial(70000, rng.dirichlet(np.full(E + B, 0.3)))
    check_products(mp, loads, np.concatenate([np.arange(E), rng.permutation(E)[:B]]), E, n, k, B)


@pytest.mark.parametrize("loads,E,n,k", [
    ([4100, 4204], 2, 4000, 328), ([8192], 1, 4100, 700), ([300, 8000, 70], 3, 4096, 256),
    ([16500, 16400], 2, 2000, 4400),            # 256 x 256 for rows in 4 bits, an odd number of lines of 256
    ([20000, 130, 19990], 3, 1500, 650),        # 256 x 128 for both
    ([9000, 8000], 2, 700, 384)])
def test_products_in_the_largest_tiles(mp, loads, E, n, k):
    """Tiles of 256 x 128 and 256 x 256, several to a workgroup; rows at the tiles' ends and some others."""
    rows = sum(loads)
    print("products4 loads=%s E=%d n=%d k=%d" % (loads, E, n, k), flush=True)
    layer = layer_for(mp, rows, E)
    dev = layer.device
    plan, off, spans = instances(mp, layer, loads, list(range(E)))
    x, w = normal(1, rows, k), normal(2, E, n, k, scale=0.05)
    x[:, k // 2:] *= 0.01
    wb = layer.quantize_weights4(w.to(dev))
    wv, sw = refs4.values(wb), refs4.spread(refs4.scales(wb), 32, k)
    for b in (layer.quantize4(x.to(dev)), layer.quantize(x.to(dev))):
        y = torch.full((rows, n), 7.0, dtype=BF, device=dev)
        layer.matmul4(b, wb, plan=plan, inst_offset=off, out=y)
        y = y.cpu()
        assert torch.equal(layer.matmul4(b, wb, plan=plan, inst_offset=off).cpu(), y)
        four = isinstance(b, mp.Blocks4)
        xv = refs4.values(b) if four else refs.values(b, rows)
        sx = None if four else refs4.spread(b.scale.cpu().double(), 128, k)
        for e, a, z in spans:
            at = torch.tensor(sorted({t for t in [*range(a, a + 40), *range(a + 240, a + 270), *range(z - 40, z),
                                                  *range(a, z, max(37, (z - a) // 300))] if a <= t < z}))
            want, off_ = xv[at] @ wv[e].t(), refs4.added(xv[at], wv[e])
            if not four:
                off_ = off_ + refs4.cut(xv[at], sx[at], wv[e], sw[e])
            assert ((y[at].double() - want).abs() <= refs4.rounded(want, off_)).all()
    assert layer.status() == 0
    layer.close()


def test_any_scale_bytes(mp, small):
    """Scales from 2^-127 to 2^127 of rows, and of matrices, as the products and the values take them."""
    dev = small.device
    x, w = normal(1, 8, 256), normal(2, 8, 40, 256)
    xb, wb = small.quantize4(x.to(dev)), small.quantize_weights4(w.to(dev))
    xb.scale.copy_(torch.arange(64, dtype=torch.uint8).view(1, 8, 8).mul(4).clamp(max=254).to(dev).view(torch.float8_e8m0fnu))
    wb.scale.view(torch.uint8).fill_(127 - 20)
    plan, off, _ = instances(mp, small, [8], [0])
    y = small.matmul4(xb, wb, plan=plan, inst_offset=off).cpu().double()
    xv, wv = refs4.values(xb), refs4.values(wb)[0]
    want, bound = xv @ wv.t(), refs4.rounded(xv @ wv.t(), refs4.added(xv, wv))
    # results below bf16's normal numbers are off by half a subnormal step too, and fp32's sums by its own
    bound = bound + 2.0 ** -134 + 2.0 ** -140
    big = want.abs() < 2.0 ** 127
    assert big.any() and ((y - want).abs() <= bound)[big].all()
    v = small.values4(xb).cpu().double()
    far = xv.abs() >= torch.finfo(BF).max
    assert ((v - xv).abs() <= 2.0 ** -134)[~far].all() and torch.isinf(v[xv.abs() > 3.4e38]).all()


def test_a_bad_plan_sets_the_status_word(mp):
    layer = layer_for(mp, 40, 4)
    dev = layer.device
    w = layer.quantize_weights4(normal(2, 4, 24, 64).to(dev))
    for x in (layer.quantize4(normal(1, 40, 64).to(dev)), layer.quantize(normal(1, 40, 64).to(dev))):
        plan, off, _ = instances(mp, layer, [20, 20], [0, 9])
        y = torch.full((40, 24), 7.0, dtype=BF, device=dev)
        layer.matmul4(x, w, plan=plan, inst_offset=off, out=y)
        assert layer.status() == mp.MOE_STATUS_PLAN_CHECK and (y[20:] == 7).all() and (y[:20] != 7).any()
        for offs in ([0, 41, 40], [0, -1, 40], [30, 10, 40]):
            bad = torch.tensor(offs + [-1, -1], dtype=torch.int32, device=dev)
            plan, _, _ = instances(mp, layer, [20, 20], [0, 1])
            layer.matmul4(x, w, plan=plan, inst_offset=bad)
            assert layer.status() == mp.MOE_STATUS_PLAN_CHECK
        plan.n_inst.fill_(5)
        layer.matmul4(x, w, plan=plan, inst_offset=off)
        assert layer.status() == mp.MOE_STATUS_PLAN_CHECK
    layer.close()


# ---- the layer of few tokens ----------------------------------------------------

def few_layer(mp, T, E, k, H, f, bits, seed=0, hot=0.0):
    layer = mp.Layer(mp.make_config(T, E, k, 2 if E > 1024 else 1, 1, H, 0), cooc=False)
    dev = layer.device
    g = torch.Generator().manual_seed(seed)
    score = torch.randn(T, E, generator=g) - hot * torch.arange(E)
    top = torch.sort(score, dim=-1, descending=True)
    idx, weight = top.indices[:, :k].to(torch.int32).contiguous(), torch.softmax(top.values[:, :k], -1).contiguous()
    w1, w2 = normal(seed + 1, E, 2 * f, H, scale=H ** -0.5), normal(seed + 2, E, H, f, scale=f ** -0.5)
    quant = layer.quantize_weights4 if bits == 4 else layer.quantize_weights
    return layer, idx.to(dev), weight.to(dev), quant(w1.to(dev)), quant(w2.to(dev))


def read(b, rows):
    """float64 values and scales of matrices in either form."""
    if hasattr(b, "padded") and type(b).__name__ == "Blocks4":
        return refs4.values(b), refs4.spread(refs4.scales(b), 32, b.cols)
    s = b.scale.cpu().double().repeat_interleave(128, -2)[:, :rows, :]
    return refs.values(b, rows, 128), 2.0 ** -6 * refs4.spread(s, 128, b.cols)


def call_with_act(mp, layer, hidden, idx, weight, w1, w2, f):
    """Layer.experts with the activations kept: (out, act values [T*k, f], their scales)."""
    T, k = idx.shape
    fp, dev = mp.Blocks4.padded(f), layer.device
    work = torch.full((mp.moex4_experts_work(layer.handle, f),), 0xff, dtype=torch.uint8, device=dev)
    out = torch.full((T, hidden.shape[1]), 7.0, dtype=BF, device=dev)
    p = lambda t: t.data_ptr()
    mp.moex4_experts(layer.handle, p(hidden), p(idx), p(weight), 4 if isinstance(w1, mp.Blocks4) else 8, f, p(w1.q),
                     p(w1.scale), p(w2.q), p(w2.scale), p(work), p(out), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    act = work[: T * k * fp].view(T * k, fp)
    scale = work[T * k * fp: T * k * (fp + fp // 32)].view(T * k, fp // 32)
    assert (act[:, f:] == 0).all()
    s = torch.exp2(scale.cpu().double() - 127).repeat_interleave(32, -1)[:, :f]
    return out.cpu(), act.cpu().view(torch.float8_e4m3fn).double()[:, :f] * s, s


def check_few(mp, T, E, k, H, f, bits, seed=0, hot=0.0):
    print("experts T=%d E=%d k=%d H=%d f=%d bits=%d" % (T, E, k, H, f, bits), flush=True)
    layer, idx, weight, w1, w2 = few_layer(mp, T, E, k, H, f, bits, seed, hot)
    hidden = normal(seed + 3, T, H)
    if T > 2:
        hidden[1] = 0
        hidden[2, : H // 2] *= 1e4
    out, act, s = call_with_act(mp, layer, hidden.to(layer.device), idx, weight, w1, w2, f)
    x, _ = refs4.quantize8(hidden.double())
    (w1v, _), (w2v, s2) = read(w1, 2 * f), read(w2, H)
    idx_, weight_ = idx.cpu(), weight.cpu().double()
    want, off = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for e in sorted(set(idx_.flatten().tolist())):
        t, j = (idx_ == e).nonzero(as_tuple=True)
        y = x[t] @ w1v[e].t()
        dy = refs4.added(x[t], w1v[e])  # exact values in bf16: nothing is cut off here
        gate, up = y[:, :f], y[:, f:]
        a = refs.swiglu(y)
        silu = gate / (1 + torch.exp(-gate))
        # silu' is at most 1.1; the activation's own arithmetic is within 2^-19
        da = 1.1 * dy[:, :f] * (up.abs() + dy[:, f:]) + silu.abs() * dy[:, f:] + 2.0 ** -19 * a.abs()
        got, each = act[t * k + j], s[t * k + j]
        near = refs4.blocks(a, 32).abs(), refs4.blocks(da, 32)
        lo = refs4.two(refs4.exponent((near[0] - near[1]).clamp(min=0).amax(-1), 448))
        hi = refs4.two(refs4.exponent((near[0] + near[1]).amax(-1), 448))
        blk = refs4.blocks(each, 32).amax(-1)
        assert (((blk >= lo) & (blk <= hi)) | (near[0].amax(-1) <= near[1].amax(-1))).all()
        step = torch.maximum(2.0 ** -4 * (a.abs() + da), 2.0 ** -10 * each)
        err = (got - a).abs()
        assert (err <= step + da).all(), "activations of expert %d: worst excess %g" % (e, float((err - step - da).max()))
        wj = weight_[t, j][:, None]
        yj = got @ w2v[e].t()
        want.index_add_(0, t, wj * yj)
        off.index_add_(0, t, wj.abs() * (refs4.added(got, w2v[e]) + refs4.cut(got, each, w2v[e], s2[e])
                                         + (k + 16) * 2.0 ** -23 * (got.abs() @ w2v[e].abs().t())))
    err, bound = (out.double() - want).abs(), refs4.rounded(want, off)
    assert (err <= bound).all(), "%d of %d outside, worst excess %g" % (int((err > bound).sum()), err.numel(),
                                                                        float((err - bound).max()))
    again = layer.experts(hidden.to(layer.device), weight, w1, w2, topk_idx=idx)
    assert torch.equal(again.cpu(), out)
    assert layer.status() == 0
    layer.close()


FEW = [(1, 8, 2, 64, 32), (1, 1, 1, 1, 1), (2, 4, 4, 130, 33), (3, 8, 2, 257, 100), (7, 8, 2, 1000, 380), (16, 4, 2, 512, 256),
       (17, 3, 3, 384, 129), (33, 2, 1, 200, 64), (64, 2, 2, 136, 72), (64, 40, 8, 264, 160), (5, 100, 32, 72, 40),
       (64, 1, 1, 520, 200), (9, 16, 4, 2048, 768), (64, 128, 8, 96, 288), (1, 16, 8, 2047, 1001)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,E,k,H,f", FEW)
def test_few_tokens(mp, T, E, k, H, f, bits):
    check_few(mp, T, E, k, H, f, bits, seed=T + H + f, hot=0.3 if E > 3 else 0.0)


def test_few_tokens_of_many_experts(mp):
    """2048 experts and 32 of them a token: 2048 slots, and the largest lists in LDS; and with sixteen waves."""
    check_few(mp, 64, 2048, 32, 40, 24, 4, seed=3)
    check_few(mp, 16, 2048, 32, 40, 24, 4, seed=4)


def test_few_tokens_none(mp):
    layer = mp.Layer(mp.make_config(0, 4, 2, 1, 1, 64, 0), cooc=False)
    dev = layer.device
    w1, w2 = layer.quantize_weights4(normal(1, 4, 64, 64).to(dev)), layer.quantize_weights4(normal(2, 4, 64, 32).to(dev))
    out = layer.experts(torch.empty(0, 64, dtype=BF, device=dev), torch.empty(0, 2, device=dev), w1, w2)
    assert out.shape == (0, 64) and layer.status() == 0
    layer.close()


@pytest.mark.parametrize("bits", [4, 8])
def test_few_tokens_bad_indices(mp, bits):
    """An index outside the experts is left out and reported, as is a repeated one; other tokens are as before."""
    layer, idx, weight, w1, w2 = few_layer(mp, 6, 8, 2, 96, 64, bits, 5)
    hidden = normal(6, 6, 96).to(layer.device)
    good = layer.experts(hidden, weight, w1, w2, topk_idx=idx).cpu()
    assert layer.status() == 0
    for value in (8, -1, 2 ** 31 - 1, -2 ** 31):
        bad = idx.clone()
        bad[2, 1] = value
        got = layer.experts(hidden, weight, w1, w2, topk_idx=bad).cpu()
        assert layer.status() == mp.MOE_STATUS_BAD_TOPK
        rest = [0, 1, 3, 4, 5]
        assert torch.equal(got[rest], good[rest]) and torch.isfinite(got[2]).all() and not torch.equal(got[2], good[2])
    bad = idx.clone()
    bad[4, 1] = bad[4, 0]
    got = layer.experts(hidden, weight, w1, w2, topk_idx=bad).cpu()
    assert layer.status() == mp.MOE_STATUS_BAD_TOPK
    assert torch.equal(got[[0, 1, 2, 3, 5]], good[[0, 1, 2, 3, 5]])
    none = torch.full_like(idx, -1)
    assert (layer.experts(hidden, weight, w1, w2, topk_idx=none).cpu() == 0).all()
    assert layer.status() == mp.MOE_STATUS_BAD_TOPK
    layer.close()


@pytest.mark.parametrize("T,k", [(6, 3), (20, 4), (64, 8)])
def test_few_tokens_repeated_indices(mp, T, k):
    """Of a token's slots with the same expert the first counts: the others are as indices outside the experts."""
    layer, idx, weight, w1, w2 = few_layer(mp, T, 16, k, 200, 96, 4, T)
    hidden = normal(T, T, 200).to(layer.device)
    idx[1] = idx[1, 0]  # all of them
    idx[T - 2, k - 1] = idx[T - 2, 0]
    idx[T - 1, 2] = idx[T - 1, 1]
    seen = torch.zeros_like(idx, dtype=torch.bool)
    for j in range(1, k):
        seen[:, j] = (idx[:, :j] == idx[:, j:j + 1]).any(1)
    want = layer.experts(hidden, weight, w1, w2, topk_idx=idx.masked_fill(seen, -1)).cpu()
    assert layer.status() == mp.MOE_STATUS_BAD_TOPK
    got = layer.experts(hidden, weight, w1, w2, topk_idx=idx).cpu()
    assert layer.status() == mp.MOE_STATUS_BAD_TOPK
    assert torch.equal(got, want)
    layer.close()


@pytest.mark.parametrize("bits", [4, 8])
def test_few_tokens_not_finite(mp, bits):
    """A token with a NaN or an infinity is NaN throughout; others are as without it.  So is one with such a weight."""
    layer, idx, weight, w1, w2 = few_layer(mp, 20, 4, 2, 200, 64, bits, 9)
    hidden = normal(6, 20, 200)
    good = layer.experts(hidden.to(layer.device), weight, w1, w2, topk_idx=idx).cpu()
    for value in (torch.nan, torch.inf, -torch.inf):
        h = hidden.clone()
        h[7, 150] = value
        got = layer.experts(h.to(layer.device), weight, w1, w2, topk_idx=idx).cpu()
        rest = [t for t in range(20) if t != 7]
        assert torch.isnan(got[7]).all() and torch.equal(got[rest], good[rest])
    w = weight.clone()
    w[3, 1] = torch.nan
    got = layer.experts(hidden.to(layer.device), w, w1, w2, topk_idx=idx).cpu()
    assert torch.isnan(got[3]).all() and int(torch.isnan(got).any(-1).sum()) == 1
    w[3, 1] = 0.0
    assert torch.isfinite(layer.experts(hidden.to(layer.device), w, w1, w2, topk_idx=idx)).all()
    layer.close()


@pytest.mark.parametrize("bits", [4, 8])
def test_few_tokens_marked_matrices(mp, bits):
    """A marked block of a matrix makes NaN of what its expert's tokens sum over it, and of nothing else."""
    for which, at in (("w1", (1, 5, 40)), ("w1", (1, 64 + 5, 40)), ("w2", (1, 70, 33))):
        layer, idx, weight, w1, w2 = few_layer(mp, 12, 4, 2, 200, 64, bits, 9)
        dev = layer.device
        hidden = normal(6, 12, 200).to(dev)
        good = layer.experts(hidden, weight, w1, w2, topk_idx=idx).cpu()
        w = normal(10 if which == "w1" else 11, 4, *((128, 200) if which == "w1" else (200, 64)),
                   scale=(200 if which == "w1" else 64) ** -0.5)
        w[at] = torch.nan
        bad = (layer.quantize_weights4 if bits == 4 else layer.quantize_weights)(w.to(dev))
        got = layer.experts(hidden, weight, *((bad, w2) if which == "w1" else (w1, bad)), topk_idx=idx).cpu()
        has = (idx.cpu() == 1).any(-1)
        assert has.any() and not has.all() and torch.equal(got[~has], good[~has])
        if which == "w1":
            assert torch.isnan(got[has]).all()
        else:  # of matrices in 8 bits a block is 128 rows
            lost = range(0, 128) if bits == 8 else [70]
            rest = [c for c in range(200) if c not in lost]
            assert torch.isnan(got[has][:, list(lost)]).all() and torch.equal(got[has][:, rest], good[has][:, rest])
        assert layer.status() == 0
        layer.close()


def test_few_tokens_take_any_scale_bytes(mp):
    """Scales of the matrices far from 1, that cancel: w1's gate and up halves, and w2."""
    layer, idx, weight, w1, w2 = few_layer(mp, 5, 4, 2, 300, 40, 4, 2)
    hidden = normal(6, 5, 300).to(layer.device)
    good = layer.experts(hidden, weight, w1, w2, topk_idx=idx)
    up = w1.scale.view(torch.uint8)
    up[:, :, 40:] -= 60
    w2.scale.view(torch.uint8).add_(60)
    assert torch.equal(layer.experts(hidden, weight, w1, w2, topk_idx=idx), good)
    layer.close()


# ---- refusals -------------------------------------------------------------------

def test_refusals(mp):
    layer = mp.Layer(mp.make_config(8, 4, 2, 1, 1, 64, 0), cooc=False)
    dev = layer.device
    x = normal(1, 16, 64).to(dev)
    w = layer.quantize_weights4(normal(2, 4, 32, 64).to(dev))
    x4, x8 = layer.quantize4(x), layer.quantize(x)
    plan, off, _ = instances(mp, layer, [16], [0])
    kw = dict(plan=plan, inst_offset=off)
    with pytest.raises(TypeError):
        layer.quantize4(x.half())
    with pytest.raises(ValueError):
        layer.quantize4(x[0])
    with pytest.raises(ValueError):
        layer.quantize4(x[:, ::2])
    with pytest.raises(ValueError):
        layer.quantize4(x.cpu())
    with pytest.raises(ValueError):
        layer.quantize4(x, out=layer.quantize4(x[:, :32].contiguous()))
    with pytest.raises(ValueError):
        layer.quantize4(x, out=layer.quantize4(x[:8]))
    with pytest.raises(ValueError):
        layer.quantize_weights4(x)
    with pytest.raises(ValueError):
        layer.swiglu4(x[:, :63].contiguous())
    with pytest.raises(ValueError):
        layer.matmul4(layer.quantize4(x[:, :32].contiguous()), w, **kw)
    with pytest.raises(ValueError):
        layer.matmul4(layer.quantize4(x[:8]), w, **kw)
    with pytest.raises(ValueError):
        layer.matmul4(x4, layer.quantize_weights4(normal(2, 3, 32, 64).to(dev)), **kw)
    with pytest.raises(TypeError):
        layer.matmul4(x8, mp.Blocks4(w.q.view(torch.uint8), w.scale, 64), **kw)
    with pytest.raises(TypeError):
        layer.matmul4(x4, w, out=torch.empty(16, 32, dtype=torch.float16, device=dev), **kw)
    with pytest.raises(ValueError):
        layer.values4(mp.Blocks4(x4.q, x4.scale, 300))
    p = lambda t: t.data_ptr()
    lib, h = mp.lib(), layer.handle
    ok = (h, p(x), 16, 64, p(x4.q), p(x4.scale), None)
    for i, bad, code in ((2, -1, mp.MOE_ERR_INVALID_ARG), (3, 0, mp.MOE_ERR_INVALID_ARG), (1, None, mp.MOE_ERR_INVALID_ARG),
                         (4, p(x4.q) + 8, mp.MOE_ERR_INVALID_ARG), (5, p(x4.scale) + 4, mp.MOE_ERR_INVALID_ARG),
                         (2, 1 << 31, mp.MOE_ERR_UNSUPPORTED), (3, (1 << 24) + 1, mp.MOE_ERR_UNSUPPORTED)):
        args = list(ok)
        args[i] = bad
        assert lib.moex4_quantize(*args) == code
        assert lib.moex4_swiglu(*args) == code
    assert lib.moex4_quantize_weights(h, p(x), 1, 16, 64, p(w.q), p(w.scale), p(w.q), None, None) == mp.MOE_ERR_INVALID_ARG
    assert lib.moex4_quantize_weights(h, p(x), 1 << 20, 4096, 4096, p(w.q), p(w.scale), None, None, None) == \
        mp.MOE_ERR_UNSUPPORTED
    assert lib.moex4_quantize_weights(h, p(x), 2 ** 31 - 1, 1 << 24, 1 << 24, p(w.q), p(w.scale), None, None, None) == \
        mp.MOE_ERR_UNSUPPORTED
    assert lib.moex4_values(h, p(x4.q), p(x4.scale), -1, 16, 64, p(x), None) == mp.MOE_ERR_INVALID_ARG
    assert lib.moex4_values(h, p(x4.q), p(x4.scale), 1 << 16, 1 << 16, 64, p(x), None) == mp.MOE_ERR_UNSUPPORTED
    import ctypes
    s = plan.struct()
    for bits, n, k, code in ((6, 32, 64, mp.MOE_ERR_INVALID_ARG), (4, 0, 64, mp.MOE_ERR_INVALID_ARG),
                             (4, 32, (1 << 20) + 1, mp.MOE_ERR_UNSUPPORTED)):
        assert lib.moex4_matmul(h, ctypes.byref(s), p(off), bits, p(x4.q), p(x4.scale), p(w.q), p(w.scale), n, k, p(x),
                                None) == code
    torch.cuda.synchronize()
    assert layer.status() == 0
    layer.close()


def test_refusals_of_few_tokens(mp):
    layer, idx, weight, w1, w2 = few_layer(mp, 8, 4, 2, 64, 32, 4)
    dev = layer.device
    hidden = normal(3, 8, 64).to(dev)
    call = lambda **kw: layer.experts(**{**dict(hidden=hidden, weight=weight, w1=w1, w2=w2, topk_idx=idx), **kw})
    call()
    eight = layer.quantize_weights(normal(2, 4, 64, 32).to(dev))
    for bad, error in ((dict(hidden=hidden.half()), TypeError), (dict(hidden=hidden[:4]), ValueError),
                       (dict(weight=weight.double()), TypeError), (dict(topk_idx=idx.long()), TypeError),
                       (dict(w2=eight), TypeError), (dict(w1=w2), ValueError), (dict(w2=w1), ValueError),
                       (dict(out=hidden), ValueError), (dict(out=torch.empty(8, 64, device=dev)), TypeError)):
        with pytest.raises(error):
            call(**bad)
    torch.cuda.synchronize()
    assert layer.status() == 0
    layer.close()
    layer, idx, weight, w1, w2 = few_layer(mp, 65, 4, 2, 64, 32, 4)
    with pytest.raises(mp.MoePlanError) as e:
        layer.experts(normal(3, 65, 64).to(dev), weight, w1, w2, topk_idx=idx)
    assert e.value.code == mp.MOE_ERR_UNSUPPORTED
    layer.close()
