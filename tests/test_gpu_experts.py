"""Block quantization, the gated activation, the experts' products and their gradients against
tests/expert_refs.py (64 bits, CPU), and a whole layer forward and backward."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

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


def same_blocks(got, q, s):
    torch.cuda.synchronize()
    assert torch.equal(got.scale.cpu().view(torch.uint8), s)
    assert torch.equal(got.q.cpu().double(), q)


# ---- quantization ---------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 128), (257, 130), (33, 136), (64, 1000), (9, 2688), (1, 16384),
                                       (2048, 8), (70, 520)])
def test_rows(mp, small, rows, cols):
    print("quantize rows %d x %d" % (rows, cols), flush=True)
    x = normal(rows + cols, rows, cols)
    x[0] *= 1e-30
    if rows > 2:
        x[1] = 0
        x[2] *= 1e30
    same_blocks(small.quantize(x.to(small.device)), *refs.quantize(x.double()))


def test_rows_at_the_borders(mp, small):
    """Largest magnitudes on both sides of 448 * 2^e, the type's extremes, halves between two e4m3 values."""
    rows = []
    for e in (-126, -120, -20, 0, 3, 100, 118):
        for top in (448, 446, 450, 447, 256, 1.0):
            r = torch.linspace(-1, 1, 128) * top * 2.0 ** e
            r[0] = top * 2.0 ** e
            rows.append(r)
    steps = torch.arange(128) / 16.0 + 8        # midpoints of e4m3 neighbours, ties to even
    rows += [torch.cat([steps[:127], torch.tensor([448.0])]), torch.full((128,), torch.finfo(BF).max),
             torch.full((128,), -torch.finfo(BF).tiny), torch.full((128,), 9.2e-41), torch.zeros(128)]
    x = torch.stack(rows).to(BF)
    same_blocks(small.quantize(x.to(small.device)), *refs.quantize(x.double()))


@pytest.mark.parametrize("value", [torch.inf, -torch.inf, torch.nan])
def test_marked_blocks(mp, small, value):
    """A block with an infinity or a NaN is marked, and every sum over it is NaN; others are as without it."""
    x = normal(1, 8, 300)
    clean = small.quantize(x.to(small.device))
    x[3, 200] = value
    b = small.quantize(x.to(small.device))
    torch.cuda.synchronize()
    s, c = b.scale.cpu().view(torch.uint8), clean.scale.cpu().view(torch.uint8)
    assert s[3, 1] == 255 and int((s != c).sum()) == 1
    q, qc = b.q.cpu().view(torch.uint8), clean.q.cpu().view(torch.uint8)
    assert torch.equal(q[:3], qc[:3]) and torch.equal(q[3, :128], qc[3, :128])
    w = small.quantize_weights(normal(2, 8, 16, 300).to(small.device))
    plan, off, spans = instances(mp, small, [8], [0])
    y = small.matmul(b, w, plan=plan, inst_offset=off).cpu()
    assert torch.isnan(y[3]).all() and torch.isfinite(y[[0, 1, 2, 4, 5, 6, 7]]).all()
    dw = small.wgrad(small.quantize(normal(3, 8, 16).to(small.device)), b, plan=plan, inst_offset=off).cpu()
    assert torch.isnan(dw[0][:, 128:256]).all() and torch.isfinite(dw[0][:, :128]).all()
    assert (dw[1:] == 0).all()


@pytest.mark.parametrize("E,n,k", [(1, 1, 1), (2, 128, 128), (3, 130, 200), (2, 760, 1000), (5, 64, 384), (1, 257, 129),
                                   (2, 512, 640)])
def test_matrices(mp, small, E, n, k):
    print("quantize matrices %d x %d x %d" % (E, n, k), flush=True)
    w = normal(E + n + k, E, n, k, scale=0.02)
    w[0, : min(n, 128), : min(k, 128)] = 0
    if n > 200:
        w[0, 200] *= 1e20
    b, t = small.quantize_weights(w.to(small.device), transposed=True)
    q, s = refs.quantize(w.double(), 128)
    same_blocks(b, q, s)
    qt, st = refs.quantize(w.double().transpose(1, 2).contiguous(), 128)
    same_blocks(t, qt, st)
    assert t.cols == n and b.cols == k
    alone = small.quantize_weights(w.to(small.device))
    assert torch.equal(alone.q.view(torch.uint8), b.q.view(torch.uint8))


def close_blocks(b, want, cols):
    """fp32 values quantized: the scale is that of a largest magnitude within 2^-19 of the exact one, and each value
    is within half an e4m3 step (2^-4 of it, or 2^-10 of the scale below 2^-6 of it) and 2^-19 of the exact one.
    2^-19: expf and its argument (2 units and |x| <= 64 of them), the divisions and the products."""
    torch.cuda.synchronize()
    got, s = refs.values(b, None), b.scale.cpu().double()[:, : refs.pad(cols) // 128]
    top = refs.block_max(want)
    lo, hi = (torch.exp2(refs.block_exponent(top * f).double()) for f in (1 - 2.0 ** -19, 1 + 2.0 ** -19))
    assert ((s == lo) | (s == hi)).all()
    step = s.repeat_interleave(128, -1)[:, :cols] * 2.0 ** -10
    off = torch.maximum(2.0 ** -4 * want.abs(), step) * (1 + 2.0 ** -10) + 2.0 ** -19 * want.abs()
    assert ((got - want).abs() <= off).all()


@pytest.mark.parametrize("rows,f", [(1, 1), (3, 20), (130, 128), (5, 384), (33, 1000), (64, 2688), (7, 77), (1024, 136)])
def test_gated_activation_and_its_gradient(mp, small, rows, f):
    print("swiglu %d x %d" % (rows, f), flush=True)
    y = normal(rows + f, rows, 2 * f, scale=2.0)
    da = normal(rows * f + 1, rows, f, scale=1e-3)
    y[0, 0], y[0, f] = -60.0, 3.0
    if rows > 2:
        y[1] = 0
        da[2] = 0
    yd, dd = y.to(small.device), da.to(small.device)
    close_blocks(small.swiglu(yd), refs.swiglu(y.double()), f)
    y64 = y.double().requires_grad_()
    want, = torch.autograd.grad(refs.swiglu(y64), y64, da.double())
    assert torch.allclose(want, refs.swiglu_grad(y.double(), da.double()), rtol=1e-9, atol=1e-18)
    close_blocks(small.swiglu_grad(yd, dd), want, 2 * f)
    # the formula's gradient against differences
    h = 1e-6
    for c in {0, f - 1, f, 2 * f - 1}:
        up, down = y.double(), y.double()
        up[-1, c] += h
        down[-1, c] -= h
        d = ((refs.swiglu(up) - refs.swiglu(down)) * da.double()).sum() / (2 * h)
        assert abs(d - want[-1, c]) <= 1e-7 * (1 + want[-1].abs().max())


def test_unaligned_rows(mp, small):
    """bf16 inputs that start 2 bytes past a 16-byte boundary."""
    x = normal(4, 20, 256)
    buf = torch.empty(20 * 256 + 1, dtype=BF, device=small.device)
    view = buf[1:].view(20, 256).copy_(x)
    same_blocks(small.quantize(view), *refs.quantize(x.double()))
    a, b = small.swiglu(view), small.swiglu(x.to(small.device))
    assert torch.equal(a.q.view(torch.uint8), b.q.view(torch.uint8))
    da = normal(5, 20, 128)
    dbuf = torch.empty(20 * 128 + 1, dtype=BF, device=small.device)
    a, b = small.swiglu_grad(view, dbuf[1:].view(20, 128).copy_(da)), small.swiglu_grad(x.to(small.device), da.to(small.device))
    assert torch.equal(a.q.view(torch.uint8), b.q.view(torch.uint8)) and torch.equal(a.scale.view(torch.uint8), b.scale.view(torch.uint8))
    w = normal(6, 1, 20, 256)
    wv = buf[1:].view(1, 20, 256).copy_(w)
    same_blocks(small.quantize_weights(wv), *refs.quantize(w.double(), 128))


@pytest.mark.parametrize("rows,cols", [(2, 9), (7, 1001), (513, 2047), (1, 15), (4, 17), (3, 129)])
def test_rows_of_odd_widths(mp, small, rows, cols):
    test_rows(mp, small, rows, cols)


@pytest.mark.parametrize("E,n,k", [(2, 33, 1001), (1, 500, 7), (3, 129, 255), (2, 9, 1), (1, 3, 2399)])
def test_matrices_of_odd_widths(mp, small, E, n, k):
    test_matrices(mp, small, E, n, k)


@pytest.mark.parametrize("rows,f", [(1, 3), (2, 5), (9, 131), (300, 1455), (17, 63), (40, 119), (3, 129), (1, 8), (2, 12)])
def test_gated_activation_of_odd_widths(mp, small, rows, f):
    test_gated_activation_and_its_gradient(mp, small, rows, f)


@pytest.mark.parametrize("value", [torch.inf, torch.nan])
def test_neighbours_stay_apart(mp, small, value):
    """Rows and matrices of odd widths are read past their ends: what stands there marks only its own blocks."""
    rows, f = 12, 133
    dev = small.device
    marked = lambda b: b.scale.view(torch.uint8).cpu() == 255
    x = normal(1, rows, f)
    x[5] = value
    m = marked(small.quantize(x.to(dev)))
    assert m[5, :2].all() and int(m.sum()) == 2
    y, da = normal(2, rows, 2 * f), normal(3, rows, f)
    y[5] = value
    m = marked(small.swiglu(y.to(dev)))
    assert m[5, :2].all() and int(m.sum()) == 2
    m = marked(small.swiglu_grad(y.to(dev), da.to(dev)))
    assert m[5, :3].all() and int(m.sum()) == 3
    da[7] = value
    m = marked(small.swiglu_grad(normal(2, rows, 2 * f).to(dev), da.to(dev)))
    assert m[7, :3].all() and int(m.sum()) == 3
    w = normal(4, 3, 130, f)
    w[1] = value
    b, t = small.quantize_weights(w.to(dev), transposed=True)
    for m in (marked(b), marked(t)):
        assert m[1, :, :2].all() and int(m.sum()) == 4


def test_no_rows(mp, small):
    b = small.quantize(torch.empty(0, 200, dtype=BF, device=small.device))
    assert b.q.shape == (0, 256) and b.scale.shape == (0, 4)
    assert small.swiglu(torch.empty(0, 200, dtype=BF, device=small.device)).q.shape == (0, 128)
    w, wt = small.quantize_weights(torch.empty(0, 4, 200, dtype=BF, device=small.device), transposed=True)
    assert w.q.shape == (0, 4, 256) and wt.q.shape == (0, 200, 128)
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
    """Forward, input gradient and weight gradient of one set of instances."""
    rows = int(sum(loads))
    print("products loads=%s.. E=%d n=%d k=%d" % (list(loads)[:8], E, n, k), flush=True)
    layer = layer_for(mp, rows, E, B)
    dev = layer.device
    plan, off, spans = instances(mp, layer, loads, experts)
    x, w = normal(seed + 1, rows, k), normal(seed + 2, E, n, k, scale=0.05)
    dy = normal(seed + 3, rows, n, scale=1e-3)
    x[rows // 2] *= 300  # rows of different scales
    xb, db = layer.quantize(x.to(dev)), layer.quantize(dy.to(dev))
    wb, wt = layer.quantize_weights(w.to(dev), transposed=True)
    y = torch.full((rows, n), 7.0, dtype=BF, device=dev)
    dx = torch.full((rows, k), 7.0, dtype=BF, device=dev)
    dw = torch.full((E, n, k), 7.0, dtype=BF, device=dev)
    kw = dict(plan=plan, inst_offset=off)
    layer.matmul(xb, wb, out=y, **kw)
    layer.matmul(db, wt, out=dx, **kw)
    layer.wgrad(db, xb, out=dw, **kw)
    torch.cuda.synchronize()
    assert layer.status() == 0
    xv, dv, wv, wtv = refs.values(xb, rows), refs.values(db, rows), refs.values(wb, n, 128), refs.values(wt, k, 128)
    assert torch.equal(wv, wtv.transpose(1, 2))
    y, dx, dw = y.cpu().double(), dx.cpu().double(), dw.cpu().double()
    for e in range(E):
        at = torch.cat([torch.arange(a, b) for f, a, b in spans if f == e] + [torch.arange(0)]).long()
        for got, (want, off_) in ((y[at], refs.product(xv[at], wv[e])), (dx[at], refs.product(dv[at], wtv[e])),
                                  (dw[e], refs.outer(dv[at], xv[at]))):
            err = (got - want).abs()
            assert (err <= off_).all(), "expert %d: %d of %d outside, worst excess %g" % (
                e, int((err > off_).sum()), err.numel(), float((err - off_).max()))
    again = layer.wgrad(db, xb, **kw)
    assert torch.equal(again.cpu().double(), dw) and torch.equal(layer.matmul(xb, wb, **kw).cpu().double(), y)
    layer.close()


@pytest.mark.parametrize("loads,experts,E,n,k,B", [
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
])
def test_products(mp, loads, experts, E, n, k, B):
    check_products(mp, loads, experts, E, n, k, B, seed=n + k)


def test_products_of_many_instances(mp):
    """A plan of 2048 experts and 1000 replicas, most of them empty."""
    rng = np.random.RandomState(0)
    E, B = 2048, 1000
    loads = rng.multinomial(900, rng.dirichlet(np.full(E + B, 0.1)))
    check_products(mp, loads, np.concatenate([np.arange(E), rng.permutation(E)[:B]]), E, 24, 40, B)


@pytest.mark.parametrize("T,E,k,n,kk", [(4096, 8, 2, 768, 1024), (64, 64, 8, 1536, 2048), (1001, 16, 4, 520, 776)])
def test_products_of_a_routed_layer_sampled(mp, T, E, k, n, kk):
    """On the plan and offsets of the layer's own calls; sampled rows and experts."""
    print("routed products T=%d E=%d k=%d n=%d k=%d" % (T, E, k, n, kk), flush=True)
    layer = mp.Layer(mp.make_config(T, E, k, 1, 1, kk, 4, slots_per_rank=4, expert_bytes=0))
    dev = layer.device
    x = normal(T, T, E).float()
    layer.gate(x.to(dev), mp.make_gate("sigmoid", scale=2.5), bias=torch.linspace(0, 0.3, E, device=dev))
    layer.plan()
    hidden = normal(T + 1, T, kk)
    d = layer.dispatch(hidden.to(dev))
    xb = layer.quantize(d.dispatch.view(BF))
    w = normal(5, E, n, kk, scale=0.03)
    wb, wt = layer.quantize_weights(w.to(dev), transposed=True)
    y = layer.matmul(xb, wb)
    dy = normal(6, T * k, n, scale=0.01)
    db = layer.quantize(dy.to(dev))
    dx, dw = layer.matmul(db, wt), layer.wgrad(db, xb)
    torch.cuda.synchronize()
    assert layer.status() == 0
    off, expert = d.inst_offset.cpu().numpy(), layer.plan_out.inst_expert.cpu().numpy()
    n_inst = int(layer.plan_out.n_inst.item())
    xv, dv = refs.values(xb, T * k), refs.values(db, T * k)
    wv = refs.values(wb, n, 128)
    y, dx, dw = y.cpu().double(), dx.cpu().double(), dw.cpu().double()
    rng = np.random.RandomState(1)
    for i in {0, n_inst - 1, *rng.randint(0, n_inst, 6).tolist()}:
        rows = np.unique(rng.randint(off[i], max(off[i] + 1, off[i + 1]), 40)) if off[i] < off[i + 1] else []
        rows = torch.tensor(list(rows), dtype=torch.long)
        for got, (want, bound) in ((y[rows], refs.product(xv[rows], wv[expert[i]])),
                                   (dx[rows], refs.product(dv[rows], wv[expert[i]].t().contiguous()))):
            assert ((got - want).abs() <= bound).all()
    for e in {0, E - 1, *rng.randint(0, E, 2).tolist()}:
        at = torch.cat([torch.arange(off[i], off[i + 1]) for i in range(n_inst) if expert[i] == e] + [torch.arange(0)]).long()
        c = torch.tensor(sorted(rng.choice(n, 60, replace=False)))
        want, bound = refs.outer(dv[at][:, c], xv[at])
        assert ((dw[e][c] - want).abs() <= bound).all()
    layer.close()


def test_products_of_many_instances_in_tiles(mp):
    """As above with enough rows for the tiled kernels: each workgroup counts the tiles of 3048 instances."""
    rng = np.random.RandomState(3)
    E, B = 2048, 1000
    loads = rng.multinomial(17000, rng.dirichlet(np.full(E + B, 0.05)))
    check_products(mp, loads, np.concatenate([np.arange(E), rng.permutation(E)[:B]]), E, 24, 40, B)


def sampled_products(layer, plan, off, spans, E, n, k, seed, rows_per_span=24, columns=40):
    """Products and gradients at sizes of the large tiles: sampled against 64 bits, and the same bytes on every run
    while other kernels come and go."""
    rows, dev = layer.cfg.T * layer.cfg.k, layer.device
    g = torch.Generator(device=dev).manual_seed(seed)
    n16 = lambda *s: torch.randn(*s, generator=g, device=dev).to(BF)
    xb, db = layer.quantize(n16(rows, k)), layer.quantize(n16(rows, n))
    wb, wt = layer.quantize_weights(0.05 * n16(E, n, k), transposed=True)
    kw = dict(plan=plan, inst_offset=off)
    y, dx, dw = layer.matmul(xb, wb, **kw), layer.matmul(db, wt, **kw), layer.wgrad(db, xb, **kw)
    for _ in range(3):
        noise = torch.randn(1 << 22, device=dev).sort().values  # other work on the chip
        assert torch.equal(layer.matmul(xb, wb, **kw), y) and torch.equal(layer.matmul(db, wt, **kw), dx)
        assert torch.equal(layer.wgrad(db, xb, **kw), dw)
        del noise
    assert layer.status() == 0
    rng = np.random.RandomState(seed)
    take = lambda b, at: refs.values(type(b)(b.q.view(torch.uint8)[at.to(dev)].view(torch.float8_e4m3fn),
                                             b.scale.view(torch.uint8)[at.to(dev)].view(torch.float8_e8m0fnu), b.cols), len(at))
    mats = lambda b, e, m: refs.values(type(b)(b.q[e], b.scale[e], b.cols), m, 128)
    for e, a, b in spans:
        if a == b:
            continue
        at = torch.tensor(np.unique(np.concatenate([[a, b - 1], rng.randint(a, b, rows_per_span)])), dtype=torch.long)
        for got, (want, bound) in ((y, refs.product(take(xb, at), mats(wb, e, n))),
                                   (dx, refs.product(take(db, at), mats(wt, e, k)))):
            assert ((got[at.to(dev)].cpu().double() - want).abs() <= bound).all(), (e, a, b)
    for e in sorted(set(rng.randint(0, E, 3).tolist()) | {0, E - 1}):
        at = torch.cat([torch.arange(a, b) for f, a, b in spans if f == e] + [torch.arange(0)]).long()
        c = torch.tensor(np.unique(np.concatenate([[0, n - 1], rng.randint(0, n, columns)])), dtype=torch.long)
        want, bound = refs.outer(take(db, at)[:, c], take(xb, at))
        assert ((dw[e].cpu()[c].double() - want).abs() <= bound).all(), e


@pytest.mark.parametrize("loads,experts,E,n,k,B", [
    ([5000, 300, 7000, 4084], [0, 1, 2, 3], 4, 2200, 1032, 0),            # 9 blocks, odd widths
    ([4096, 4097, 4095, 0, 1, 4095], [0, 1, 2, 3, 0, 2], 4, 2304, 2048, 2),
    ([9000, 7384], [1, 0], 2, 2100, 100, 0),                              # a single block of the long axis
    ([100, 37, 250, 64, 1, 129, 65, 500, 300, 200, 77, 90, 31, 63, 128, 700], list(range(16)), 16, 1576, 2050, 0),
])
def test_large_tiles_sampled(mp, loads, experts, E, n, k, B):
    print("large tiles loads=%s E=%d n=%d k=%d" % (loads, E, n, k), flush=True)
    layer = layer_for(mp, sum(loads), E, B)
    plan, off, spans = instances(mp, layer, loads, experts)
    sampled_products(layer, plan, off, spans, E, n, k, n + k)
    layer.close()


def test_offsets_past_32_bits(mp):
    """More than 2^32 bytes of rows: quantization, products and gradients at the end of the buffers."""
    rows, E, n, k = 655360, 8, 136, 7168
    print("past 32 bits: %d rows of %d" % (rows, k), flush=True)
    layer = layer_for(mp, rows, E)
    dev = layer.device
    x = torch.randn(rows, k, device=dev, dtype=BF, generator=torch.Generator(device=dev).manual_seed(1))
    xb = layer.quantize(x)
    last = torch.arange(rows - 3, rows, device=dev)
    q, s = refs.quantize(x[last].cpu().double())
    assert torch.equal(xb.q[last].cpu().double(), q) and torch.equal(xb.scale.view(torch.uint8)[last].cpu(), s)
    del x
    loads = [rows // E] * E
    plan, off, spans = instances(mp, layer, loads, list(range(E)))
    w = layer.quantize_weights((0.02 * torch.randn(E, n, k, device=dev)).to(BF))
    y = layer.matmul(xb, w, plan=plan, inst_offset=off)
    xv = refs.values(mp.Blocks(xb.q[last], xb.scale[last], k), 3)
    wv = refs.values(mp.Blocks(w.q[E - 1], w.scale[E - 1], k), n, 128)
    want, bound = refs.product(xv, wv)
    assert ((y[last].cpu().double() - want).abs() <= bound).all()
    # a gradient that only the last rows feed
    dy = torch.zeros(rows, n, dtype=BF, device=dev)
    dy[last] = 1
    dw = layer.wgrad(layer.quantize(dy), xb, plan=plan, inst_offset=off)
    want, bound = refs.outer(torch.ones(3, n, dtype=torch.float64), xv)
    assert ((dw[E - 1].cpu().double() - want).abs() <= bound).all() and (dw[: E - 1] == 0).all()
    assert layer.status() == 0
    layer.close()


@pytest.mark.parametrize("rows,n,k", [(6, 5, 2 ** 20), (12, 5, 2 ** 20), (6, 2 ** 20, 40), (12, 2 ** 20, 40)])
def test_longest_axes(mp, rows, n, k):
    """The largest widths, in the kernel for few rows and in tiles."""
    print("longest axes %d x %d x %d" % (rows, n, k), flush=True)
    layer = layer_for(mp, rows, 1)
    dev = layer.device
    plan, off, _ = instances(mp, layer, [rows], [0])
    kw = dict(plan=plan, inst_offset=off)
    x, d = layer.quantize(normal(1, rows, k).to(dev)), layer.quantize(normal(2, rows, n).to(dev))
    w = layer.quantize_weights(normal(3, 1, n, k, scale=0.1).to(dev))
    y, dw = layer.matmul(x, w, **kw), layer.wgrad(d, x, **kw)
    assert layer.status() == 0
    c = torch.cat([torch.arange(min(n, 200)), torch.arange(max(0, n - 200), n)]).unique()
    xv = refs.values(x, rows)
    wv = refs.values(mp.Blocks(w.q[0], w.scale[0], k), n, 128)[c]
    want, bound = refs.product(xv, wv)
    assert ((y.cpu().double()[:, c] - want).abs() <= bound).all()
    want, bound = refs.outer(refs.values(d, rows)[:, c], xv)
    assert ((dw[0].cpu()[c].double() - want).abs() <= bound).all()
    layer.close()
    with pytest.raises(mp.MoePlanError):
        big = layer_for(mp, rows, 1)
        big.matmul(big.quantize(torch.zeros(rows, 2 ** 20 + 1, dtype=BF, device=dev)),
                   big.quantize_weights(torch.zeros(1, 2, 2 ** 20 + 1, dtype=BF, device=dev)))


def test_no_tokens(mp):
    layer = mp.Layer(mp.make_config(0, 4, 2, 1, 1, 64, 0), cooc=False)
    dev = layer.device
    layer.plan_out.n_inst.fill_(4)
    layer.plan_out.inst_expert.copy_(torch.arange(4))
    layer.dispatch_out.inst_offset.zero_()
    rows = layer.quantize(torch.empty(0, 64, dtype=BF, device=dev))
    w, wt = layer.quantize_weights(normal(1, 4, 48, 64).to(dev), transposed=True)
    assert layer.matmul(rows, w).shape == (0, 48)
    dw = torch.full((4, 48, 64), 7.0, dtype=BF, device=dev)
    layer.wgrad(layer.quantize(torch.empty(0, 48, dtype=BF, device=dev)), rows, out=dw)
    torch.cuda.synchronize()
    assert layer.status() == 0 and (dw == 0).all()
    layer.close()


def test_bad_plans_set_the_status_and_leave_rows_alone(mp):
    rows, E, n, k = 64, 4, 48, 96   # 16 rows an expert: the tiled kernel
    layer = layer_for(mp, rows, E, 2)
    dev = layer.device
    xb, wb = layer.quantize(normal(1, rows, k).to(dev)), layer.quantize_weights(normal(2, E, n, k).to(dev))
    db = layer.quantize(normal(3, rows, n).to(dev))
    loads, experts = [20, 20, 20, 4], [0, 1, 2, 3]
    plan, off, _ = instances(mp, layer, loads, experts)
    good = layer.matmul(xb, wb, plan=plan, inst_offset=off)
    assert layer.status() == 0

    def run(change):
        p, o, _ = instances(mp, layer, loads, experts)
        change(p, o)
        out = torch.full((rows, n), 7.0, dtype=BF, device=dev)
        layer.matmul(xb, wb, plan=p, inst_offset=o, out=out)
        assert layer.status() == mp.MOE_STATUS_PLAN_CHECK
        dw = layer.wgrad(db, xb, plan=p, inst_offset=o)
        assert layer.status() == mp.MOE_STATUS_PLAN_CHECK and torch.isfinite(dw).all()
        return out

    def count(v):
        return lambda p, o: p.n_inst.fill_(v)
    for v in (-1, 7, 2 ** 31 - 1, -2 ** 31):
        assert (run(count(v)) == 7).all()
    for v in (-1, E, 2 ** 31 - 1, -2 ** 31):
        out = run(lambda p, o: p.inst_expert[1].fill_(v))
        assert (out[20:40] == 7).all() and torch.equal(out[:20], good[:20]) and torch.equal(out[40:], good[40:])
    for v in (-1, 70, 2 ** 31 - 1, -2 ** 31):   # the border of instances 1 and 2
        out = run(lambda p, o: o[2].fill_(v))
        # a row of the instances beside is the product or left alone
        for span in (slice(0, 20), slice(60, 64)):
            assert ((out[span] == good[span]).all(1) | (out[span] == 7).all(1)).all()
    # fewer instances than rows: the rest stays
    p, o, _ = instances(mp, layer, loads[:2], experts[:2])
    out = torch.full((rows, n), 7.0, dtype=BF, device=dev)
    layer.matmul(xb, wb, plan=p, inst_offset=o, out=out)
    assert layer.status() == 0 and (out[40:] == 7).all() and torch.equal(out[:40], good[:40])
    layer.close()


@pytest.mark.parametrize("rows,n", [(64, 48), (2048, 17000), (12, 48)])
def test_offsets_that_fall(mp, rows, n):
    """Every second instance holds all rows, those between would hold fewer than none: for each kernel (128 and 256
    rows to a tile, and few rows) the status tells, and each row is its expert's product or as it was."""
    E, k, B = 4, 96, 60
    layer = layer_for(mp, rows, E, B)
    dev = layer.device
    xb = layer.quantize(normal(1, rows, k).to(dev))
    wb = layer.quantize_weights(normal(2, E, n, k).to(dev))
    db = layer.quantize(normal(3, rows, n).to(dev))
    layer.plan_out.n_inst.fill_(E + B)
    layer.plan_out.inst_expert.fill_(1)
    layer.dispatch_out.inst_offset.copy_(torch.tensor([0, rows] * 32 + [0], dtype=torch.int32))
    y = torch.full((rows, n), 7.0, dtype=BF, device=dev)
    layer.matmul(xb, wb, out=y)
    dw = layer.wgrad(db, xb)
    assert dw.shape == (E, n, k)
    torch.cuda.synchronize()
    assert layer.status() & mp.MOE_STATUS_PLAN_CHECK
    at = torch.arange(0, rows, 1 + rows // 50)
    xv = refs.values(xb, rows)[at] if rows < 100 else refs.values(
        mp.Blocks(xb.q[at.to(dev)], xb.scale[at.to(dev)], k), len(at))
    want, bound = refs.product(xv, refs.values(mp.Blocks(wb.q[1], wb.scale[1], k), n, 128))
    got = y[at.to(dev)].cpu().double()
    assert (((got - want).abs() <= bound) | (got == 7)).all()
    layer.close()


def test_scales_far_apart(mp):
    """Blocks whose products differ by many powers of two, and scale bytes at the ends of their range."""
    rows, n, k = 20, 32, 512
    layer = layer_for(mp, rows, 1)
    dev = layer.device
    x, w = normal(1, rows, k).float(), normal(2, 1, n, k).float()
    x[:, :128] *= 2.0 ** 60
    x[:, 256:384] *= 2.0 ** -60
    w[..., :128] *= 2.0 ** -70
    w[..., 256:384] *= 2.0 ** 70
    x[3] *= 2.0 ** 40
    x[4] *= 2.0 ** -50
    plan, off, _ = instances(mp, layer, [rows], [0])
    xb, wb = layer.quantize(x.to(BF).to(dev)), layer.quantize_weights(w.to(BF).to(dev))
    y = layer.matmul(xb, wb, plan=plan, inst_offset=off).cpu().double()
    xv, wv = refs.values(xb, rows), refs.values(wb, n, 128)
    want, bound = refs.product(xv, wv[0])
    # block by block the bound scales with the block; the accumulator adds them in fp32
    assert ((y - want).abs() <= bound).all()
    layer.close()


def test_refusals(mp):
    layer = layer_for(mp, 32, 4)
    dev, lib = layer.device, mp.lib()
    xb, wb = layer.quantize(normal(1, 32, 64).to(dev)), layer.quantize_weights(normal(2, 4, 16, 64).to(dev))
    plan, off, _ = instances(mp, layer, [8] * 4, [0, 1, 2, 3])
    with pytest.raises(ValueError):
        layer.matmul(layer.quantize(normal(1, 32, 65).to(dev)), wb, plan=plan, inst_offset=off)
    with pytest.raises(ValueError):
        layer.matmul(layer.quantize(normal(1, 31, 64).to(dev)), wb, plan=plan, inst_offset=off)
    with pytest.raises(ValueError):
        layer.matmul(xb, layer.quantize_weights(normal(2, 3, 16, 64).to(dev)), plan=plan, inst_offset=off)
    with pytest.raises(TypeError):
        layer.matmul(mp.Blocks(xb.q.view(torch.uint8), xb.scale, 64), wb, plan=plan, inst_offset=off)
    with pytest.raises(ValueError):
        layer.matmul(xb, wb, plan=plan, inst_offset=off[:-1])
    with pytest.raises(ValueError):
        layer.matmul(xb, wb, plan=plan, inst_offset=off, out=torch.empty(32, 17, dtype=BF, device=dev))
    with pytest.raises(ValueError):
        layer.matmul(mp.Blocks(xb.q.cpu(), xb.scale, 64), wb, plan=plan, inst_offset=off)
    with pytest.raises(TypeError):
        layer.quantize(torch.zeros(4, 8, device=dev))
    with pytest.raises(ValueError):
        layer.swiglu(torch.zeros(4, 7, dtype=BF, device=dev))
    # the C entry points: sizes, missing pointers, pointers between the vectors that the kernels load
    import ctypes
    p = lambda t, add=0: ctypes.c_void_p(t.data_ptr() + add)
    ps, y = plan.struct(), torch.empty(32, 16, dtype=BF, device=dev)
    args = [layer.handle, ctypes.byref(ps), p(off), p(xb.q), p(xb.scale), p(wb.q), p(wb.scale), 16, 64, p(y), None]
    for at, bad in ((1, None), (2, None), (3, None), (4, None), (5, None), (6, None), (7, 0), (8, 0), (7, -5), (9, None),
                    (3, p(xb.q, 8)), (4, p(xb.scale, 2)), (5, p(wb.q, 4)), (6, p(wb.scale, 1))):
        a = list(args)
        a[at] = bad
        assert lib.moex_matmul(*a) == mp.MOE_ERR_INVALID_ARG, at
        assert lib.moex_wgrad(*a) == mp.MOE_ERR_INVALID_ARG, at
    for at in (7, 8):
        a = list(args)
        a[at] = (1 << 24) + 1
        assert lib.moex_matmul(*a) == mp.MOE_ERR_UNSUPPORTED and lib.moex_wgrad(*a) == mp.MOE_ERR_UNSUPPORTED
    x = torch.zeros(4, 256, dtype=BF, device=dev)
    assert lib.moex_quantize(layer.handle, p(x), -1, 8, p(xb.q), p(xb.scale), None) == mp.MOE_ERR_INVALID_ARG
    assert lib.moex_quantize(layer.handle, p(x), 4, 0, p(xb.q), p(xb.scale), None) == mp.MOE_ERR_INVALID_ARG
    assert lib.moex_quantize(layer.handle, p(x), 4, 8, p(xb.q, 1), p(xb.scale), None) == mp.MOE_ERR_INVALID_ARG
    assert lib.moex_quantize(layer.handle, p(x), 1 << 31, 8, p(xb.q), p(xb.scale), None) == mp.MOE_ERR_UNSUPPORTED
    assert lib.moex_quantize_weights(layer.handle, p(x), 1, 4, 256, p(wb.q), p(wb.scale), p(wb.q), None,
                                     None) == mp.MOE_ERR_INVALID_ARG
    assert lib.moex_quantize_weights(layer.handle, p(x), 1 << 20, 4096, 4096, p(wb.q), p(wb.scale), None, None,
                                     None) == mp.MOE_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert layer.status() == 0
    layer.close()


# ---- a whole layer ----------------------------------------------------------------

def whole_layer(mp, layer, st):
    """One training pass of an expert layer, every call of include/moe_experts.h in order."""
    r, weight = layer.gate(st["logits"], st["gate"], bias=st["bias"])
    layer.plan()
    d = layer.dispatch(st["hidden"])
    x = layer.quantize(d.dispatch.view(BF))
    w1, w1t = layer.quantize_weights(st["w1"], transposed=True)
    w2, w2t = layer.quantize_weights(st["w2"], transposed=True)
    y1 = layer.matmul(x, w1)
    a = layer.swiglu(y1)
    y2 = layer.matmul(a, w2)
    out = layer.combine_weighted(y2, weight)
    dy2, dweight = layer.combine_grad(y2, st["grad"], weight)
    dy2q = layer.quantize(dy2)
    da, dw2 = layer.matmul(dy2q, w2t), layer.wgrad(dy2q, a)
    dy1q = layer.swiglu_grad(y1, da)
    dx, dw1 = layer.matmul(dy1q, w1t), layer.wgrad(dy1q, x)
    dhidden = layer.combine_weighted(dx)
    dlogits = layer.gate_grad(st["logits"], st["gate"], dweight)
    return dict(topk=r.topk_idx, weight=weight, y1=y1, y2=y2, out=out, dy2=dy2, dweight=dweight, da=da, dw2=dw2,
                dx=dx, dw1=dw1, dhidden=dhidden, dlogits=dlogits, a=a.q.view(torch.uint8), dy1=dy1q.q.view(torch.uint8))


def layer_inputs(mp, T, E, k, H, F, dev, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, scale=1.0: (scale * torch.randn(*s, generator=g))
    return dict(logits=n(T, E).to(dev), bias=(0.1 * n(E)).to(dev), gate=mp.make_gate("sigmoid", 4, 2, 2, True, 2.5),
                hidden=n(T, H).to(BF).to(dev), grad=n(T, H).to(BF).to(dev),
                w1=n(E, 2 * F, H, scale=H ** -0.5).to(BF).to(dev), w2=n(E, H, F, scale=F ** -0.5).to(BF).to(dev))


def test_half_precision_is_refused(mp):
    T, E, k, H = 8, 4, 2, 128
    layer = mp.Layer(mp.make_config(T, E, k, 1, 1, H, 0), cooc=False)
    z = lambda *s: torch.zeros(*s, dtype=torch.float16, device=layer.device)
    b = lambda *s: z(*s).to(BF)
    w = torch.ones(T, k, device=layer.device)
    for call in (lambda: layer.quantize(z(4, H)), lambda: layer.quantize_weights(z(E, 8, H)),
                 lambda: layer.swiglu(z(4, H)), lambda: layer.swiglu_grad(b(4, 2 * H), z(4, H)),
                 lambda: layer.combine_weighted(z(T * k, H)), lambda: layer.combine_weighted(b(T * k, H), out=z(T, H)),
                 lambda: layer.combine_grad(b(T * k, H), z(T, H), w)):
        with pytest.raises(TypeError):
            call()
    layer.close()


def test_results_belong_to_the_stream_of_the_call(mp):
    """With stream=, a result that is dropped at once leaves its memory to that stream alone."""
    layer = layer_for(mp, 64, 4)
    dev, side = layer.device, torch.cuda.Stream()
    x, w = normal(1, 64, 256).to(dev), normal(2, 4, 48, 256).to(dev)
    want = layer.quantize(x)
    plan, off, _ = instances(mp, layer, [16] * 4, list(range(4)))
    kw = dict(plan=plan, inst_offset=off)
    torch.cuda.synchronize()
    xb = layer.quantize(x, stream=side)
    wb, wt = layer.quantize_weights(w, transposed=True, stream=side)
    y = layer.matmul(xb, wb, stream=side, **kw)
    dw = layer.wgrad(layer.quantize(y, stream=side), xb, stream=side, **kw)
    side.synchronize()
    assert torch.equal(xb.q.view(torch.uint8), want.q.view(torch.uint8))
    assert torch.equal(y, layer.matmul(xb, wb, **kw)) and dw.shape == (4, 48, 256)
    torch.cuda.synchronize()
    for t in (xb.q, wb.q, wt.q, y, dw):
        like, at = (t.shape, t.dtype), t.data_ptr()
        hold = torch.empty(like[0], dtype=like[1], device=dev)
        assert hold.data_ptr() != at
    freed = {t.data_ptr() for t in (y, dw)}
    shapes = [t.shape for t in (y, dw)]
    del y, dw, t
    again = [torch.empty(s, dtype=BF, device=dev) for s in shapes for _ in range(4)]
    assert not freed & {t.data_ptr() for t in again}
    assert layer.status() == 0
    layer.close()


def test_a_layer_forward_and_backward(mp):
    """Against the same layer in 64 bits with automatic differentiation.  Each tensor that is quantized moves by at
    most 2^-4 of itself, element by element, and by 3 % in the root mean square (an e4m3 step is 1/8 to 1/16 of a
    value, its rounding error's root mean square 1 / (12^0.5 * 11) of it); a path through up to five products adds
    those shares, so a tenth to a fifth of the result is the most that independent errors come to, and the check is
    that the result has the right direction and size: within a quarter in the 2-norm."""
    T, E, k, R, G, H, F = 96, 16, 4, 4, 2, 256, 96
    layer = mp.Layer(mp.make_config(T, E, k, R, G, H, 4, expert_bytes=0))
    st = layer_inputs(mp, T, E, k, H, F, layer.device)
    got = whole_layer(mp, layer, st)
    torch.cuda.synchronize()
    assert layer.status() == 0
    c = {n: (t.cpu().double() if torch.is_tensor(t) else t) for n, t in st.items()}
    leaf = {n: c[n].clone().requires_grad_() for n in ("logits", "hidden", "w1", "w2")}
    idx = got["topk"].cpu().long()
    assert torch.equal(idx, refs.select(c["logits"], c["bias"], "sigmoid", k, 4, 2, 2))
    weight = refs.gate_weights(leaf["logits"], idx, "sigmoid", True, 2.5)
    parts = []
    for j in range(k):
        y1 = torch.einsum("tfh,th->tf", leaf["w1"][idx[:, j]], leaf["hidden"])
        parts.append(torch.einsum("thf,tf->th", leaf["w2"][idx[:, j]], refs.swiglu(y1)) * weight[:, j:j + 1])
    out = sum(parts)
    grads = torch.autograd.grad(out, list(leaf.values()), c["grad"])
    for name, want in zip(("out", "dlogits", "dhidden", "dw1", "dw2"), (out.detach(), *grads)):
        off = (got[name].cpu().double() - want).norm() / want.norm()
        assert off < 0.25, (name, float(off))
    layer.close()


def test_a_captured_layer_replays(mp):
    """The whole pass captured into a graph: every replay equals the eager pass, with eager work in between and with
    other inputs in the same buffers."""
    T, E, k, R, G, H, F = 64, 16, 4, 2, 1, 264, 72
    layer = mp.Layer(mp.make_config(T, E, k, R, G, H, 2, expert_bytes=0))
    other = mp.Layer(mp.make_config(T, E, k, R, G, H, 2, expert_bytes=0))
    st = layer_inputs(mp, T, E, k, H, F, layer.device)
    whole_layer(mp, layer, st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = whole_layer(mp, layer, st)
    for i in range(4):
        new = layer_inputs(mp, T, E, k, H, F, layer.device, seed=i)
        for n, t in new.items():
            if torch.is_tensor(t):
                st[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in res.items()}
        want = whole_layer(mp, other, new)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n].view(torch.uint8), want[n].view(torch.uint8)), (i, n)
    assert layer.status() == 0 and other.status() == 0
    layer.close()
    other.close()


def test_one_layer_on_two_streams(mp):
    """Input and weight gradients of one handle side by side, eager and as two captured graphs."""
    loads, E, n, k = [700, 1, 0, 333, 500, 64], 6, 520, 392
    layer = layer_for(mp, sum(loads), E)
    dev = layer.device
    plan, off, _ = instances(mp, layer, loads, list(range(E)))
    kw = dict(plan=plan, inst_offset=off)
    rows = sum(loads)
    x, d = layer.quantize(normal(1, rows, k).to(dev)), layer.quantize(normal(2, rows, n).to(dev))
    w, wt = layer.quantize_weights(normal(3, E, n, k).to(dev), transposed=True)
    want_dx, want_dw = layer.matmul(d, wt, **kw), layer.wgrad(d, x, **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        dx = [layer.matmul(d, wt, stream=streams[0], **kw) for _ in range(4)]
        dw = [layer.wgrad(d, x, stream=streams[1], **kw) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(t, want_dx) for t in dx) and all(torch.equal(t, want_dw) for t in dw)
    graphs, got = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g, call in zip(graphs, (lambda: layer.matmul(d, wt, **kw), lambda: layer.wgrad(d, x, **kw))):
        with torch.cuda.graph(g):
            got.append(call())
    for _ in range(5):
        for t in got:
            t.fill_(3)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want_dx) and torch.equal(got[1], want_dw)
    assert layer.status() == 0
    layer.close()


def test_two_layers_on_two_streams(mp):
    T, E, k, R, G, H, F = 128, 16, 4, 2, 1, 256, 128
    layers = [mp.Layer(mp.make_config(T, E, k, R, G, H, 2, expert_bytes=0)) for _ in range(2)]
    sts = [layer_inputs(mp, T, E, k, H, F, layers[0].device, seed=i) for i in range(2)]
    want = [{n: t.clone() for n, t in whole_layer(mp, layers[i], sts[i]).items()} for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for rep in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = whole_layer(mp, layers[i], sts[i])
        torch.cuda.synchronize()
        for i in range(2):
            for n in want[i]:
                assert torch.equal(got[i][n].view(torch.uint8), want[i][n].view(torch.uint8)), (rep, i, n)
    for l in layers:
        assert l.status() == 0
        l.close()
