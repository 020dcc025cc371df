"""A layer with 4-bit matrices, forward and backward: every operand of the pass against the formula and the operands
that the GPU held, and what the whole chain gives against the same layer in 64 bits."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from tests import expert4_refs as refs4
from tests import expert_refs as refs
from tests.test_gpu_experts4 import BF
from tests.test_gpu_experts4_more import layer_inputs, spans_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import load_balance_planning_amd as m
    m.lib()
    return m


def near_blocks(got, want, scale, off=0.0):
    """e4m3 blocks of `want`, which was off by `off` times its value before: half a step is 2^-4 of the value, or 2^-10
    of the scale among the subnormals."""
    return ((got - want).abs() <= torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * scale) * (1 + 2.0 ** -10)
            + off * want.abs()).all()


def products(spans, x, w, got, cut=None):
    """Rows of every instance times its expert's matrix; cut: scales of x and w (rows in 8 bits)."""
    seen = 0
    for e, a, z in spans:
        want, off = x[a:z] @ w[e].t(), refs4.added(x[a:z], w[e])
        if cut:
            off = off + refs4.cut(x[a:z], cut[0][a:z], w[e], cut[1][e])
        if not ((got[a:z] - want).abs() <= refs4.rounded(want, off)).all():
            return False
        seen += z - a
    return seen == len(got)


def spread8(b):
    return refs4.spread(b.scale.cpu().double(), 128, b.cols)


def spread4(b):
    return refs4.spread(refs4.scales(b), 32, b.cols)


def passes(layer, st, router, q):
    """One forward and one backward pass; everything in it."""
    (q1, t1), (q2, t2) = q
    r = {}
    route, r["weight"] = layer.gate(st["logits"], router, bias=st["bias"])
    layer.plan()
    r["idx"] = route.topk_idx.cpu().long()
    r["rows"] = layer.dispatch(st["hidden"]).dispatch.view(BF)
    r["x"] = layer.quantize(r["rows"])
    r["y1"] = layer.matmul4(r["x"], q1)
    r["a"] = layer.swiglu(r["y1"])
    r["y2"] = layer.matmul4(r["a"], q2)
    r["out"] = layer.combine_weighted(r["y2"], r["weight"])
    r["g_y2"], r["g_weight"] = layer.combine_grad(r["y2"], st["g_out"], r["weight"])
    r["g2"] = layer.quantize(r["g_y2"])
    r["g_a"] = layer.matmul4(r["g2"], t2)
    r["g1"] = layer.swiglu_grad(r["y1"], r["g_a"])
    r["g_x"] = layer.matmul4(r["g1"], t1)
    r["g_hidden"] = layer.combine_weighted(r["g_x"])
    r["g_w2"], r["g_w1"] = layer.wgrad(r["g2"], r["a"]), layer.wgrad(r["g1"], r["x"])
    r["g_logits"] = layer.gate_grad(st["logits"], router, r["g_weight"])
    torch.cuda.synchronize()
    return r


def in_64_bits(idx, scale):
    """The layer's result, differentiable, without a rounding, for the experts as chosen."""
    def f(hidden, logits, w1, w2):
        s = 1 / (1 + torch.exp(-logits)).gather(1, idx)
        weight = scale * s / (s.sum(-1, keepdim=True) + 1e-20)
        out = torch.zeros_like(hidden)
        for e in sorted(set(idx.flatten().tolist())):
            t, j = (idx == e).nonzero(as_tuple=True)
            out = out.index_add(0, t, weight[t, j][:, None] * (refs.swiglu(hidden[t] @ w1[e].t()) @ w2[e].t()))
        return out
    return f


@pytest.mark.parametrize("T,E,k,R,H,F,B,seed", [(96, 8, 2, 2, 264, 72, 2, 0), (160, 6, 3, 1, 200, 130, 0, 5)])
def test_every_operand_of_a_pass(mp, T, E, k, R, H, F, B, seed):
    layer = mp.Layer(mp.make_config(T, E, k, R, 1, H, B, expert_bytes=0))
    st = layer_inputs(T, E, H, F, layer.device, seed)
    q = (q1, t1), (q2, t2) = [layer.quantize_weights4(st[n], transposed=True) for n in ("w1", "w2")]
    r = passes(layer, st, mp.make_gate("sigmoid", scale=2.5), q)
    assert layer.status() == 0
    spans, rows = spans_of(layer), T * k
    v = {n: refs.values(r[n], rows) for n in ("x", "a", "g2", "g1")}
    d = {n: r[n].cpu().double() for n in ("rows", "y1", "y2", "out", "weight", "g_y2", "g_weight", "g_a", "g_x", "g_hidden",
                                          "g_w1", "g_w2", "g_logits")}
    pos = layer.dispatch_out.slot_pos.cpu().long().view(T, k)
    assert pos.flatten().sort().values.equal(torch.arange(rows))
    g_out, grow = st["g_out"].cpu().double(), 1 + 2.0 ** -8
    # forward
    assert torch.equal(d["rows"][pos], st["hidden"].cpu().double()[:, None].expand(T, k, H))
    assert near_blocks(v["x"], d["rows"], spread8(r["x"]))
    assert products(spans, v["x"], refs4.values(q1), d["y1"], (spread8(r["x"]), spread4(q1)))
    assert near_blocks(v["a"], refs.swiglu(d["y1"]), spread8(r["a"]), 2.0 ** -19)
    assert products(spans, v["a"], refs4.values(q2), d["y2"], (spread8(r["a"]), spread4(q2)))
    y, mag = (d["y2"][pos] * d["weight"][..., None]).sum(1), (d["y2"][pos].abs() * d["weight"].abs()[..., None]).sum(1)
    assert ((d["out"] - y).abs() <= 2.0 ** -8 * y.abs() + grow * (k + 2) * 2.0 ** -24 * mag).all()
    # backward, from the result's gradient to that of the hidden rows
    want = d["weight"][..., None] * g_out[:, None]
    assert ((d["g_y2"][pos] - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -23) * want.abs()).all()
    dots = d["y2"][pos] * g_out[:, None]
    assert ((d["g_weight"] - dots.sum(-1)).abs() <= (H / 64 + 16) * 2.0 ** -24 * dots.abs().sum(-1)).all()
    assert near_blocks(v["g2"], d["g_y2"], spread8(r["g2"]))
    assert products(spans, v["g2"], refs4.values(t2), d["g_a"], (spread8(r["g2"]), spread4(t2)))
    # 1 + g (1 - sigmoid) cancels near g = -1.28: off by 2^-20 of its terms, and so of the other factors
    g, u = d["y1"][:, :F], d["y1"][:, F:]
    s = 1 / (1 + torch.exp(-g))
    off = 2.0 ** -20 * torch.cat([(d["g_a"] * u * s * (1 + g.abs())).abs(), (d["g_a"] * g * s).abs()], 1)
    want = refs.swiglu_grad(d["y1"], d["g_a"])
    step = torch.maximum(2.0 ** -4 * (want.abs() + off), 2.0 ** -10 * spread8(r["g1"])) * (1 + 2.0 ** -10)
    assert ((v["g1"] - want).abs() <= step + off).all()
    assert products(spans, v["g1"], refs4.values(t1), d["g_x"], (spread8(r["g1"]), spread4(t1)))
    y, mag = d["g_x"][pos].sum(1), d["g_x"][pos].abs().sum(1)
    assert ((d["g_hidden"] - y).abs() <= 2.0 ** -8 * y.abs() + grow * (k + 2) * 2.0 ** -24 * mag).all()
    # the matrices' gradients
    for name, dy, x in (("g_w2", v["g2"], v["a"]), ("g_w1", v["g1"], v["x"])):
        for e in range(E):
            at = torch.cat([torch.arange(a, z) for f, a, z in spans if f == e] + [torch.arange(0)]).long()
            want, bound = refs.outer(dy[at], x[at])
            assert ((d[name][e] - want).abs() <= bound).all(), (name, e)
    # the router's: the formula's Jacobian, its scores and sums in fp32
    lg = st["logits"].cpu().double().requires_grad_()
    s = refs.scores(lg, "sigmoid").gather(1, r["idx"])
    weight = 2.5 * s / (s.sum(-1, keepdim=True) + 1e-20)
    assert torch.allclose(weight.detach(), d["weight"], rtol=2.0 ** -18, atol=0)
    want, = torch.autograd.grad(weight, lg, d["g_weight"])
    big = d["g_weight"].abs().amax(-1, keepdim=True) * 2.5
    assert ((d["g_logits"] - want).abs() <= 2.0 ** -18 * big).all() and (want != 0).sum() == rows
    layer.close()


def apart(a, b):
    return float((a - b).norm() / b.norm())


def share(a, b):
    """How much of b is in a: 1 where a is b and what is across it."""
    return float((a * b).sum() / (b * b).sum())


def test_a_pass_against_the_layer_in_64_bits(mp):
    """Result and gradients of the layer whose matrices are the 4-bit values and that rounds nothing else, by its
    formula; and that gradient by differences.

    What the GPU rounds more: rows, activations and both gradients of rows to e4m3, by 2^-4 of a value at the most, and
    (of the input gradient) the transposed matrices to other 4-bit values, each by a fifth at the most above a scale.
    Roundings of many summands are as good as independent: the lengths of what they bring add as squares, and are below
    sqrt(4) 2^-4 = 0.125 of a result that only e4m3 goes into and sqrt(4 * 2^-8 + 4 / 25) = 0.42 of the input gradient
    (as large as that only if every single rounding were the worst one)."""
    T, E, k, H, F = 128, 8, 2, 512, 256
    layer = mp.Layer(mp.make_config(T, E, k, 1, 1, H, 0))
    st = layer_inputs(T, E, H, F, layer.device, 11)
    q = (q1, _), (q2, _) = [layer.quantize_weights4(st[n], transposed=True) for n in ("w1", "w2")]
    r = passes(layer, st, mp.make_gate("sigmoid", scale=2.5), q)
    assert layer.status() == 0
    f = in_64_bits(r["idx"], 2.5)
    at = [t.cpu().double().requires_grad_() for t in (st["hidden"], st["logits"], refs4.values(q1), refs4.values(q2))]
    g_out = st["g_out"].cpu().double()
    out = f(*at)
    want = torch.autograd.grad(out, at, g_out)
    for name, w, limit in (("out", out.detach(), 0.125), ("g_w1", want[2], 0.125), ("g_w2", want[3], 0.125),
                           ("g_logits", want[1], 0.125), ("g_hidden", want[0], 0.42)):
        got = r[name].cpu().double()
        print("%s: apart %.3f share %.3f" % (name, apart(got, w), share(got, w)), flush=True)
        assert apart(got, w) <= limit and abs(share(got, w) - 1) <= limit, name
    # the formula's gradient along what the GPU found, by differences
    for i, name in enumerate(("g_hidden", "g_logits", "g_w1", "g_w2")):
        step = r[name].cpu().double()
        h = 1e-5 / float(step.norm())
        moved = [[t.detach() + (sign * h * step if i == j else 0) for j, t in enumerate(at)] for sign in (1, -1)]
        slope = float(((f(*moved[0]) - f(*moved[1])) * g_out).sum()) / (2 * h)
        exact = float((want[i] * step).sum())
        assert exact > 0 and abs(slope - exact) <= 1e-6 * exact, name
    layer.close()


def test_the_ways_through_a_layer(mp):
    """32 tokens through experts() and through the plan, matrices in 4 and in 8 bits, rows in 8 and in 4: each step's
    products from the operands that it had, and the results side by side.

    Two ways that round rows and activations to e4m3 in blocks of their own are sqrt(4) 2^-4 = 0.125 of a result's length
    apart at the most, with the argument of the test before; with rows and activations in 4 bits on one side
    sqrt(2 / 25 + 2 / 256) = 0.30."""
    T, E, k, H, F = 32, 16, 4, 512, 160
    layer = mp.Layer(mp.make_config(T, E, k, 1, 1, H, 0))
    st = layer_inputs(T, E, H, F, layer.device, 3)
    router = mp.make_gate("softmax", scale=1.5)
    route, weight = layer.gate(st["logits"], router, bias=st["bias"])
    layer.plan()
    rows = layer.dispatch(st["hidden"]).dispatch.view(BF)
    spans, many = spans_of(layer), {}
    for bits, quant, matmul in ((8, layer.quantize_weights, layer.matmul), (4, layer.quantize_weights4, layer.matmul4)):
        q1, q2 = quant(st["w1"]), quant(st["w2"])
        few = layer.experts(st["hidden"], weight, q1, q2).cpu().double()
        many[bits] = layer.combine_weighted(matmul(layer.swiglu(matmul(layer.quantize(rows), q1)), q2), weight).cpu().double()
        print("few and many, %d bits: apart %.3f share %.3f" % (bits, apart(few, many[bits]), share(few, many[bits])), flush=True)
        assert apart(few, many[bits]) <= 0.125 and abs(share(few, many[bits]) - 1) <= 0.125
    x = layer.quantize4(rows)
    y1 = layer.matmul4(x, q1)
    a = layer.swiglu4(y1)
    y2 = layer.matmul4(a, q2)
    four = layer.combine_weighted(y2, weight).cpu().double()
    torch.cuda.synchronize()
    assert layer.status() == 0
    assert products(spans, refs4.values(x), refs4.values(q1), y1.cpu().double())
    assert products(spans, refs4.values(a), refs4.values(q2), y2.cpu().double())
    # each within half a step of e2m1, a fifth of the value or a quarter of the scale
    for b, want, off in ((x, rows.cpu().double(), 0.0), (a, refs.swiglu(y1.cpu().double()), 2.0 ** -19)):
        each = spread4(b)
        ratio = want.abs() / each
        half = torch.where(ratio < 2, 0.25, torch.where(ratio < 4, 0.5, 1.0)) * each
        assert ((refs4.values(b) - want).abs() <= half * (1 + 2.0 ** -10) + 2 * off * want.abs()).all()
    pos = layer.dispatch_out.slot_pos.cpu().long().view(T, k)
    y, w = y2.cpu().double()[pos], weight.cpu().double()[..., None]
    want, mag = (y * w).sum(1), (y.abs() * w).sum(1)
    assert ((four - want).abs() <= 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * (k + 2) * 2.0 ** -24 * mag).all()
    print("rows in 4 and 8 bits: apart %.3f share %.3f" % (apart(four, many[4]), share(four, many[4])), flush=True)
    assert apart(four, many[4]) <= 0.30 and abs(share(four, many[4]) - 1) <= 0.30
    layer.close()
