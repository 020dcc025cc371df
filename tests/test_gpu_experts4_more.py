"""The 4-bit operators and the layer of few tokens as they are used: a whole layer with its backward pass, captured
graphs, several streams, memory past 32 bits, rows that belong to nobody."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import expert4_refs as refs4
from tests import expert_refs as refs
from tests.test_gpu_experts4 import BF, few_layer, instances, layer_for, normal, u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import load_balance_planning_amd as m
    m.lib()
    return m


# ---- a layer ----------------------------------------------------------------------

def layer_inputs(T, E, H, F, dev, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    n = lambda *s, by=1.0: (by * torch.randn(*s, generator=g, device=dev)).to(BF)
    return dict(logits=torch.randn(T, E, generator=g, device=dev), bias=0.1 * torch.randn(E, generator=g, device=dev),
                hidden=n(T, H), w1=n(E, 2 * F, H, by=H ** -0.5), w2=n(E, H, F, by=F ** -0.5), g_out=n(T, H))


def train(mp, layer, st, router, q):
    """One forward and backward pass with matrices in 4 bits, rows and gradients in 8."""
    (q1, t1), (q2, t2) = q
    route, weight = layer.gate(st["logits"], router, bias=st["bias"])
    layer.plan()
    x = layer.quantize(layer.dispatch(st["hidden"]).dispatch)
    y1 = layer.matmul4(x, q1)
    a = layer.swiglu(y1)
    y2 = layer.matmul4(a, q2)
    out = layer.combine_weighted(y2, weight)
    g_y2, g_weight = layer.combine_grad(y2, st["g_out"], weight)
    g2 = layer.quantize(g_y2)
    g_a = layer.matmul4(g2, t2)
    g1 = layer.swiglu_grad(y1, g_a)
    g_hidden = layer.combine_weighted(layer.matmul4(g1, t1))
    return dict(x=x, y1=y1, a=a, y2=y2, out=out, g2=g2, g_a=g_a, g1=g1, g_hidden=g_hidden, g_w2=layer.wgrad(g2, a),
                g_w1=layer.wgrad(g1, x), g_logits=layer.gate_grad(st["logits"], router, g_weight), weight=weight)


def spans_of(layer):
    n = int(layer.plan_out.n_inst.item())
    off, e = layer.dispatch_out.inst_offset.cpu().tolist(), layer.plan_out.inst_expert.cpu().tolist()
    return [(e[i], off[i], off[i + 1]) for i in range(n)]


def test_a_layer_forward_and_backward(mp):
    """Every product of a pass, with 4-bit matrices in the place of 8-bit ones, from the operands it had; the gradients
    of its rows are those of the forward product's formula, and differences of it."""
    T, E, k, R, H, F = 96, 8, 2, 2, 264, 72
    layer = mp.Layer(mp.make_config(T, E, k, R, 1, H, 2, expert_bytes=0))
    st = layer_inputs(T, E, H, F, layer.device)
    q = [layer.quantize_weights4(st[n], transposed=True) for n in ("w1", "w2")]
    r = train(mp, layer, st, mp.make_gate("sigmoid", scale=2.5), q)
    torch.cuda.synchronize()
    assert layer.status() == 0
    spans = spans_of(layer)
    for name, x, w, cols in (("y1", r["x"], q[0][0], H), ("y2", r["a"], q[1][0], F), ("g_a", r["g2"], q[1][1], H)):
        xv, wv = refs.values(x, T * k), refs4.values(w)
        sx, sw = refs4.spread(x.scale.cpu().double(), 128, cols), refs4.spread(refs4.scales(w), 32, cols)
        got = r[name].cpu().double()
        for e, a, z in spans:
            want = xv[a:z] @ wv[e].t()
            bound = refs4.rounded(want, refs4.added(xv[a:z], wv[e]) + refs4.cut(xv[a:z], sx[a:z], wv[e], sw[e]))
            assert ((got[a:z] - want).abs() <= bound).all(), name
    # y = x w^t is linear: its gradient for x is dy w, and that is what differences of dy . y say
    wt = refs4.values(q[1][1])
    g = refs.values(r["g2"], T * k)
    for e, a, z in spans:
        if a == z:
            continue
        x = torch.randn(F, dtype=torch.float64, generator=torch.Generator().manual_seed(e))
        f = lambda v: (wt[e].t() @ v) @ g[a]
        grad, h = g[a] @ wt[e].t(), 1e-4
        for c in (0, F // 2, F - 1):
            d = torch.zeros(F, dtype=torch.float64)
            d[c] = h
            assert abs((f(x + d) - f(x - d)) / (2 * h) - grad[c]) <= 1e-8 * (1 + grad.abs().max())
    layer.close()


def test_few_tokens_and_many(mp):
    """The two ways through a layer of 32 tokens.  Each rounds the rows and the activations to e4m3, by at most 2^-4 of a
    value; random matrices keep relative lengths, so that the results are not further apart than 4 * 2^-4."""
    T, E, k, H, F = 32, 16, 4, 512, 160
    layer = mp.Layer(mp.make_config(T, E, k, 1, 1, H, 0))
    st = layer_inputs(T, E, H, F, layer.device, 3)
    router = mp.make_gate("softmax", scale=1.5)
    for quant, matmul in ((layer.quantize_weights4, layer.matmul4), (layer.quantize_weights, layer.matmul)):
        q1, q2 = quant(st["w1"]), quant(st["w2"])
        route, weight = layer.gate(st["logits"], router, bias=st["bias"])
        few = layer.experts(st["hidden"], weight, q1, q2)          # the layer's own top-k
        layer.plan()
        y2 = matmul(layer.swiglu(matmul(layer.quantize(layer.dispatch(st["hidden"]).dispatch), q1)), q2)
        many = layer.combine_weighted(y2, weight)
        torch.cuda.synchronize()
        few, many = few.cpu().double(), many.cpu().double()
        assert float((few - many).norm() / many.norm()) <= 4 * 2.0 ** -4
    # rows and activations in 4 bits: half a step of e2m1 is at most a fifth of a value, or a quarter of the scale
    y2 = layer.matmul4(layer.swiglu4(layer.matmul4(layer.quantize4(layer.dispatch_out.dispatch),
                                                   layer.quantize_weights4(st["w1"]))), layer.quantize_weights4(st["w2"]))
    four = layer.combine_weighted(y2, weight).cpu().double()
    assert float((four - many).norm() / many.norm()) <= 1
    assert layer.status() == 0
    layer.close()


# ---- graphs -----------------------------------------------------------------------

def raw(t):
    return t.view(torch.uint8)


def test_a_captured_pass_replays(mp):
    T, E, k, R, H, F = 64, 16, 4, 2, 264, 72
    cfg = lambda: mp.make_config(T, E, k, R, 1, H, 2, expert_bytes=0)
    layer, other = mp.Layer(cfg()), mp.Layer(cfg())
    router = mp.make_gate("sigmoid", scale=2.5)
    st = layer_inputs(T, E, H, F, layer.device)
    q = [layer.quantize_weights4(st[n], transposed=True) for n in ("w1", "w2")]

    def whole(layer, st, q):
        for b, n in zip(q, ("w1", "w2")):   # the matrices again, in place
            layer.quantize_weights4(st[n], transposed=True, out=b)
        r = train(mp, layer, st, router, q)
        four = layer.swiglu4(layer.matmul4(layer.quantize4(layer.dispatch_out.dispatch), q[0][0]))
        return dict(out=r["out"], g_hidden=r["g_hidden"], g_w1=r["g_w1"], g_w2=r["g_w2"], y4=layer.matmul4(four, q[1][0]),
                    v=layer.values4(q[0][1]), few=layer.experts(st["hidden"], r["weight"], q[0][0], q[1][0]))

    whole(layer, st, q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = whole(layer, st, q)
    for i in range(4):
        new = layer_inputs(T, E, H, F, layer.device, seed=i)
        for n, t in new.items():
            st[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in res.items()}
        want = whole(other, new, [other.quantize_weights4(new[n], transposed=True) for n in ("w1", "w2")])
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(raw(got[n]), raw(want[n])), (i, n)
    assert layer.status() == 0 and other.status() == 0
    layer.close()
    other.close()


@pytest.mark.parametrize("T,E,k,H,f,bits", [(1, 8, 4, 512, 96, 4), (12, 32, 4, 2048, 300, 4), (64, 16, 4, 768, 256, 8),
                                            (40, 64, 8, 512, 520, 4)])
def test_captured_few_tokens_replay(mp, T, E, k, H, f, bits):
    """Replays with other tokens, weights and top-k in the same memory, eager calls in between."""
    layer, idx, weight, w1, w2 = few_layer(mp, T, E, k, H, f, bits, 1)
    dev = layer.device
    hidden = normal(1, T, H).to(dev)
    call = lambda i, w, h, **kw: layer.experts(h, w, w1, w2, topk_idx=i, **kw)
    call(idx, weight, hidden)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(idx, weight, hidden)
    for s in range(5):
        g = torch.Generator(device=dev).manual_seed(s)
        hidden.copy_(torch.randn(T, H, generator=g, device=dev).to(BF))
        idx.copy_(torch.rand(T, E, generator=g, device=dev).argsort(-1)[:, :k].to(torch.int32))
        weight.copy_(torch.rand(T, k, generator=g, device=dev))
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(call(idx.clone(), weight.clone(), hidden.clone()), got), s
        graph.replay()
        assert torch.equal(out, got)
    assert layer.status() == 0
    layer.close()


# ---- streams ----------------------------------------------------------------------

def test_one_layer_on_two_streams(mp):
    """Products and few-token calls of one handle side by side, eager and as captured graphs."""
    T, E, k, H, f = 24, 16, 4, 768, 200
    layer, idx, weight, w1, w2 = few_layer(mp, T, E, k, H, f, 4, 1)
    dev = layer.device
    hidden = [normal(i, T, H).to(dev) for i in range(2)]
    loads = [T * k // 2, 0, T * k - T * k // 2]
    plan, off, _ = instances(mp, layer, loads, [3, 1, 0])
    x = [layer.quantize4(normal(7, T * k, H).to(dev)), layer.quantize(normal(8, T * k, H).to(dev))]
    few = [lambda s=None, i=i: layer.experts(hidden[i], weight, w1, w2, topk_idx=idx, stream=s) for i in range(2)]
    product = [lambda s=None, i=i: layer.matmul4(x[i], w1, plan=plan, inst_offset=off, stream=s) for i in range(2)]
    calls = [(few[0], few[1]), (few[0], product[0]), (product[1], few[1])]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for pair in calls:
        want = [c().clone() for c in pair]
        torch.cuda.synchronize()
        for _ in range(5):
            got = [[c(s) for _ in range(4)] for c, s in zip(pair, streams)]
            torch.cuda.synchronize()
            assert all(torch.equal(t, w) for ts, w in zip(got, want) for t in ts)
        graphs, got = [torch.cuda.CUDAGraph() for _ in range(2)], []
        for g, c in zip(graphs, pair):
            with torch.cuda.graph(g):
                got.append(c())
        for _ in range(5):
            for t in got:
                t.fill_(3)
            torch.cuda.synchronize()
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(t, w) for t, w in zip(got, want))
    assert layer.status() == 0
    layer.close()


def test_no_result_of_a_side_stream_goes_to_another(mp):
    """What a call on a stream returns, and the memory it works in, is that stream's: tensors of the current stream made
    right after it get none of it while the call may still run."""
    T, E, k, H, f = 32, 8, 2, 2048, 1024
    layer, idx, weight, w1, w2 = few_layer(mp, T, E, k, H, f, 4, 1)
    dev = layer.device
    hidden, rows = normal(1, T, H).to(dev), normal(2, T * k, H).to(dev)
    plan, off, _ = instances(mp, layer, [T * k], [0])
    x = layer.quantize4(rows)
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device=dev)
    calls = dict(experts=lambda s: layer.experts(hidden, weight, w1, w2, topk_idx=idx, stream=s),
                 quantize4=lambda s: layer.quantize4(rows, stream=s).q, values4=lambda s: layer.values4(x, stream=s),
                 swiglu4=lambda s: layer.swiglu4(rows, stream=s).scale,
                 matmul4=lambda s: layer.matmul4(x, w1, plan=plan, inst_offset=off, stream=s),
                 weights=lambda s: layer.quantize_weights4(rows.view(1, T * k, H), stream=s).q)
    for name, call in calls.items():
        want = raw(call(None)).clone()
        torch.cuda.synchronize()
        for _ in range(3):
            with torch.cuda.stream(side):
                for _ in range(4):
                    busy = busy @ busy * 1e-4
            got = call(side)
            others = [torch.full((got.numel() * got.element_size() + 512,), 0xaa, dtype=torch.uint8, device=dev)
                      for _ in range(8)]
            torch.cuda.synchronize()
            assert torch.equal(raw(got), want), name
            assert all((o == 0xaa).all() for o in others), name
    with pytest.raises(ValueError):
        layer.experts(hidden, weight, w1, w2, topk_idx=idx, out=hidden)
    layer.close()


# ---- sizes ------------------------------------------------------------------------

def test_offsets_past_32_bits(mp):
    """More than 2^32 bytes of rows: their end as by itself."""
    rows, cols = 700000, 7168
    print("past 32 bits: %d rows of %d" % (rows, cols), flush=True)
    layer = layer_for(mp, rows, 4)
    dev = layer.device
    x = torch.randn(rows, cols, device=dev, dtype=BF, generator=torch.Generator(device=dev).manual_seed(1))
    b = layer.quantize4(x)
    last = x[-70:].clone()
    alone = layer.quantize4(last)
    assert torch.equal(u8(b.q[-70:]), u8(alone.q)) and torch.equal(u8(b.scale[:, -70:]), u8(alone.scale))
    assert torch.equal(layer.values4(b)[-70:], layer.values4(alone))
    half = layer.swiglu4(x)
    assert torch.equal(u8(half.q[-70:]), u8(layer.swiglu4(last).q))
    del x, half
    n = 160
    plan, off, _ = instances(mp, layer, [rows - 70, 0, 70], [0, 1, 3])
    w = layer.quantize_weights4(normal(2, 4, n, cols, scale=0.02).to(dev))
    y = layer.matmul4(b, w, plan=plan, inst_offset=off)
    xv, wv = refs4.values(alone), refs4.values(mp.Blocks4(w.q[3:], w.scale[3:], cols))[0]
    want = xv @ wv.t()
    assert ((y[-70:].cpu().double() - want).abs() <= refs4.rounded(want, refs4.added(xv, wv))).all()
    assert layer.status() == 0
    layer.close()


def test_matrices_past_32_bits(mp):
    """The last of experts whose matrices take more than 2^32 bytes, in the products and for few tokens."""
    T, E, H, f = 3, 34, 16384, 8192
    print("matrices past 32 bits: %d experts of %d x %d" % (E, 2 * f, H), flush=True)
    layer = mp.Layer(mp.make_config(T, E, 1, 1, 1, H, 0), cooc=False)
    dev = layer.device
    g = torch.Generator(device=dev).manual_seed(1)
    w1 = layer.quantize_weights4(torch.randn(E, 2 * f, H, device=dev, dtype=BF, generator=g) * 2 ** -7)
    w2 = layer.quantize_weights4(torch.randn(E, H, f, device=dev, dtype=BF, generator=g) * 2 ** -7)
    assert w1.q.numel() > 1 << 32
    hidden = normal(3, T, H).to(dev)
    idx, weight = torch.full((T, 1), E - 1, dtype=torch.int32, device=dev), torch.ones(T, 1, device=dev)
    one = mp.Layer(mp.make_config(T, 1, 1, 1, 1, H, 0), cooc=False)
    cut = lambda b: mp.Blocks4(raw(b.q)[E - 1:].clone().view(b.q.dtype), raw(b.scale)[E - 1:].clone().view(b.scale.dtype), b.cols)
    c1, c2 = cut(w1), cut(w2)
    got, want = layer.experts(hidden, weight, w1, w2, topk_idx=idx), one.experts(hidden, weight, c1, c2, topk_idx=idx * 0)
    # the shares of the second product may be others: fp32 sums in another order, and bf16's half step each way
    assert torch.allclose(got.float(), want.float(), rtol=2.0 ** -7, atol=1e-5 * float(want.float().abs().max()))
    x = layer.quantize4(hidden)
    plan, off, _ = instances(mp, layer, [T], [E - 1])
    plan1, off1, _ = instances(mp, one, [T], [0])
    assert torch.equal(layer.matmul4(x, w1, plan=plan, inst_offset=off), one.matmul4(x, c1, plan=plan1, inst_offset=off1))
    assert layer.status() == 0 and one.status() == 0
    layer.close()
    one.close()


@pytest.mark.parametrize("rows,n", [(40, 24), (4000, 300), (9000, 2048)])
def test_rows_of_no_instance_are_left_alone(mp, rows, n):
    """Rows behind the last instance and between two of them, in every kernel of the products."""
    layer = layer_for(mp, rows, 3)
    dev = layer.device
    w = layer.quantize_weights4(normal(2, 3, n, 136).to(dev))
    a, b, c, d = rows // 8, rows // 2, rows // 2 + 3, rows - 5
    off = torch.tensor([a, b, c, d], dtype=torch.int32, device=dev)[:4]
    plan, _, _ = instances(mp, layer, [1, 1, 1], [0, 2, 1])
    plan.inst_expert[1] = 7        # the middle instance is bad: its rows stay too
    for x in (layer.quantize4(normal(1, rows, 136).to(dev)), layer.quantize(normal(1, rows, 136).to(dev))):
        y = torch.full((rows, n), 7.0, dtype=BF, device=dev)
        layer.matmul4(x, w, plan=plan, inst_offset=off, out=y)
        assert layer.status() == mp.MOE_STATUS_PLAN_CHECK
        for p, q in ((0, a), (b, c), (d, rows)):
            assert (y[p:q] == 7).all()
        assert (y[a:b] != 7).any() and (y[c:d] != 7).any()
    layer.close()


@pytest.mark.parametrize("H,f", [(1, 1), (32, 256), (7168, 33), (4100, 64), (9000, 40), (40, 9001)])
def test_few_tokens_of_any_width(mp, H, f):
    """Widths at which the second product's channels are shared out differently, against the same tokens one by one."""
    layer, idx, weight, w1, w2 = few_layer(mp, 6, 5, 2, H, f, 4, 3)
    one = mp.Layer(mp.make_config(1, 5, 2, 1, 1, H, 0), cooc=False)
    hidden = normal(4, 6, H).to(layer.device)
    together = layer.experts(hidden, weight, w1, w2, topk_idx=idx).float()
    for t in range(6):
        alone = one.experts(hidden[t:t + 1], weight[t:t + 1], w1, w2, topk_idx=idx[t:t + 1]).float()
        assert torch.allclose(alone[0], together[t], rtol=2.0 ** -7, atol=2e-3 * float(together.abs().max()))
    assert layer.status() == 0 and one.status() == 0
    layer.close()
    one.close()


def test_results_into_given_memory(mp):
    layer, idx, weight, w1, w2 = few_layer(mp, 16, 4, 2, 300, 64, 4, 3)
    dev = layer.device
    rows = normal(1, 32, 300).to(dev)
    b = layer.quantize4(rows)
    raw(b.q).fill_(0xff)
    raw(b.scale).fill_(0)
    again = layer.quantize4(rows, out=b)
    fresh = layer.quantize4(rows)
    assert again is b and torch.equal(u8(b.q), u8(fresh.q)) and torch.equal(u8(b.scale), u8(fresh.scale))
    out = torch.full((16, 300), 7.0, dtype=BF, device=dev)
    assert layer.experts(rows[:16], weight, w1, w2, topk_idx=idx, out=out) is out
    assert torch.equal(out, layer.experts(rows[:16], weight, w1, w2, topk_idx=idx))
    bits = layer.experts(rows[:16].view(torch.int16), weight, w1, w2, topk_idx=idx)
    assert bits.dtype == torch.int16 and torch.equal(bits, out.view(torch.int16))
    layer.close()
