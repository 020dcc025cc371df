"""moex_gate where fp32 does not tell the order: long ties with a few experts a little above or below, group values
whose terms cancel or whose sum leaves fp32, against the selection in 64 bits.

Every case runs with co-selection counts (two launches) and without (one workgroup where the tokens are few)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from tests import expert_refs as refs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import load_balance_planning_amd as m
    m.lib()
    return m


def check(mp, x, bias, k, kind, groups=(1, 1, 1), cooc=True, R=1):
    """Indices, counts and weights; the weight's bound is that of tests/test_gpu_gate.py at a range of 200, and what a
    score below 2^-126 loses: fp32 values are 2^-149 apart there, the exponential and its product with 1 / sum round by
    half of that each, so a weight scale * s / (sum s + 1e-20) is off by up to scale * 2^-149 / (sum s + 1e-20)."""
    T, E = x.shape
    layer = mp.Layer(mp.make_config(T, E, k, R, 1, 8, 0), cooc=cooc)
    for t in (layer.route_out.topk_idx, layer.route_out.expert_count, layer.route_out.omega):
        t.fill_(-7)
    r, w = layer.gate(x.to(layer.device), mp.make_gate(kind, *groups, True, 2.5),
                      bias=None if bias is None else bias.to(layer.device))
    torch.cuda.synchronize()
    assert layer.status() == 0
    idx = refs.select(x.double(), None if bias is None else bias.double(), kind, k, *groups)
    got = r.topk_idx.cpu().long()
    assert torch.equal(got, idx), "%d of %d tokens differ, first %s for %s" % (
        int((got != idx).any(1).sum()), T, got[(got != idx).any(1)][:1].tolist(), idx[(got != idx).any(1)][:1].tolist())
    want = refs.gate_weights(x.double(), idx, kind, True, 2.5)
    total = refs.scores(x.double(), kind).gather(1, idx).sum(-1, keepdim=True) + 1e-20
    assert ((w.cpu().double() - want).abs() <= (E / 8 + 2 * k + 432) * 2.0 ** -24 * want.abs() + 2.5 * 2.0 ** -149 / total
            + 1e-37).all()
    omega = torch.nn.functional.one_hot(idx, E).sum(1).view(R, T // R, E).sum(1).int()
    assert torch.equal(r.omega.cpu(), omega) and torch.equal(r.expert_count.cpu(), omega.sum(0).int())
    layer.close()


def ties(T, E, seed, kind):
    """Rows of equal logits in which a few experts, at any index, stand above or below by less than fp32 tells."""
    g = torch.Generator().manual_seed(seed)
    x = torch.zeros(T, E)
    for t in range(T):
        at = torch.randperm(E, generator=g)
        if t % 5 == 0:
            x[t, E - 1 - t % (E // 2)] = 1e-9                    # one above
        elif t % 5 == 1:
            x[t, at[:3]] = torch.tensor([1e-9, 3e-9, 2e-9])      # several, each its own
        elif t % 5 == 2:
            x[t, t % 7] = -1e-9                                  # one below, among the lowest
        elif t % 5 == 3:
            x[t, at[: E // 2]] = 1e-9                            # half of them
    return x


SHAPES = [(32, 256, 8), (64, 256, 8), (4100, 256, 8), (16, 896, 16), (40, 896, 16), (16, 2048, 8), (40, 2048, 8), (4098, 128, 4), (20, 60, 2)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("cooc", [True, False])
def test_long_ties_with_a_few_apart(mp, T, E, k, kind, cooc):
    print("long ties T=%d E=%d k=%d %s cooc=%s" % (T, E, k, kind, cooc), flush=True)
    R = 2 if E > 1024 else 1
    x = ties(T, E, T + E, kind)
    level = torch.full((E,), 0.25)
    unit = level.clone()
    unit[E - E // 5] = 0.25 + 2.0 ** -25    # below a unit of 0.75
    for groups in ((1, 1, 1), (4, 2, 2), (4, 2, 1)):
        for bias in (torch.zeros(E), level, unit):
            check(mp, x, bias, k, kind, groups, cooc, R)
        check(mp, torch.zeros(T, E), unit, k, kind, groups, cooc, R)


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("cooc", [True, False])
def test_small_scores_under_a_shared_bias(mp, T, E, k, cooc):
    """Most experts masked, score 0; live ones whose scores vanish beside the bias in fp32 come before them."""
    print("masked ties T=%d E=%d k=%d cooc=%s" % (T, E, k, cooc), flush=True)
    R = 2 if E > 1024 else 1
    g = torch.Generator().manual_seed(E)
    x = torch.full((T, E), -torch.inf)
    for t in range(T):
        at = torch.randperm(E, generator=g)[: 1 + t % (k + 2)]
        x[t, at] = -20.0 - torch.arange(len(at))
        x[t, at[0]] = 0.0
    for groups in ((1, 1, 1), (4, 3, 2)):
        check(mp, x, torch.ones(E), k, "softmax", groups, cooc, R)
        check(mp, x, torch.ones(E), k, "sigmoid", groups, cooc, R)


@pytest.mark.parametrize("T", [24, 64, 4100])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("per,n_group", [(8, 8), (16, 16), (5, 12), (2, 64)])
@pytest.mark.parametrize("C", [1e2, 1e3, 1e4, 1e30, 1.9e38])
def test_group_values_whose_terms_cancel(mp, T, kind, per, n_group, C):
    """One expert of each group at +C, the others at -C: the sums are of the scores' size, their error of C's."""
    print("cancelling groups T=%d %s %d x %d C=%g" % (T, kind, n_group, per, C), flush=True)
    E = per * n_group
    g = torch.Generator().manual_seed(T + E)
    x = 1e-4 * torch.randn(T, E, generator=g)
    bias = torch.full((n_group, per), -C)
    bias[torch.arange(n_group), torch.randint(0, per, (n_group,), generator=g)] = C
    for cooc in (True, False):
        check(mp, x, bias.flatten(), 2, kind, (n_group, 3, 2), cooc)


@pytest.mark.parametrize("T", [24, 64, 4100])
@pytest.mark.parametrize("cooc", [True, False])
def test_group_values_past_fp32(mp, T, cooc):
    """Sums of two biases that overflow in fp32, of either sign, beside groups of -infinity and ordinary ones."""
    print("groups past fp32 T=%d cooc=%s" % (T, cooc), flush=True)
    E, n_group, k = 64, 8, 4
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, E, generator=g)
    for n_top in (1, 2, 3, 5, 7):
        bias = torch.zeros(n_group, E // n_group)
        bias[1], bias[4] = 3.3e38, 3.0e38      # both sums are infinite in fp32, and 1 is before 4,
        bias[4, 0] = 3.4e38                    # though 4 has the largest expert
        bias[2, :1] = 3.4e38                   # one large term
        bias[0], bias[6] = -3.3e38, -3.0e38    # 6 before 0, both before -infinity
        bias[5] = -torch.inf
        bias[7, 1:] = -torch.inf               # its second largest is -infinity
        for top in (1, 2):
            check(mp, x, bias.flatten(), k, "sigmoid", (n_group, n_top, top), cooc)
            check(mp, x, bias.flatten(), k, "softmax", (n_group, n_top, top), cooc)


# ---- the same borders in one workgroup (no co-selection counts, few tokens) as in two launches ------------------

FEW = [(16, 256, 8, (1, 1, 1)), (32, 256, 8, (8, 4, 2)), (13, 896, 16, (8, 4, 2)), (16, 100, 5, (10, 3, 1)), (32, 64, 4, (1, 1, 1))]


@pytest.mark.parametrize("T,E,k,groups", FEW)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_ties_of_few_tokens(mp, T, E, k, groups, kind):
    g = torch.Generator().manual_seed(E)
    coarse = (torch.randn(T, E, generator=g) * 4).round() / 4
    near = torch.full((T, E), 1.5) + torch.randint(0, 50, (T, E), generator=g) * 2.0 ** -23
    bias = torch.randint(0, 3, (E,), generator=g) * 2.0 ** -24
    for x, b in ((coarse, None), (coarse, torch.zeros(E)), (torch.zeros(T, E), torch.zeros(E)), (near, None), (near, bias),
                 (near + torch.randn(T, E, generator=g), 1e-7 * torch.randn(E, generator=g))):
        check(mp, x, b, k, kind, groups, cooc=False)


@pytest.mark.parametrize("T,E,k,groups", FEW)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_masked_and_extreme_logits_of_few_tokens(mp, T, E, k, groups, kind, biased):
    g = torch.Generator().manual_seed(E + 1)
    x, b = torch.randn(T, E, generator=g), 0.1 * torch.randn(E, generator=g)
    low = torch.finfo(torch.float32).min
    x[0], x[1, 5:], x[2, 3:], x[3], x[4, ::2] = -torch.inf, -torch.inf, -torch.inf, low, low
    x[5] = torch.linspace(-100, 100, E)
    x[6] = torch.linspace(1e-30, 64e-30, E)
    x[7, : E // 2], x[7, E // 2:] = -0.0, 0.0
    if kind == "sigmoid":
        x[8, :3] = torch.inf
    check(mp, x, b if biased else None, k, kind, groups, cooc=False)
    if biased:
        b[: E // 2] = -torch.inf
        check(mp, x, b, k, kind, groups, cooc=False)


@pytest.mark.parametrize("T,E,k,groups", FEW)
def test_wrong_inputs_of_few_tokens(mp, T, E, k, groups):
    """The status tells, the indices stay distinct experts, and other tokens are as without the wrong one."""
    g = torch.Generator().manual_seed(E + 2)
    x, b = torch.randn(T, E, generator=g), 0.1 * torch.randn(E, generator=g)
    nan_x, inf_x, nan_b = x.clone(), x.clone(), b.clone()
    nan_x[3, 7], inf_x[3, 1], nan_b[9] = torch.nan, torch.inf, torch.nan
    for xs, bias, kind, want in ((nan_x, None, "softmax", 1), (nan_x, b, "sigmoid", 1), (inf_x, b, "softmax", 1),
                                 (inf_x, b, "sigmoid", 0), (x, nan_b, "sigmoid", 1), (x, torch.full((E,), torch.inf), "softmax", 1)):
        layer = mp.Layer(mp.make_config(T, E, k, 1, 1, 8, 0), cooc=False)
        r, _ = layer.gate(xs.to(layer.device), mp.make_gate(kind, *groups), bias=None if bias is None else bias.to(layer.device))
        assert layer.status() == (mp.MOE_STATUS_NAN_LOGIT if want else 0)
        idx = r.topk_idx.cpu().long()
        assert all(len(set(row.tolist())) == k and 0 <= min(row) and max(row) < E for row in idx)
        if bias is None or bias is b:
            good = [t for t in range(T) if t != 3]
            ref = refs.select(x.double(), None if bias is None else b.double(), kind, k, *groups)
            assert torch.equal(idx[good], ref[good])
        layer.close()


@pytest.mark.parametrize("T,E,k,groups", FEW)
def test_unaligned_logits_of_few_tokens(mp, T, E, k, groups):
    g = torch.Generator().manual_seed(E + 3)
    x, b = torch.randn(T, E, generator=g), 0.1 * torch.randn(E, generator=g)
    layer = mp.Layer(mp.make_config(T, E, k, 1, 1, 8, 0), cooc=False)
    gate, bd = mp.make_gate("sigmoid", *groups, True, 2.5), b.to(layer.device)
    view = torch.empty(T * E + 1, device=layer.device)[1:].view(T, E).copy_(x)
    r, w = layer.gate(view, gate, bias=bd)
    idx = r.topk_idx.clone()
    r, w2 = layer.gate(x.to(layer.device), gate, bias=bd)
    assert torch.equal(r.topk_idx, idx) and torch.equal(w, w2) and layer.status() == 0
    assert torch.equal(idx.cpu().long(), refs.select(x.double(), b.double(), "sigmoid", k, *groups))
    layer.close()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_the_largest_scale(mp, kind):
    """At 2^32 a masked row has weights and gradients of zero, not of infinity times zero; above it the call is refused."""
    T, E, k = 16, 32, 4
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(1))
    x[3] = -torch.inf
    layer = mp.Layer(mp.make_config(T, E, k, 1, 1, 8, 0), cooc=False)
    xd, ones = x.to(layer.device), torch.ones(T, k, device=layer.device)
    for scale in (2.0 ** 32, -2.0 ** 32):
        gate = mp.make_gate(kind, scale=scale)
        r, w = layer.gate(xd, gate)
        g = layer.gate_grad(xd, gate, 1e6 * ones)
        assert torch.isfinite(w).all() and torch.isfinite(g).all() and (w[3] == 0).all() and (g[3] == 0).all()
        want = refs.gate_weights(x.double(), r.topk_idx.cpu().long(), kind, True, scale)
        assert ((w.cpu().double() - want).abs() <= (E / 8 + 2 * k + 432) * 2.0 ** -24 * want.abs()).all()
    for scale in (2.0 ** 33, -1e30, float("inf"), float("nan")):
        for call in (lambda gate: layer.gate(xd, gate), lambda gate: layer.gate_grad(xd, gate, ones)):
            with pytest.raises(mp.MoePlanError) as e:
                call(mp.make_gate(kind, scale=scale))
            assert e.value.code == mp.MOE_ERR_INVALID_ARG
    assert layer.status() == 0
    layer.close()


@pytest.mark.parametrize("cooc", [True, False])
def test_sigmoid_far_below_zero(mp, cooc):
    """Scores down to fp32's smallest, alone in their row: weights of s / (s + 1e-20), and their gradients."""
    T, E = 32, 8
    x = torch.linspace(-104, -60, T * E).view(T, E)
    for k in (1, 3):
        check(mp, x, None, k, "sigmoid", cooc=cooc)
        layer = mp.Layer(mp.make_config(T, E, k, 1, 1, 8, 0), cooc=cooc)
        for renorm in (True, False):
            gate, xd = mp.make_gate("sigmoid", renorm=renorm, scale=2.5), x.to(layer.device)
            r, w = layer.gate(xd, gate)
            gw = torch.randn(T, k, generator=torch.Generator().manual_seed(k))
            got = layer.gate_grad(xd, gate, gw.to(layer.device)).cpu().double()
            idx, x64 = r.topk_idx.cpu().long(), x.double().requires_grad_()
            want, = torch.autograd.grad(refs.gate_weights(x64, idx, "sigmoid", renorm, 2.5), x64, gw.double())
            # the share of the magnitudes that are added, and half of 2^-149 for each score that goes in
            s = refs.scores(x.double(), "sigmoid").gather(1, idx)
            size = 2.5 * gw.double().abs()
            if renorm:
                S = s.sum(-1, keepdim=True) + 1e-20
                size = 2.5 / S * (gw.double().abs() + (gw.double().abs() * s).sum(-1, keepdim=True) / S)
            bound = torch.zeros(T, E, dtype=torch.float64).scatter(
                1, idx, size * (s * (2 * k + 432) * 2.0 ** -24 + (k + 1) * 2.0 ** -149)) + 2.0 ** -149
            assert ((got - want).abs() <= bound).all()
        assert layer.status() == 0
        layer.close()


@pytest.mark.parametrize("T,E,k,groups", FEW)
def test_few_tokens_captured(mp, T, E, k, groups):
    """The router of one workgroup and its gradient in a graph: every replay equals the eager call on new inputs, with
    eager work between the replays."""
    layer, other = (mp.Layer(mp.make_config(T, E, k, 1, 1, 8, 0), cooc=False) for _ in range(2))
    dev, g = layer.device, torch.Generator().manual_seed(E + T)
    gate, bias = mp.make_gate("sigmoid", *groups, True, 2.5), (0.1 * torch.randn(E, generator=g)).to(dev)
    x, gw = torch.randn(T, E, generator=g).to(dev), torch.randn(T, k, generator=g).to(dev)
    layer.gate(x, gate, bias=bias)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, w = layer.gate(x, gate, bias=bias)
        dx = layer.gate_grad(x, gate, gw)
    for _ in range(4):
        x.copy_(torch.randn(T, E, generator=g))
        for t in (w, dx, r.topk_idx, r.omega, r.expert_count):
            t.fill_(-3)
        graph.replay()
        torch.cuda.synchronize()
        r2, w2 = other.gate(x, gate, bias=bias)
        assert torch.equal(r.topk_idx, r2.topk_idx) and torch.equal(w, w2) and torch.equal(dx, other.gate_grad(x, gate, gw))
        assert torch.equal(r.omega, r2.omega) and torch.equal(r.expert_count, r2.expert_count)
    assert layer.status() == 0 and other.status() == 0
    layer.close()
    other.close()


def test_the_most_tokens(mp):
    """Just below 2^22 tokens, the most a layer takes: router, gradient, weighted sum and its gradient, sampled."""
    T, E, k, H = (1 << 22) - 2, 8, 2, 8
    layer = mp.Layer(mp.make_config(T, E, k, 1, 1, H, 0), cooc=False)
    dev = layer.device
    g = torch.Generator(device=dev).manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)
    x, gate, gw = rnd(T, E), mp.make_gate("softmax", 4, 2, 1, True, 1.0), rnd(T, k)
    r, w = layer.gate(x, gate)
    dx = layer.gate_grad(x, gate, gw)
    pos = torch.randperm(T * k, generator=g, device=dev).int()
    rows, grad = rnd(T * k, H).bfloat16(), rnd(T, H).bfloat16()
    out = layer.combine_weighted(rows, w, slot_pos=pos)
    drows, dw = layer.combine_grad(rows, grad, w, slot_pos=pos)
    assert layer.status() == 0
    assert torch.equal(r.expert_count, torch.bincount(r.topk_idx.flatten(), minlength=E).int())
    at = torch.cat([torch.arange(300), torch.arange(T - 300, T), torch.randint(0, T, (300,), generator=torch.Generator().manual_seed(1))])
    xs, ws, gs = x[at.to(dev)].cpu(), w[at.to(dev)].cpu().double(), gw[at.to(dev)].cpu().double()
    idx = refs.select(xs.double(), None, "softmax", k, 4, 2, 1)
    assert torch.equal(r.topk_idx[at.to(dev)].cpu().long(), idx)
    share = (E / 8 + 2 * k + 432) * 2.0 ** -24
    want = refs.gate_weights(xs.double(), idx, "softmax", True, 1.0)
    assert ((ws - want).abs() <= share * want).all()
    x64 = xs.double().requires_grad_()
    want, = torch.autograd.grad(refs.gate_weights(x64, idx, "softmax", True, 1.0), x64, gs)
    # what is added, s_e (ds_e + sum s ds): each s ds is at most (|g| + sum |g| s / S) s / S, together 2 sum |g|, and so
    # is s_e ds_e: 4 sum |g| at most
    assert ((dx[at.to(dev)].cpu().double() - want).abs() <= share * 4 * gs.abs().sum(-1, keepdim=True)).all()
    p = pos.view(T, k)[at.to(dev)].long()
    xr, gr = rows[p].cpu().double(), grad[at.to(dev)].cpu().double()
    want = (ws[..., None] * xr).sum(1)
    assert ((out[at.to(dev)].cpu().double() - want).abs()
            <= 2.0 ** -8 * want.abs() + 2 * k * 2.0 ** -24 * (ws[..., None] * xr).abs().sum(1)).all()
    want = ws[..., None] * gr[:, None]
    assert ((drows[p].cpu().double() - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs()).all()
    want = (gr[:, None] * xr).sum(-1)
    assert ((dw[at.to(dev)].cpu().double() - want).abs() <= 2 * H * 2.0 ** -24 * (gr[:, None] * xr).abs().sum(-1)).all()
    layer.close()
