"""moex_gate and moex_gate_grad against their definitions in 64 bits.

Indices, counts and matrices have to be equal.  A weight goes through the
exponentials of a row, their sum, a division and the sum of the k scores, in
fp32: with range = max |x - max| of the row (the argument of an exponential is
rounded by 2^-24 of itself, and so is its logarithm's neighbour in expf), it is
off by at most (E / 8 + 2 k + 2 range + 32) 2^-24 of itself; a gradient by the
same share of the magnitudes that are added in it.
"""
from __future__ import annotations

import numpy as np
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


def unit(x, k):
    top = x.amax(-1)
    rng = (x.abs().amax() if not torch.isfinite(top).all() else (top[:, None] - x).clamp(max=200).amax()).item()
    return (x.shape[1] / 8 + 2 * k + 2 * min(rng, 200) + 32) * 2.0 ** -24


def run(mp, x, bias, k, R, kind, groups=(1, 1, 1), renorm=True, scale=1.0, trans=None):
    T, E = x.shape
    layer = mp.Layer(mp.make_config(T, E, k, R, 1, 8, 0), cooc=True, trans=trans is not None)
    dev = layer.device
    gate = mp.make_gate(kind, *groups, renorm, scale)
    for t in (layer.route_out.topk_idx, layer.route_out.expert_count, layer.route_out.omega):
        t.fill_(-7)
    r, w = layer.gate(x.to(dev), gate, bias=None if bias is None else bias.to(dev),
                      prev_topk=None if trans is None else trans.to(dev))
    torch.cuda.synchronize()
    return layer, gate, r, w


def check(mp, x, bias, k, R, kind, groups=(1, 1, 1), renorm=True, scale=1.0):
    layer, gate, r, w = run(mp, x, bias, k, R, kind, groups, renorm, scale)
    assert layer.status() == 0
    x64 = x.double()
    idx = refs.select(x64, None if bias is None else bias.double(), kind, k, *groups)
    got = r.topk_idx.cpu().long()
    assert torch.equal(got, idx), "%d of %d tokens differ" % (int((got != idx).any(1).sum()), len(x))
    assert torch.equal(r.topk_val.cpu().view(torch.int32), x.gather(1, idx).view(torch.int32))
    want = refs.gate_weights(x64, idx, kind, renorm, scale)
    assert ((w.cpu().double() - want).abs() <= unit(x64[torch.isfinite(x64).all(1)] if not torch.isfinite(x64).all()
                                                    and torch.isfinite(x64).all(1).any() else x64, k) * want.abs()
            + 1e-37).all()
    T, E = x.shape
    hot = torch.nn.functional.one_hot(idx, E).sum(1)
    omega = hot.view(R, T // R, E).sum(1).int()
    assert torch.equal(r.omega.cpu(), omega) and torch.equal(r.expert_count.cpu(), omega.sum(0).int())
    pairs = (hot.double().t() @ hot.double()).int()
    pairs.fill_diagonal_(0)
    assert torch.equal(r.cooc.cpu(), pairs)
    layer.close()


def logits(seed, T, E, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return spread * torch.randn(T, E, generator=g), 0.1 * torch.randn(E, generator=g)


SHAPES = [(1, 8, 1, 1), (1, 8, 8, 1), (7, 100, 8, 1), (64, 256, 8, 8), (130, 128, 8, 2), (200, 64, 16, 4), (96, 896, 16, 8),
          (34, 2048, 32, 2), (70, 30, 3, 10), (128, 6, 2, 2), (65, 17, 5, 1), (64, 2048, 8, 64), (257, 512, 1, 1)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_router_without_groups(mp, shape, kind, biased):
    T, E, k, R = shape
    print("gate T=%d E=%d k=%d R=%d %s bias=%s" % (*shape, kind, biased), flush=True)
    x, b = logits(T + E + k, T, E)
    check(mp, x, b if biased else None, k, R, kind, renorm=T % 2 == 0, scale=2.5 if E > 100 else 1.0)


@pytest.mark.parametrize("shape", [(64, 256, 8, 8, 8, 4, 2), (40, 256, 8, 1, 8, 1, 2), (50, 160, 6, 2, 8, 3, 1), (33, 64, 4, 1, 64, 8, 1),
                                   (20, 2048, 16, 4, 16, 5, 2), (35, 96, 8, 1, 3, 2, 2), (30, 60, 2, 1, 20, 2, 2),
                                   (64, 128, 32, 64, 4, 4, 2), (48, 512, 8, 1, 2, 1, 2), (9, 896, 16, 1, 8, 8, 1)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_router_with_groups(mp, shape, kind, biased):
    T, E, k, R = shape[:4]
    print("gate groups %s %s bias=%s" % (shape, kind, biased), flush=True)
    x, b = logits(sum(shape), T, E)
    check(mp, x, b if biased else None, k, R, kind, shape[4:], True, 2.5)


@pytest.mark.parametrize("shape", [(4104, 256, 8, 8, 8, 4, 2), (4097, 128, 8, 1, 1, 1, 1), (4100, 512, 8, 2, 1, 1, 1),
                                   (4104, 896, 16, 8, 8, 4, 1), (4099, 8, 2, 1, 1, 1, 1), (4098, 160, 6, 2, 8, 3, 1),
                                   (4101, 100, 4, 1, 1, 1, 1), (4104, 2048, 8, 8, 16, 5, 2), (4096, 384, 8, 1, 1, 1, 1)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_many_tokens(mp, shape, kind, biased):
    """Above 4096 tokens a token has fewer lanes."""
    T, E, k, R = shape[:4]
    print("gate many tokens %s %s bias=%s" % (shape, kind, biased), flush=True)
    x, b = logits(sum(shape), T, E)
    check(mp, x, b if biased else None, k, R, kind, shape[4:], True, 2.5)


@pytest.mark.parametrize("T,E,k,R", [(1, 8, 2, 1), (1, 256, 8, 1), (8, 256, 8, 1), (8, 256, 8, 4), (9, 256, 8, 1), (16, 64, 8, 4),
                                     (17, 64, 8, 1), (32, 16, 2, 8), (33, 16, 2, 3), (8, 2048, 8, 8), (4, 896, 16, 2), (6, 30, 3, 6), (32, 256, 8, 8), (31, 256, 8, 1), (16, 896, 16, 1),
                                     (17, 896, 16, 1), (16, 2048, 8, 2), (24, 128, 6, 2), (32, 64, 20, 1)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_few_tokens_without_masks(mp, T, E, k, R, kind):
    """Without co-selection or transition counts, one workgroup's tokens take one launch: the same outputs as with
    them, into buffers that held other values, and the planner goes on from them."""
    E = E if E % R == 0 else E + R - E % R
    print("gate few tokens T=%d E=%d k=%d R=%d" % (T, E, k, R), flush=True)
    x, b = logits(T * E, T, E)
    check(mp, x, b, k, R, kind)
    layer, gate, full, w = run(mp, x, b, k, R, kind)
    lean = mp.Layer(mp.make_config(T, E, k, R, 1, 8, 0), cooc=False)
    for t in (lean.route_out.topk_idx, lean.route_out.expert_count, lean.route_out.omega):
        t.fill_(-7)
    for _ in range(2):
        r, w2 = lean.gate(x.to(lean.device), gate, bias=b.to(lean.device))
        assert torch.equal(r.topk_idx, full.topk_idx) and torch.equal(w2, w) and torch.equal(r.topk_val, full.topk_val)
        assert torch.equal(r.omega, full.omega) and torch.equal(r.expert_count, full.expert_count)
    p, q = layer.plan(), lean.plan()
    torch.cuda.synchronize()
    assert torch.equal(p.inst_expert, q.inst_expert) and torch.equal(p.slot_inst, q.slot_inst)
    assert layer.status() == 0 and lean.status() == 0
    layer.close()
    lean.close()


@pytest.mark.parametrize("T,E,k,R,groups", [(16, 2000, 8, 2, (10, 4, 2)), (14, 1530, 4, 2, (5, 2, 2)), (16, 1020, 8, 1, (60, 9, 2)),
                                            (32, 250, 8, 2, (10, 4, 2)), (32, 96, 4, 4, (32, 8, 2)), (5, 60, 2, 1, (20, 2, 1))])
def test_few_tokens_with_groups_without_masks(mp, T, E, k, R, groups):
    print("gate few tokens groups T=%d E=%d %s" % (T, E, groups), flush=True)
    x, b = logits(T * E, T, E)
    layer, gate, full, w = run(mp, x, b, k, R, "sigmoid", groups)
    idx = refs.select(x.double(), b.double(), "sigmoid", k, *groups)
    lean = mp.Layer(mp.make_config(T, E, k, R, 1, 8, 0), cooc=False)
    r, w2 = lean.gate(x.to(lean.device), gate, bias=b.to(lean.device))
    assert torch.equal(r.topk_idx.cpu().long(), idx) and torch.equal(full.topk_idx.cpu().long(), idx)
    assert torch.equal(w2, w) and torch.equal(r.omega, full.omega) and torch.equal(r.expert_count, full.expert_count)
    assert layer.status() == 0 and lean.status() == 0
    layer.close()
    lean.close()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_ties_of_many_tokens(mp, kind):
    T, E, k = 4110, 256, 8
    g = torch.Generator().manual_seed(5)
    coarse = (torch.randn(T, E, generator=g) * 4).round() / 4
    coarse[100:110] = 0.0
    coarse[200:210, ::3] = -torch.inf
    coarse[300:310] = -torch.inf
    near = torch.full((T, E), 1.5) + torch.randint(0, 50, (T, E), generator=g) * 2.0 ** -23
    bias = torch.randint(0, 3, (E,), generator=g) * 2.0 ** -24
    for groups in ((1, 1, 1), (8, 4, 2)):
        check(mp, coarse, None, k, 1, kind, groups)
        check(mp, coarse, torch.zeros(E), k, 1, kind, groups)
        check(mp, near, bias, k, 1, kind, groups)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_ties_and_near_ties(mp, kind):
    """Logits on a coarse grid (equal choices by the dozen, with and without a bias of zeros) and logits a few units
    in the last place apart, where 32-bit choices do not tell."""
    T, E, k = 96, 256, 8
    g = torch.Generator().manual_seed(3)
    coarse = (torch.randn(T, E, generator=g) * 4).round() / 4
    zero = torch.zeros(E)
    for groups in ((1, 1, 1), (8, 4, 2), (8, 4, 1)):
        check(mp, coarse, None, k, 1, kind, groups)
        check(mp, coarse, zero, k, 1, kind, groups)
        check(mp, torch.zeros(T, E), zero, k, 1, kind, groups)
    near = torch.full((T, E), 1.5) + torch.randint(0, 50, (T, E), generator=g) * 2.0 ** -23
    bias = torch.randint(0, 3, (E,), generator=g) * 2.0 ** -24
    for groups in ((1, 1, 1), (8, 3, 2)):
        check(mp, near, None, k, 1, kind, groups)
        check(mp, near, bias, k, 1, kind, groups)
        check(mp, near + torch.randn(T, E, generator=g), 1e-7 * torch.randn(E, generator=g), k, 1, kind, groups)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_masked_and_extreme_logits(mp, kind, biased):
    T, E, k = 40, 64, 4
    x, b = logits(11, T, E)
    x[0] = -torch.inf                       # a row whose mask leaves nothing
    x[1, 5:] = -torch.inf
    x[2, 3:] = -torch.inf                   # fewer experts than k
    x[3] = torch.finfo(torch.float32).min   # a mask of the lowest value
    x[4, ::2] = torch.finfo(torch.float32).min
    x[5] = torch.linspace(-300, 300, E)
    x[6] = torch.linspace(1e-30, 64e-30, E)
    x[7, :8] = -0.0
    x[7, 8:] = 0.0
    if kind == "sigmoid":
        x[8, :3] = torch.inf
    for groups in ((1, 1, 1), (8, 4, 2)):
        check(mp, x, b if biased else None, k, 1, kind, groups, scale=1.5)
    if biased:
        b[torch.arange(0, 40)] = -torch.inf  # experts kept from being chosen
        check(mp, x, b, k, 1, kind)


def test_wrong_inputs_set_the_status(mp):
    T, E, k = 24, 32, 4
    x, b = logits(2, T, E)
    bad_x, bad_b, inf_x = x.clone(), b.clone(), x.clone()
    bad_x[3, 7], bad_b[9], inf_x[5, 1] = torch.nan, torch.nan, torch.inf
    for xs, bias, kind, want in ((bad_x, None, "softmax", True), (bad_x, b, "sigmoid", True), (x, bad_b, "sigmoid", True),
                                 (x, torch.full((E,), torch.inf), "softmax", True), (inf_x, None, "softmax", True),
                                 (inf_x, None, "sigmoid", False)):
        layer, gate, r, w = run(mp, xs, bias, k, 1, kind)
        assert (layer.status() == mp.MOE_STATUS_NAN_LOGIT) == want
        idx = r.topk_idx.cpu()
        assert all(len(set(row.tolist())) == k and 0 <= min(row) and max(row) < E for row in idx)
        good = [t for t in range(T) if t not in (3, 5)]
        if bias is None:
            assert torch.equal(idx[good].long(), refs.select(x.double(), None, kind, k, 1, 1, 1)[good])
        layer.close()


def test_transitions_and_refusals(mp):
    T, E, k = 64, 32, 4
    x, b = logits(5, T, E)
    prev = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k] for t in range(T)]).int()
    layer, gate, r, w = run(mp, x, b, k, 2, "sigmoid", trans=prev)
    assert layer.status() == 0
    hot = lambda i: torch.nn.functional.one_hot(i.long(), E).sum(1).double()
    assert torch.equal(r.trans.cpu(), (hot(prev).t() @ hot(r.topk_idx.cpu())).int())
    dev = layer.device
    xd = x.to(dev)
    for bad in (dict(n_group=3), dict(n_group=8, topk_group=0), dict(n_group=8, topk_group=9), dict(n_group=32, topk_group=3),
                dict(n_group=4, topk_group=2, group_top=3), dict(n_group=32, topk_group=8, group_top=2), dict(n_group=0),
                dict(scale=float("nan"))):
        with pytest.raises(mp.MoePlanError) as e:
            layer.gate(xd, mp.make_gate("sigmoid", **bad))
        assert e.value.code == mp.MOE_ERR_INVALID_ARG, bad
        with pytest.raises(mp.MoePlanError):
            layer.gate_grad(xd, mp.make_gate("sigmoid", **bad), torch.zeros(T, k, device=dev))
    odd = mp.make_gate("sigmoid")
    odd.score = 2
    with pytest.raises(mp.MoePlanError):
        layer.gate(xd, odd)
    with pytest.raises(ValueError):
        layer.gate(xd[:, :16].contiguous(), mp.make_gate())
    with pytest.raises(TypeError):
        layer.gate(xd.double(), mp.make_gate())
    with pytest.raises(ValueError):
        layer.gate(xd, mp.make_gate(), bias=torch.zeros(E + 1, device=dev))
    layer.close()
    wide = mp.Layer(mp.make_config(8, 256, 2, 1, 1, 8, 0))
    with pytest.raises(mp.MoePlanError) as e:
        wide.gate(torch.zeros(8, 256, device=dev), mp.make_gate("softmax", 128, 64))
    assert e.value.code == mp.MOE_ERR_UNSUPPORTED
    wide.close()


def test_no_tokens(mp):
    layer = mp.Layer(mp.make_config(0, 32, 4, 4, 2, 8, 0))
    layer.route_out.expert_count.fill_(-7)
    layer.route_out.omega.fill_(-7)
    r, w = layer.gate(torch.empty(0, 32, device=layer.device), mp.make_gate("sigmoid"))
    g = layer.gate_grad(torch.empty(0, 32, device=layer.device), mp.make_gate("sigmoid"),
                        torch.empty(0, 4, device=layer.device))
    torch.cuda.synchronize()
    assert layer.status() == 0 and w.shape == (0, 4) and g.shape == (0, 32)
    assert int(r.expert_count.abs().sum()) == 0 and int(r.omega.abs().sum()) == 0
    layer.close()


def test_unaligned_logits(mp):
    """Logits that start 4 bytes past a 16-byte boundary, as a view into a larger buffer does."""
    T, E, k = 64, 128, 8
    x, b = logits(21, T, E)
    layer = mp.Layer(mp.make_config(T, E, k, 1, 1, 8, 0))
    buf = torch.empty(T * E + 1, device=layer.device)
    xd = buf[1:].view(T, E).copy_(x)
    gate = mp.make_gate("sigmoid", 8, 4, 2, True, 2.5)
    r, w = layer.gate(xd, gate, bias=b.to(layer.device))
    gw = torch.randn(T, k, generator=torch.Generator().manual_seed(1)).to(layer.device)
    g = layer.gate_grad(xd, gate, gw)
    idx, wv = r.topk_idx.clone(), w.clone()
    r, w = layer.gate(x.to(layer.device), gate, bias=b.to(layer.device))
    assert torch.equal(r.topk_idx, idx) and torch.equal(w, wv)
    assert torch.equal(g, layer.gate_grad(x.to(layer.device), gate, gw))
    assert layer.status() == 0
    layer.close()


def grad_bound(x, idx, gw, kind, renorm, scale):
    s = refs.scores(x, kind)
    sj = s.gather(1, idx)
    if renorm:
        S = sj.sum(-1, keepdim=True) + 1e-20
        ds = scale / S * (gw.abs() + (gw.abs() * sj).sum(-1, keepdim=True) / S)
    else:
        ds = scale * gw.abs()
    full = torch.zeros_like(s).scatter(1, idx, ds)
    if kind == "softmax":
        return s * (full + (sj * ds).sum(-1, keepdim=True))
    return full * s


@pytest.mark.parametrize("shape", [(1, 8, 2), (37, 100, 8), (64, 256, 8), (130, 128, 6), (50, 896, 16), (22, 2048, 32),
                                   (66, 30, 3), (5, 6, 6), (200, 17, 1)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient(mp, shape, kind, renorm):
    T, E, k = shape
    print("gate grad T=%d E=%d k=%d %s renorm=%s" % (T, E, k, kind, renorm), flush=True)
    x, b = logits(T * E + k, T, E, 2.0)
    if T > 30:
        x[1, : E // 2] = -torch.inf
        x[2] = -torch.inf
        x[3] = torch.finfo(torch.float32).min
    layer, gate, r, w = run(mp, x, b, k, 2 if E > 1024 else 1, kind, renorm=renorm, scale=2.5)
    gw = torch.randn(T, k, generator=torch.Generator().manual_seed(9))
    got = layer.gate_grad(x.to(layer.device), gate, gw.to(layer.device)).cpu().double()
    assert layer.status() == 0
    idx = r.topk_idx.cpu().long()
    x64 = x.double().requires_grad_()
    # through the definition by automatic differentiation, rows of nothing but -infinity apart
    live = torch.isfinite(x).any(1)
    wref = refs.gate_weights(torch.where(torch.isfinite(x64), x64, -1e4), idx, kind, renorm, 2.5)
    want, = torch.autograd.grad(wref[live], x64, gw.double()[live])
    assert (got[~live] == 0).all()
    xf = x.double()
    bound = unit(xf[torch.isfinite(xf).all(1)], k) * grad_bound(torch.where(torch.isfinite(xf), xf, -1e4), idx, gw.double(),
                                                                kind, renorm, 2.5)
    err = (got - want.nan_to_num()).abs()
    assert (err[live] <= bound[live] + 1e-30).all(), float((err - bound)[live].max())
    # and against differences of the definition, on some logits of the first token
    for e in range(0, E, max(1, E // 8)):
        h = 1e-5
        up, down = x.double(), x.double()
        up[0, e] += h
        down[0, e] -= h
        f = [(refs.gate_weights(z[:1], idx[:1], kind, renorm, 2.5) * gw.double()[:1]).sum() for z in (up, down)]
        d = (f[0] - f[1]) / (2 * h)
        # h^2 / 6 times a third derivative of a few, and 2^-53 / h of rounding
        assert abs(d - got[0, e]) <= bound[0, e] + 1e-8 * (1 + gw.abs().sum()), e
    layer.close()


def test_gradient_of_bad_indices(mp):
    T, E, k = 16, 32, 4
    x, _ = logits(1, T, E)
    layer = mp.Layer(mp.make_config(T, E, k, 1, 1, 8, 0))
    dev = layer.device
    gate = mp.make_gate("softmax")
    r, w = layer.gate(x.to(dev), gate)
    gw = torch.ones(T, k, device=dev)
    clean = layer.gate_grad(x.to(dev), gate, gw)
    assert layer.status() == 0
    for value in (-1, E, 2 ** 31 - 1, -2 ** 31, None):
        idx = r.topk_idx.clone()
        idx[5, 2] = idx[5, 1] if value is None else value
        got = layer.gate_grad(x.to(dev), gate, gw, topk_idx=idx)
        assert layer.status() == mp.MOE_STATUS_BAD_TOPK
        rest = [t for t in range(T) if t != 5]
        assert torch.equal(got[rest], clean[rest])
    layer.close()
