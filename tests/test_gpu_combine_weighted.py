"""moex_combine and moex_combine_grad against 64 bits.

Forward: |gpu - y| <= 2^-8 |y| + (k + 2) 2^-24 sum_j |w_j x_j| (1 + 2^-8): k fp32 FMAs, one rounding to bf16.
Row gradient: one product and one rounding, 2^-8 |w g| (1 + 2^-23).
Weight gradient: H fp32 FMAs per thread chain and a tree, (H / 64 + 16) 2^-24 sum_c |g_c x_c| (a thread adds at most
H / 256 * 8 / 8 + ... <= H / 64 products, then six levels of a wave and three of the workgroup)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import load_balance_planning_amd as m
    m.lib()
    return m


def data(seed, T, k, H):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    return (n(T * k, H).to(BF), n(T, H).to(BF), n(T, k), torch.randperm(T * k, generator=g).int())


def layer_of(mp, T, k, H):
    return mp.Layer(mp.make_config(T, max(8, k), k, 1, 1, H, 0), cooc=False)


@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (3, 2, 13), (64, 8, 512), (40, 6, 264), (17, 16, 7168), (9, 32, 24),
                                   (12, 8, 2048), (12, 8, 2056), (5, 4, 8200), (30, 5, 1001), (7, 3, 16400),
                                   # around 512 tokens, where a token's work is no longer split
                                   (511, 2, 2056), (512, 3, 2056), (700, 5, 2048), (1000, 6, 264), (600, 2, 8200),
                                   (513, 9, 1001), (520, 7, 4104),
                                   # rows of less than a vector, of one, and whose last overlaps the one before
                                   (5, 3, 7), (4, 2, 8), (6, 4, 9), (3, 8, 15), (40, 8, 2049), (600, 3, 7167), (30, 4, 2047),
                                   (700, 2, 5), (515, 2, 10),
                                   # several tokens to a workgroup
                                   (2000, 8, 512), (777, 4, 37), (512, 5, 8), (1500, 3, 505), (640, 32, 148), (2049, 1, 16),
                                   (900, 9, 513)])
def test_weighted_sum_and_gradients(mp, T, k, H):
    print("combine weighted T=%d k=%d H=%d" % (T, k, H), flush=True)
    rows, g, w, pos = data(T + k + H, T, k, H)
    layer = layer_of(mp, T, k, H)
    dev = layer.device
    d = lambda t: t.to(dev)
    out = layer.combine_weighted(d(rows), d(w), slot_pos=d(pos))
    plain = layer.combine_weighted(d(rows), slot_pos=d(pos))
    gr, gw = layer.combine_grad(d(rows), d(g), d(w), slot_pos=d(pos))
    torch.cuda.synchronize()
    assert layer.status() == 0
    r64 = rows.double().requires_grad_()
    w64 = w.double().requires_grad_()
    picked = r64[pos.long()].view(T, k, H)
    y = (picked * w64[..., None]).sum(1)
    want_r, want_w = torch.autograd.grad(y, (r64, w64), g.double())
    mag = (picked.detach().abs() * w.double().abs()[..., None]).sum(1)
    grow = 1 + 2.0 ** -8
    assert ((out.cpu().double() - y.detach()).abs() <= 2.0 ** -8 * y.detach().abs() + grow * (k + 2) * 2.0 ** -24 * mag).all()
    s = picked.detach().sum(1)
    assert ((plain.cpu().double() - s).abs() <= 2.0 ** -8 * s.abs()
            + grow * (k + 2) * 2.0 ** -24 * picked.detach().abs().sum(1)).all()
    assert ((gr.cpu().double() - want_r).abs() <= 2.0 ** -8 * (1 + 2.0 ** -23) * want_r.abs()).all()
    dots = (picked.detach().abs() * g.double().abs()[:, None]).sum(-1)
    assert ((gw.cpu().double() - want_w).abs() <= (H / 64 + 16) * 2.0 ** -24 * dots).all()
    # and against differences (the sum is linear in each weight)
    h = 0.5
    for t, j in ((0, 0), (T - 1, k - 1)):
        up, down = w.double(), w.double()
        up[t, j] += h
        down[t, j] -= h
        f = [((picked.detach() * v[..., None]).sum(1) * g.double()).sum() for v in (up, down)]
        assert abs((f[0] - f[1]) / (2 * h) - gw.cpu().double()[t, j]) <= (H / 64 + 16) * 2.0 ** -24 * dots[t, j] + 1e-9
    layer.close()


@pytest.mark.parametrize("T,k,H", [(20000, 8, 7168), (33000, 6, 6003)])
def test_large_layers_sampled(mp, T, k, H):
    """More than 2^31 bytes of rows, where a thread takes four vectors of a row at a time; rows of odd width too."""
    print("combine large T=%d k=%d H=%d" % (T, k, H), flush=True)
    layer = layer_of(mp, T, k, H)
    dev = layer.device
    g0 = torch.Generator(device=dev).manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g0, device=dev)
    rows, g, w = torch.empty(T * k, H, dtype=BF, device=dev), n(T, H).to(BF), n(T, k)
    for part in rows.split(20000):
        part.copy_(n(*part.shape))
    pos = torch.randperm(T * k, generator=g0, device=dev).int()
    out = layer.combine_weighted(rows, w, slot_pos=pos)
    gr, gw = layer.combine_grad(rows, g, w, slot_pos=pos)
    assert layer.status() == 0
    at = torch.cat([torch.tensor([0, T - 1]), torch.randint(0, T, (60,), generator=torch.Generator().manual_seed(1))])
    p = pos.view(T, k)[at.to(dev)].long()
    x, wt, gt = rows[p].cpu().double(), w[at.to(dev)].cpu().double(), g[at.to(dev)].cpu().double()
    y, mag = (x * wt[..., None]).sum(1), (x.abs() * wt.abs()[..., None]).sum(1)
    grow = 1 + 2.0 ** -8
    assert ((out[at.to(dev)].cpu().double() - y).abs() <= 2.0 ** -8 * y.abs() + grow * (k + 2) * 2.0 ** -24 * mag).all()
    want = wt[..., None] * gt[:, None]
    assert ((gr[p].cpu().double() - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -23) * want.abs()).all()
    dots = (x.abs() * gt.abs()[:, None]).sum(-1)
    assert ((gw[at.to(dev)].cpu().double() - (x * gt[:, None]).sum(-1)).abs() <= (H / 64 + 16) * 2.0 ** -24 * dots).all()
    layer.close()


def test_weights_that_are_no_softmax(mp):
    T, k, H = 24, 4, 64
    rows, g, w, pos = data(1, T, k, H)
    layer = layer_of(mp, T, k, H)
    d = lambda t: t.to(layer.device)
    w[0] = 0
    w[1, 2] = torch.inf
    w[2, 0] = torch.nan
    out = layer.combine_weighted(d(rows), d(w), slot_pos=d(pos)).cpu()
    gr, gw = layer.combine_grad(d(rows), d(g), d(w), slot_pos=d(pos))
    assert layer.status() == 0
    assert (out[0] == 0).all() and not torch.isfinite(out[1]).any() and torch.isnan(out[2]).all()
    assert torch.isfinite(out[3:]).all() and torch.isfinite(gw).all()
    assert (gr.cpu()[pos.long().view(T, k)[0]] == 0).all()
    layer.close()


@pytest.mark.parametrize("T,H", [(20, 13), (600, 13), (20, 2051)])
def test_an_infinity_counts_once(mp, T, H):
    """The last vectors of a row of odd width overlap: an infinity in both, with a gradient of zero or not."""
    k = 2
    rows, g, w, pos = data(3, T, k, H)
    layer = layer_of(mp, T, k, H)
    d = lambda t: t.to(layer.device)
    at = H - H % 8 - 1                      # in the last vector and the one before
    rows[pos[0], at] = torch.inf
    rows[pos[2 * k], 0] = -torch.inf
    g[0, at] = 2.0
    g[2, 0] = 0.5
    out = layer.combine_weighted(d(rows), d(w), slot_pos=d(pos)).cpu()
    gr, gw = layer.combine_grad(d(rows), d(g), d(w), slot_pos=d(pos))
    assert layer.status() == 0
    gw = gw.cpu()
    assert gw[0, 0] == torch.inf and gw[2, 0] == -torch.inf and torch.isfinite(gw.flatten()[[1, 2, 3, 5]]).all()
    bad = ~torch.isfinite(out)
    assert bad[0, at] and bad[2, 0] and int(bad.sum()) == 2 and torch.isfinite(gr).all()
    layer.close()


@pytest.mark.parametrize("H", [64, 13])
def test_positions_outside_and_refusals(mp, H):
    T, k = 16, 4
    rows, g, w, pos = data(2, T, k, H)
    layer = layer_of(mp, T, k, H)
    dev = layer.device
    d = lambda t: t.to(dev)
    for bad in (-1, T * k, 2 ** 31 - 1, -2 ** 31):
        p = pos.clone()
        p[9] = bad  # token 2, slot 1
        out = layer.combine_weighted(d(rows), d(w), slot_pos=d(p)).cpu().double()
        assert layer.status() == mp.MOE_STATUS_PLAN_CHECK
        gr, gw = layer.combine_grad(d(rows), d(g), d(w), slot_pos=d(p))
        assert layer.status() == mp.MOE_STATUS_PLAN_CHECK
        assert gw[2, 1] == 0
        keep = w.double().clone()
        keep[2, 1] = 0
        y = (rows.double()[pos.long()].view(T, k, H) * keep[..., None]).sum(1)
        mag = (rows.double()[pos.long()].view(T, k, H) * keep[..., None]).abs().sum(1)
        assert ((out - y).abs() <= 2.0 ** -8 * y.abs() + (k + 2) * 2.0 ** -23 * mag).all()
    with pytest.raises(ValueError):
        layer.combine_weighted(d(rows), d(w)[:, :2].contiguous(), slot_pos=d(pos))
    with pytest.raises(ValueError):
        layer.combine_grad(d(rows), d(g)[1:], d(w), slot_pos=d(pos))
    with pytest.raises(TypeError):
        layer.combine_weighted(d(rows).float(), d(w), slot_pos=d(pos))
    import ctypes
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    R, G, W, P = d(rows), d(g), d(w), d(pos)
    full = [layer.handle, p(W), p(P), p(R), p(G), p(R), p(W), None]
    for at in range(1, 7):
        a = list(full)
        a[at] = None
        assert mp.lib().moex_combine_grad(*a) == mp.MOE_ERR_INVALID_ARG
    for at in (2, 3, 4):
        a = [layer.handle, None, p(P), p(R), p(G), None]
        a[at] = None
        assert mp.lib().moex_combine(*a) == mp.MOE_ERR_INVALID_ARG
    layer.close()


@pytest.mark.parametrize("H", [24, 509])
def test_positions_outside_among_many_tokens(mp, H):
    T, k = 700, 5
    rows, g, w, pos = data(4, T, k, H)
    layer = layer_of(mp, T, k, H)
    d = lambda t: t.to(layer.device)
    p = pos.clone()
    for slot, bad in ((3 * k + 1, -1), (699 * k + 4, T * k), (300 * k, 2 ** 31 - 1)):
        p[slot] = bad
    off = ~((p >= 0) & (p < T * k)).view(T, k)
    wz = w.masked_fill(off, 0.0)
    out = layer.combine_weighted(d(rows), d(w), slot_pos=d(p))
    assert layer.status() == mp.MOE_STATUS_PLAN_CHECK
    want = layer.combine_weighted(d(rows), d(wz), slot_pos=d(pos))
    assert torch.equal(out, want) and layer.status() == 0
    gr, gw = layer.combine_grad(d(rows), d(g), d(w), slot_pos=d(p))
    assert layer.status() == mp.MOE_STATUS_PLAN_CHECK
    gr0, gw0 = layer.combine_grad(d(rows), d(g), d(w), slot_pos=d(pos))
    assert (gw.cpu()[off] == 0).all() and torch.equal(gw.cpu()[~off], gw0.cpu()[~off])
    ok = p.view(T, k)[~off].long()
    assert torch.equal(gr.cpu()[ok], gr0.cpu()[ok])
    layer.close()


def test_unaligned_and_no_tokens(mp):
    T, k, H = 10, 4, 64
    rows, g, w, pos = data(3, T, k, H)
    layer = layer_of(mp, T, k, H)
    dev = layer.device
    d = lambda t: t.to(dev)
    shift = lambda t: torch.empty(t.numel() + 1, dtype=BF, device=dev)[1:].view(t.shape).copy_(t)
    a = layer.combine_weighted(shift(rows), d(w), slot_pos=d(pos))
    b = layer.combine_weighted(d(rows), d(w), slot_pos=d(pos))
    assert torch.equal(a, b)
    a, aw = layer.combine_grad(shift(rows), shift(g), d(w), slot_pos=d(pos))
    b, bw = layer.combine_grad(d(rows), d(g), d(w), slot_pos=d(pos))
    assert torch.equal(a, b) and torch.allclose(aw, bw, rtol=1e-4, atol=1e-4)
    layer.close()
    empty = mp.Layer(mp.make_config(0, 8, 2, 1, 1, 16, 0))
    z = torch.empty(0, 16, dtype=BF, device=dev)
    assert empty.combine_weighted(z, slot_pos=torch.empty(0, dtype=torch.int32, device=dev)).shape == (0, 16)
    gr, gw = empty.combine_grad(z, z, torch.empty(0, 2, device=dev), slot_pos=torch.empty(0, dtype=torch.int32, device=dev))
    assert gr.shape == (0, 16) and gw.shape == (0, 2) and empty.status() == 0
    empty.close()
