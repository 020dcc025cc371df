"""Scale bytes that the quantizer does not write, products of very different size in one step of the matrix
instruction, two forward passes of a layer before their backward passes, and whose memory results on a stream are."""
from __future__ import annotations

import dataclasses

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


def one_instance_each(mp, layer, loads):
    cap, dev = int(layer.sizes.inst_cap), layer.device
    off = torch.zeros(cap + 1, dtype=torch.int32, device=dev)
    off[1:] = torch.tensor(loads).cumsum(0).to(dev)
    plan = mp.PlanBuffers(torch.tensor([cap], dtype=torch.int32, device=dev),
                          torch.arange(cap, dtype=torch.int32, device=dev), None, None, None, None, None, None)
    return dict(plan=plan, inst_offset=off)


def blocks(mp, q, s, cols, dev):
    """Blocks of given bytes."""
    return mp.Blocks(q.to(torch.uint8).to(dev).view(torch.float8_e4m3fn), s.to(torch.uint8).to(dev).view(torch.float8_e8m0fnu),
                     cols)


def e4m3_value(byte):
    return torch.tensor([byte], dtype=torch.uint8).view(torch.float8_e4m3fn).double().item()


@pytest.mark.parametrize("rows", [6, 40, 256])
@pytest.mark.parametrize("byte", [0x38, 0x7e, 0x01, 0xc4])   # 1, 448, the least subnormal 2^-9, -3
def test_any_scale_byte(mp, rows, byte):
    """Row r of x is one value under scale byte r * step: y is that value times 2^(byte - 127), rounded to bf16, and so
    is the weight gradient of that row alone, where the value in bf16 is finite; a marked block's are NaN.  Kernels for
    few rows and for tiles (a mean of more than 8 rows an expert)."""
    n, v = 16, e4m3_value(byte)
    layer = mp.Layer(mp.make_config(rows, 1, 1, 1, 1, 8, 0), cooc=False)
    dev = layer.device
    print("scale bytes rows=%d value=%g" % (rows, v), flush=True)
    kw = one_instance_each(mp, layer, [rows])
    s = torch.full((rows, 4), 127)
    s[:, 0] = torch.linspace(0, 255, rows).round().int()
    x = blocks(mp, torch.full((rows, 128), byte), s, 128, dev)
    w = layer.quantize_weights(torch.eye(n, 128).to(BF)[None].contiguous().to(dev))
    y = layer.matmul(x, w, **kw).cpu()
    want = (v * torch.exp2(s[:, 0].double() - 127)).float().to(BF)
    marked = s[:, 0] == 255
    # 2^-149 v and above is an fp32 value exactly; bf16's rounding is the only one
    assert torch.equal(y[~marked], want[~marked, None].expand(-1, n)) and torch.isnan(y[marked]).all()
    # as the rows' gradient: dy row r is (1, 0, 0, ..) in row r's instance
    for r in range(0, rows, max(1, rows // 12)):
        lone = s.clone()
        lone[:, 0] = 127
        lone[r, 0] = s[r, 0]
        dy = torch.zeros(rows, n, dtype=BF)
        dy[r, 0] = 1
        dw = layer.wgrad(layer.quantize(dy.to(dev)), blocks(mp, torch.full((rows, 128), byte), lone, 128, dev), **kw).cpu()[0]
        if marked[r] or torch.isinf(want[r]):
            assert not torch.isfinite(dw[0]).any()
        else:
            assert (dw[0] == want[r]).all() and (dw[1:] == 0).all(), (r, int(s[r, 0]))
        # and as the gradient's scale: x row r is ones
        one = torch.zeros(rows, 128)
        one[r] = 0x38
        dw = layer.wgrad(blocks(mp, torch.full((rows, 128), byte), s.where(torch.arange(rows)[:, None] == r, 127), n, dev),
                         blocks(mp, one, torch.full((rows, 4), 127), 128, dev), **kw).cpu()[0]
        if marked[r] or torch.isinf(want[r]):
            assert not torch.isfinite(dw).any()
        else:
            assert (dw == want[r]).all(), (r, int(s[r, 0]))
    assert layer.status() == 0
    layer.close()


@pytest.mark.parametrize("bytes_", [(0, 0, 7, 254), (1, 254, 0, 130)])
def test_any_scale_byte_of_matrices(mp, bytes_):
    """The matrices' scales, one per 128 x 128, in both layouts and both kernels."""
    n, k = 200, 256
    for rows in (4, 64):
        layer = mp.Layer(mp.make_config(rows, 1, 1, 1, 1, 8, 0), cooc=False)
        dev = layer.device
        kw = one_instance_each(mp, layer, [rows])
        ws = torch.full((1, 2, 4), 127)
        ws[0, :, :2] = torch.tensor(bytes_).view(2, 2)
        w = blocks(mp, torch.full((1, n, k), 0x38), ws, k, dev)
        for half in range(2):
            q = torch.zeros(rows, k)
            q[:, 128 * half] = 0x38      # one value of 1
            y = layer.matmul(blocks(mp, q, torch.full((rows, 4), 127), k, dev), w, **kw).cpu()
            for b in range(2):
                want = torch.tensor(2.0, dtype=torch.float64) ** (bytes_[2 * b + half] - 127)
                got = y[:, 128 * b: min(n, 128 * (b + 1))].double()
                assert (got == want).all(), (rows, half, b)
        assert layer.status() == 0
        layer.close()


@pytest.mark.parametrize("rows", [8, 64])
@pytest.mark.parametrize("seed", range(3))
def test_small_products_beside_large_ones(mp, rows, seed):
    """Pairs of large products that cancel exactly, and small ones whose sum is all that is left: what the matrix
    instruction drops when it aligns a step's products to the largest stays within the bound of refs.product, and bf16's
    rounding of the small result does not hide it."""
    g = torch.Generator().manual_seed(seed)
    n, k = 64, 128
    e4 = lambda *s: torch.randn(*s, generator=g).clamp(-3, 3).to(torch.float8_e4m3fn).double()
    layer = mp.Layer(mp.make_config(rows, 1, 1, 1, 1, 8, 0), cooc=False)
    dev = layer.device
    kw = one_instance_each(mp, layer, [rows])
    worst = 0.0
    for shift in range(0, 15):
        x, w = e4(rows, k), e4(n, k)
        x[:, 1:32:2], w[:, 1:32:2] = x[:, 0:32:2], -w[:, 0:32:2]      # 16 pairs that cancel
        x[:, 32:] = (x[:, 32:] * 2.0 ** -(shift // 2)).to(torch.float8_e4m3fn).double()
        w[:, 32:] = (w[:, 32:] * 2.0 ** -(shift - shift // 2)).to(torch.float8_e4m3fn).double()
        byte = lambda v: v.to(torch.float8_e4m3fn).view(torch.uint8)
        y = layer.matmul(blocks(mp, byte(x), torch.full((rows, 4), 127), k, dev),
                         blocks(mp, byte(w)[None], torch.full((1, 1, 4), 127), k, dev), **kw).cpu().double()
        want, bound = refs.product(x, w)
        err = (y - want).abs()
        assert (err <= bound).all(), (shift, float((err - bound).max()))
        top = (x.abs()[:, None] * w.abs()[None]).amax(-1)
        worst = max(worst, float(((err - 2.0 ** -8 * want.abs()).clamp(min=0) / top).max()))
    print("beyond bf16's rounding: %.3g of the largest product" % worst, flush=True)
    layer.close()


def cut_bound(x, w):
    """Bound of a product's error at scales of 1, from what the matrix instruction keeps: in each group of eight
    consecutive values of the long axis, a product is cut off, towards zero, below 2^-13 of the group's largest
    2^(exponent of x + exponent of w), a subnormal's exponent being -6.  The largest itself, of 8 bits, loses nothing,
    so a group is off by less than seven times that.  Groups and steps are added in fp32 (2^-24 of a partial sum each)
    and the result rounded to bf16."""
    power = lambda v: torch.where(v == 0, 0.0, torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))))
    xp, wp = power(x).unflatten(1, (-1, 8)), power(w).unflatten(1, (-1, 8))
    quantum = 2.0 ** -13 * (xp[:, None] * wp[None]).amax(-1)
    y = x @ w.t()
    off = 7 * quantum.sum(-1) + (x.shape[1] / 8 + 4) * 2.0 ** -24 * (x.abs() @ w.abs().t())
    return y, 2.0 ** -8 * y.abs() + (1 + 2.0 ** -8) * off


@pytest.mark.parametrize("rows", [8, 64])
def test_what_the_matrix_instruction_keeps(mp, rows):
    """Random values over all of e4m3's range; groups of a pair that cancels and six products just below what is kept;
    and products that are all kept, whose sum is exact."""
    n, k, g = 48, 256, torch.Generator().manual_seed(rows)
    layer = mp.Layer(mp.make_config(rows, 1, 1, 1, 1, 8, 0), cooc=False)
    dev = layer.device
    kw = one_instance_each(mp, layer, [rows])

    def product(x, w):
        byte = lambda v: v.to(torch.float8_e4m3fn).view(torch.uint8)
        return layer.matmul(blocks(mp, byte(x), torch.full((rows, 4), 127), k, dev),
                            blocks(mp, byte(w)[None], torch.full((1, 1, 4), 127), k, dev), **kw).cpu().double()

    def any_value(*shape):
        b = torch.randint(0, 127, shape, generator=g) + 128 * torch.randint(0, 2, shape, generator=g)
        return b.to(torch.uint8).view(torch.float8_e4m3fn).double()

    def pairs(small):
        x, w = torch.ones(rows, k, dtype=torch.float64), torch.full((n, k), small, dtype=torch.float64)
        w[:, 0::8], w[:, 1::8] = 2.0 ** 8, -2.0 ** 8
        return x, w

    below = pairs(1.875 * 2.0 ** -6)
    for x, w in [(any_value(rows, k), any_value(n, k)) for _ in range(4)] + [below]:
        want, bound = cut_bound(x, w)
        assert ((product(x, w) - want).abs() <= bound).all()
    kept = pairs(2.0 ** -5)
    assert (product(*kept) == k * 6 / 8 * 2.0 ** -5).all()
    assert layer.status() == 0
    layer.close()


def forward(layer, st, m):
    """A forward pass of an expert layer and what its backward pass needs, as copies."""
    r, weight = layer.gate(m["logits"], st["gate"], bias=st["bias"])
    layer.plan()
    x = layer.quantize(layer.dispatch(m["hidden"]).dispatch)
    y1 = layer.matmul(x, st["w1"][0])
    a = layer.swiglu(y1)
    y2 = layer.matmul(a, st["w2"][0])
    out = layer.combine_weighted(y2, weight)
    d, p = layer.dispatch_out, layer.plan_out
    plan = dataclasses.replace(p, n_inst=p.n_inst.clone(), inst_expert=p.inst_expert.clone())
    return out, dict(x=x, y1=y1, a=a, y2=y2, weight=weight, topk_idx=r.topk_idx.clone(), slot_pos=d.slot_pos.clone(),
                     on=dict(plan=plan, inst_offset=d.inst_offset.clone()))


def backward(layer, st, m, s):
    at = dict(slot_pos=s["slot_pos"])
    dy2, dweight = layer.combine_grad(s["y2"], m["grad"], s["weight"], **at)
    dy2 = layer.quantize(dy2)
    dw2 = layer.wgrad(dy2, s["a"], **s["on"])
    dy1 = layer.swiglu_grad(s["y1"], layer.matmul(dy2, st["w2"][1], **s["on"]))
    dw1 = layer.wgrad(dy1, s["x"], **s["on"])
    dhidden = layer.combine_weighted(layer.matmul(dy1, st["w1"][1], **s["on"]), **at)
    return dw1, dw2, dhidden, layer.gate_grad(m["logits"], st["gate"], dweight, topk_idx=s["topk_idx"])


def test_two_forward_passes_before_their_backward_passes(mp):
    """With the kept top-k, plan, offsets and positions, each backward pass is that of its own forward pass."""
    T, E, k, R, G, H, F = 96, 16, 4, 2, 1, 256, 72
    cfg = mp.make_config(T, E, k, R, G, H, 2, expert_bytes=0)
    layer = mp.Layer(cfg)
    dev = layer.device
    g = torch.Generator().manual_seed(4)
    n = lambda *s, scale=1.0: (scale * torch.randn(*s, generator=g)).to(dev)
    st = dict(gate=mp.make_gate("sigmoid", 4, 2, 2, True, 2.5), bias=n(E, scale=0.1),
              w1=layer.quantize_weights(n(E, 2 * F, H, scale=H ** -0.5).to(BF), transposed=True),
              w2=layer.quantize_weights(n(E, H, F, scale=F ** -0.5).to(BF), transposed=True))
    batches = [dict(logits=n(T, E), hidden=n(T, H).to(BF), grad=n(T, H).to(BF)) for _ in range(2)]
    want = []
    for m in batches:
        alone = mp.Layer(cfg)
        out, s = forward(alone, st, m)
        want.append((out, *backward(alone, st, m, s)))
        assert alone.status() == 0
        alone.close()
    saved = [forward(layer, st, m) for m in batches]
    got = [(out, *backward(layer, st, m, s)) for m, (out, s) in zip(batches, saved)]
    for a, b in zip(got, want):
        assert all(torch.equal(t, u) for t, u in zip(a, b))
    assert not torch.equal(saved[0][1]["topk_idx"], saved[1][1]["topk_idx"]) and layer.status() == 0
    layer.close()


def test_no_result_of_a_side_stream_goes_to_another(mp):
    """Results of calls on a stream are dropped while the stream may still write them: tensors of the current stream,
    of the same sizes, never get their memory."""
    T, E, k, H, n = 64, 4, 1, 256, 48
    layer, side = mp.Layer(mp.make_config(T, E, k, 1, 1, H, 0), cooc=False), torch.cuda.Stream()
    dev = layer.device
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dev)
    kw = one_instance_each(mp, layer, [16] * 4)
    x, w, lg, gw = rnd(T, H).to(BF), rnd(E, n, H).to(BF), rnd(T, E), rnd(T, k)
    pos = torch.arange(T * k, dtype=torch.int32, device=dev)
    router = mp.make_gate("sigmoid")
    torch.cuda.synchronize()

    def everything():
        xb = layer.quantize(x, stream=side)
        wb, wt = layer.quantize_weights(w, transposed=True, stream=side)
        _, weight = layer.gate(lg, router, stream=side)
        y = layer.matmul(xb, wb, stream=side, **kw)
        yb = layer.quantize(y, stream=side)
        a, da = layer.swiglu(x, stream=side), layer.swiglu_grad(x, x[:, : H // 2].contiguous(), stream=side)
        return [xb.q, xb.scale, wb.q, wb.scale, wt.q, wt.scale, weight, y, yb.q, yb.scale, a.q, a.scale, da.q, da.scale,
                layer.matmul(yb, wt, stream=side, **kw), layer.wgrad(yb, xb, stream=side, **kw),
                layer.gate_grad(lg, router, gw, stream=side), layer.combine_weighted(x, gw, slot_pos=pos, stream=side),
                *layer.combine_grad(x, x, gw, slot_pos=pos, stream=side)]

    results = everything()
    freed, shapes = {t.data_ptr() for t in results}, [(t.shape, t.dtype) for t in results]
    assert len(freed) == len(results)
    del results
    taken = [torch.empty(s, dtype=d, device=dev) for s, d in shapes for _ in range(4)]
    assert not freed & {t.data_ptr() for t in taken}
    side.synchronize()
    assert layer.status() == 0
    layer.close()


def test_limits_of_sizes(mp):
    """Each stated limit is the last size taken; the sizes past it are refused before any device work."""
    layer = mp.Layer(mp.make_config(8, 4, 1, 1, 1, 8, 0), cooc=False)
    lib, h, big, bad, dev = mp.lib(), layer.handle, mp.MOE_ERR_UNSUPPORTED, mp.MOE_ERR_INVALID_ARG, layer.device
    x = torch.zeros(1 << 12, dtype=torch.uint8, device=dev)
    p = x.data_ptr()
    row = {"quantize": lambda r, c: lib.moex_quantize(h, p, r, c, p, p, None),
           "swiglu": lambda r, c: lib.moex_swiglu(h, p, r, c, p, p, None),
           "swiglu_grad": lambda r, c: lib.moex_swiglu_grad(h, p, p, r, c, p, p, None)}
    for name, call in row.items():
        assert call(1 << 31, 1) == big and call(1, (1 << 24) + 1) == big, name
        assert call(-1, 1) == bad and call(1, 0) == bad, name
        assert call(0, 1 << 24) == mp.MOE_OK, name
    mats = lambda e, n, k: lib.moex_quantize_weights(h, p, e, n, k, p, p, None, None, None)
    assert mats(1, (1 << 24) + 1, 1) == big and mats(1, 1, (1 << 24) + 1) == big
    assert mats(1 << 24, 1, 1) == big and mats(1 << 14, 1 << 12, 1 << 12) == big
    assert mats(-1, 1, 1) == bad and mats(1, 0, 1) == bad and mats(1, 1, 0) == bad
    assert mats(0, 1 << 24, 1 << 24) == mp.MOE_OK
    # the widest row: the last value of 2^24 and its block
    wide = torch.zeros(1, 1 << 24, dtype=BF, device=dev)
    wide[0, -1] = 3.0
    b = layer.quantize(wide)
    assert b.q[0, -1].item() * 2.0 ** (int(b.scale.view(torch.uint8)[0, -1]) - 127) == 3.0
    assert int((b.q.view(torch.uint8) != 0).sum()) == 1
    torch.cuda.synchronize()
    assert layer.status() == 0 and int((x != 0).sum()) == 0
    layer.close()


def test_counts_of_blocks_past_64_bits_are_refused(mp):
    """experts * blocks per matrix would be 2^63, 2^64 and more, negative or small where it wraps."""
    layer = mp.Layer(mp.make_config(8, 4, 1, 1, 1, 8, 0), cooc=False)
    p = torch.zeros(64, dtype=torch.uint8, device=layer.device).data_ptr()
    for experts, n, k in ((1 << 29, 1 << 24, 1 << 24), (1 << 30, 1 << 24, 1 << 24), ((1 << 31) - 1, 1 << 24, 1 << 24),
                          ((1 << 30) + 1, (1 << 24) - 128, (1 << 24) - 256), (1 << 30, 1 << 23, 1 << 24)):
        assert mp.lib().moex_quantize_weights(layer.handle, p, experts, n, k, p, p, None, None, None) == mp.MOE_ERR_UNSUPPORTED
    assert layer.status() == 0
    layer.close()


def test_a_bad_plan_of_no_tokens(mp):
    """The status word tells of a bad count, expert or offset also where there are no rows."""
    layer = mp.Layer(mp.make_config(0, 4, 2, 1, 1, 64, 0), cooc=False)
    dev = layer.device
    rows = layer.quantize(torch.empty(0, 64, dtype=BF, device=dev))
    dy = layer.quantize(torch.empty(0, 48, dtype=BF, device=dev))
    w = layer.quantize_weights(torch.zeros(4, 48, 64, dtype=BF, device=dev))
    for change, want in ((lambda: None, 0), (lambda: layer.plan_out.n_inst.fill_(5), mp.MOE_STATUS_PLAN_CHECK),
                         (lambda: layer.plan_out.inst_expert[2].fill_(4), mp.MOE_STATUS_PLAN_CHECK),
                         (lambda: layer.dispatch_out.inst_offset[1].fill_(1), mp.MOE_STATUS_PLAN_CHECK)):
        layer.plan_out.n_inst.fill_(4)
        layer.plan_out.inst_expert.copy_(torch.arange(4))
        layer.dispatch_out.inst_offset.zero_()
        change()
        assert layer.matmul(rows, w).shape == (0, 48)
        assert layer.status() == want
        assert (layer.wgrad(dy, rows) == 0).all()
        assert layer.status() == want
    layer.close()


@pytest.mark.parametrize("rows,n,k", [(2048, 48, 96), (2048, 8200, 2100)])
def test_repeated_rows_end_at_the_buffer_s_rows(mp, rows, n, k):
    """Every second of 32 instances holds all rows, and those between fall back: an expert's rows are summed until
    there were T*k of them, in both tile sizes."""
    E, B = 4, 28
    layer = mp.Layer(mp.make_config(rows, E, 1, 1, 1, 8, B), cooc=False)
    dev = layer.device
    g = torch.Generator().manual_seed(n)
    x, dy = (layer.quantize(torch.randn(rows, c, generator=g).to(BF).to(dev)) for c in (k, n))
    layer.plan_out.inst_expert.copy_(torch.arange(E + B) // 2 % E)   # two instances an expert, in turn: a whole and a bad one
    layer.plan_out.n_inst.fill_(E + B)
    layer.dispatch_out.inst_offset.copy_(torch.tensor([0, rows] * 16 + [0], dtype=torch.int32))
    got = layer.wgrad(dy, x)
    assert layer.status() == mp.MOE_STATUS_PLAN_CHECK
    one = one_instance_each(mp, layer, [rows] + [0] * (E + B - 1))
    one["plan"].n_inst.fill_(1)
    want = layer.wgrad(dy, x, **one)[0]
    assert layer.status() == 0 and bool(want.abs().sum() > 0)
    for e in range(E):
        assert torch.equal(got[e], want), e
    layer.close()


def test_results_into_given_memory(mp):
    """Every call that returns new memory writes the same bytes into `out`, and refuses one of another shape or type."""
    T, E, k, H, n = 48, 6, 2, 264, 136
    layer = mp.Layer(mp.make_config(T, E, k, 1, 1, H, 0), cooc=False)
    dev = layer.device
    g = torch.Generator().manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dev)
    x, w, lg, gw = rnd(T * k, H).to(BF), rnd(E, n, H).to(BF), rnd(T, E), rnd(T, k)
    pos = torch.randperm(T * k, generator=g).int().to(dev)
    router = mp.make_gate("softmax")
    half, grad = x[:, : H // 2].contiguous(), rnd(T, H).to(BF)

    def flat(r):
        if isinstance(r, mp.Blocks):
            return [r.q, r.scale]
        return [t for part in r for t in flat(part)] if isinstance(r, tuple) else [r]

    calls = (lambda **o: layer.quantize(x, **o), lambda **o: layer.quantize_weights(w, **o),
             lambda **o: layer.quantize_weights(w, transposed=True, **o), lambda **o: layer.swiglu(x, **o),
             lambda **o: layer.swiglu_grad(x, half, **o), lambda **o: layer.gate(lg, router, **o)[1],
             lambda **o: layer.combine_grad(x, grad, gw, slot_pos=pos, **o))
    for i, call in enumerate(calls):
        want, out = call(), call()
        for t in flat(out):
            t.view(torch.uint8).fill_(0x55)
        got = call(out=out)
        assert all(a is b for a, b in zip(flat(got), flat(out))), i
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(flat(got), flat(want))), i
    blocks_ = layer.quantize(x)
    for bad in (lambda: layer.quantize(x[:-1].contiguous(), out=blocks_), lambda: layer.quantize(half, out=blocks_),
                lambda: layer.quantize(x, out=mp.Blocks(blocks_.q, blocks_.scale, H + 1)),
                lambda: layer.swiglu(x, out=blocks_), lambda: layer.swiglu_grad(x, half, out=layer.quantize(half)),
                lambda: layer.quantize_weights(w, out=blocks_), lambda: layer.gate(lg, router, out=gw[:-1].contiguous()),
                lambda: layer.combine_grad(x, grad, gw, slot_pos=pos, out=(x[:-1].contiguous(), gw))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: layer.gate(lg, router, out=gw.double()),
                lambda: layer.quantize(x, out=mp.Blocks(blocks_.q.view(torch.uint8), blocks_.scale, H)),
                lambda: layer.combine_grad(x, grad, gw, slot_pos=pos, out=(x.to(torch.float16), gw))):
        with pytest.raises(TypeError):
            bad()
    assert layer.status() == 0
    layer.close()


def test_a_graph_sees_matrices_quantized_in_place(mp):
    """A captured product, and matrices that an optimizer step changed, quantized into the Blocks that it reads."""
    E, n, k, rows = 4, 136, 264, 64
    layer = mp.Layer(mp.make_config(rows, E, 1, 1, 1, 8, 0), cooc=False)
    dev = layer.device
    kw = one_instance_each(mp, layer, [20, 0, 40, 4])
    g = torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF).to(dev)
    x, d = layer.quantize(rnd(rows, k)), layer.quantize(rnd(rows, n))
    pair = layer.quantize_weights(rnd(E, n, k), transposed=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx = layer.matmul(x, pair[0], **kw), layer.matmul(d, pair[1], **kw)
    for _ in range(4):
        w = rnd(E, n, k)
        layer.quantize_weights(w, transposed=True, out=pair)
        graph.replay()
        torch.cuda.synchronize()
        new = layer.quantize_weights(w, transposed=True)
        assert torch.equal(y, layer.matmul(x, new[0], **kw)) and torch.equal(dx, layer.matmul(d, new[1], **kw))
    assert layer.status() == 0
    layer.close()


@pytest.mark.parametrize("f", [128, 200])
def test_gates_far_below_zero(mp, f):
    """Blocks whose gates are all far below zero, down to where fp32 ends.  expf and its argument are good to 2 + |x|
    units, so a value is off by 2^-17 of itself; a sigmoid below 2^-128 counts as 0, which takes up to 2^-128 of what it
    is multiplied by; then e4m3's half step."""
    rows = 24
    g = torch.Generator().manual_seed(f)
    y = torch.randn(rows, 2 * f, generator=g)
    y[:, :f] = -torch.linspace(78, 99, rows)[:, None] - 0.3 * torch.rand(rows, f, generator=g)
    y, da = y.to(BF), torch.randn(rows, f, generator=g).to(BF)
    layer = mp.Layer(mp.make_config(8, 8, 1, 1, 1, 8, 0), cooc=False)
    dev = layer.device
    y64 = y.double().requires_grad_()
    act = refs.swiglu(y64)
    grad, = torch.autograd.grad(act, y64, da.double())
    gate, up, d = y.double()[:, :f].abs(), y.double()[:, f:].abs(), da.double().abs()
    for got, want, size, c in ((layer.swiglu(y.to(dev)), act.detach(), gate * up, f),
                               (layer.swiglu_grad(y.to(dev), da.to(dev)), grad,
                                torch.cat([d * up * (1 + gate), d * gate], 1), 2 * f)):
        scale = (got.scale.view(torch.uint8).cpu().double()[:, : refs.pad(c) // 128] - 127).exp2().repeat_interleave(128, -1)[:, :c]
        off = 2.0 ** -17 * want.abs() + 2.0 ** -128 * size + 2.0 ** -148
        half = torch.maximum(2.0 ** -4 * (want.abs() + off), 2.0 ** -10 * scale)
        assert ((refs.values(got, rows) - want).abs() <= off + half).all()
        # the block's scale is no larger than its largest value needs, or 1 where all are 0
        top, zero = refs.block_max(want.abs() + off), refs.block_max(refs.values(got, rows)) == 0
        assert ((scale[:, ::128] <= torch.exp2(refs.block_exponent(top).double())) | (zero & (scale[:, ::128] == 1))).all()
    assert layer.status() == 0
    layer.close()
