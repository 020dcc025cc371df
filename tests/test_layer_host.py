"""Layer's own part of a call, on host tensors: what it needs of torch, and what it refuses before the library (no GPU
needed)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")


def made_on_host(m, monkeypatch, T=6, E=4, k=2, H=64):
    """A Layer by its own constructor, on the CPU and without a handle."""
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "device", lambda index: contextlib.nullcontext())
    monkeypatch.setattr(m, "moe_plan_create", lambda cfg: None)
    layer = m.Layer(m.make_config(T, E, k, 1, 1, H, 0), device=torch.device("cpu", 0))
    layer._index, layer._current_stream = -1, lambda index: 0  # as host tensors have it
    return layer


def test_a_layer_needs_no_narrow_types_of_torch(monkeypatch):
    """A torch without the 4-bit type, or without the scales' type, still plans; the calls that need one name it."""
    import load_balance_planning_amd as m
    for name in ("float4_e2m1fn_x2", "float8_e8m0fnu"):
        with monkeypatch.context() as patch:
            patch.delattr(torch, name)
            layer = made_on_host(m, patch)
            assert layer.route_out.topk_idx.shape == (6, 2) and layer.dispatch_out.dispatch.shape == (12, 64)
            # past every check, to the library that refuses the missing handle
            with pytest.raises(m.MoePlanError):
                layer.route(torch.zeros(6, 4))
            x = torch.zeros(5, 70, dtype=torch.bfloat16)
            with pytest.raises(AttributeError, match=name):
                layer.quantize4(x)


def matrices4(m, E, n, k):
    q, scale = m.Blocks4.shapes((E, n), k)
    return m.Blocks4(torch.zeros(q, dtype=torch.uint8).view(torch.float4_e2m1fn_x2),
                     torch.full(scale, 127, dtype=torch.uint8).view(torch.float8_e8m0fnu), k)


def test_few_tokens_results_lie_over_nothing_that_is_read(monkeypatch):
    """`out` in the memory of any argument of experts(), at its beginning and at its end, is refused; beside them all
    it passes to the library (which refuses the handle)."""
    import load_balance_planning_amd as m
    T, E, k, H, f = 4, 8, 8, 64, 32
    layer = made_on_host(m, monkeypatch, T, E, k, H)
    monkeypatch.setattr(m, "moex4_experts_work", lambda h, f: 4096)
    layer._few = {}
    size = T * H * 2
    # every argument in one buffer, each with room for a result before and behind it
    w1, w2 = matrices4(m, E, 2 * f, H), matrices4(m, E, H, f)
    args = dict(hidden=torch.zeros(T, H, dtype=torch.bfloat16), topk_idx=torch.zeros(T, k, dtype=torch.int32),
                weight=torch.zeros(T, k), q1=w1.q, s1=w1.scale, q2=w2.q, s2=w2.scale)
    buf = torch.zeros(len(args) * (size + (1 << 16)), dtype=torch.uint8)
    at, placed, ends = 0, {}, {}
    for name, t in args.items():
        at += size
        n = t.numel() * t.element_size()
        placed[name] = buf[at:at + n].view(t.dtype).view(t.shape)
        ends[name] = (at, at + n)
        at += n + 512
    call = lambda out: layer.experts(placed["hidden"], placed["weight"], m.Blocks4(placed["q1"], placed["s1"], H),
                                     m.Blocks4(placed["q2"], placed["s2"], f), topk_idx=placed["topk_idx"], out=out)
    result = lambda begin: buf[begin:begin + size].view(torch.bfloat16).view(T, H)
    for name, (begin, end) in ends.items():
        for over in (begin - size + 2, begin, end - 2):
            with pytest.raises(ValueError, match="overlaps"):
                call(result(over))
        with pytest.raises(m.MoePlanError):
            call(result(begin - size))


@pytest.mark.parametrize("four", [True, False])
def test_both_layouts_into_the_same_memory_are_refused(monkeypatch, four):
    """Square matrices, whose two layouts have the same shapes."""
    import load_balance_planning_amd as m
    layer = made_on_host(m, monkeypatch)
    w = torch.zeros(2, 256, 256, dtype=torch.bfloat16)
    if four:
        quant, one = layer.quantize_weights4, lambda: matrices4(m, 2, 256, 256)
    else:
        quant = layer.quantize_weights
        one = lambda: m.Blocks(torch.zeros(2, 256, 256, dtype=torch.uint8).view(torch.float8_e4m3fn),
                               torch.zeros(2, 2, 4, dtype=torch.uint8).view(torch.float8_e8m0fnu), 256)
    a, b = one(), one()
    for pair in ((a, a), (a, type(a)(b.q, a.scale, 256)), (a, type(a)(a.q, b.scale, 256))):
        with pytest.raises(ValueError, match="overlap"):
            quant(w, transposed=True, out=pair)
    with pytest.raises(m.MoePlanError):  # past every check: the library refuses the handle
        quant(w, transposed=True, out=(a, b))


@pytest.mark.parametrize("lead,cols", [((5,), 256), ((3,), 32), ((4,), 300), ((2, 7), 1000), ((3, 40), 2688)])
def test_matrices_in_the_published_order(lead, cols):
    """The documented way to bring values and scales, both row by row, into Blocks4: the same values, padding of zeros."""
    import os
    import load_balance_planning_amd as m
    from tests import expert4_refs as refs4
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    code = text[text.index("def published_blocks4"):]
    scope = {"torch": torch, "mp": m}
    exec(code[: code.index("```")], scope)
    g = torch.Generator().manual_seed(cols)
    n = -(-cols // 32)
    code4 = torch.randint(0, 16, (*lead, 2 * -(-cols // 2)), generator=g)
    code4[..., cols:] = 0
    scale = torch.randint(90, 160, (*lead, n), generator=g)
    table = torch.cat([refs4.CODES, -refs4.CODES])
    want = (table[code4][..., :cols] * torch.exp2(scale.double() - 127).repeat_interleave(32, -1)[..., :cols])
    q = (code4[..., ::2] | code4[..., 1::2] << 4).to(torch.uint8)
    b = scope["published_blocks4"](q, scale.to(torch.uint8), cols)
    assert (tuple(b.q.shape), tuple(b.scale.shape)) == m.Blocks4.shapes(lead, cols)
    assert b.q.is_contiguous() and b.scale.is_contiguous()
    assert torch.equal(refs4.values(b), want)
    assert (refs4.codes(b)[..., cols:] == 0).all() and (refs4.scales(b)[..., n:] == 1).all()
