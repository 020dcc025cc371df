"""include/moe_experts4.h: every declared entry point is exported, bound and refuses a null handle before any device
work; the binding's shapes follow the header's layout (no GPU needed)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def declared():
    text = open(os.path.join(ROOT, "include", "moe_experts4.h")).read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*int\s+(moex4_\w+)\s*\(", text, flags=re.M)))


def test_every_declared_entry_point_is_exported_and_bound():
    import load_balance_planning_amd as m
    lib = m.lib()
    out = subprocess.run(["nm", "-D", "--defined-only", m.lib_path()], capture_output=True, text=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert len(declared()) == 7
    assert set(declared()) <= exported
    assert set(m.EXPERT4_EXPORTS) == set(declared())
    for name in declared():
        assert callable(getattr(m, name)) and getattr(lib, name).argtypes is not None, name


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "moe_experts4.h"\nint main(void) { return moex4_quantize == 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-Wno-address", "-fsyntax-only", "-I",
                    os.path.join(ROOT, "include"), str(src)], check=True)


def test_a_null_handle_is_refused():
    import load_balance_planning_amd as m
    lib = m.lib()
    calls = {
        "moex4_quantize": (None, None, 1, 1, None, None, None),
        "moex4_quantize_weights": (None, None, 1, 1, 1, None, None, None, None, None),
        "moex4_values": (None, None, None, 1, 1, 1, None, None),
        "moex4_swiglu": (None, None, 1, 1, None, None, None),
        "moex4_matmul": (None, None, None, 4, None, None, None, None, 1, 1, None, None),
        "moex4_experts_work": (None, 1, None),
        "moex4_experts": (None, None, None, None, 4, 1) + (None,) * 7,
    }
    assert set(calls) == set(declared())
    for name, args in calls.items():
        assert getattr(lib, name)(*args) == m.MOE_ERR_INVALID_ARG, name


@pytest.mark.parametrize("cols,padded", [(1, 256), (256, 256), (257, 512), (2048, 2048), (2688, 2816), (7168, 7168)])
def test_shapes(cols, padded):
    import load_balance_planning_amd as m
    assert m.Blocks4.padded(cols) == padded
    assert m.Blocks4.shapes((5,), cols) == ((5, padded // 2), (padded // 256, 5, 8))
    assert m.Blocks4.shapes((3, 5), cols) == ((3, 5, padded // 2), (3, padded // 256, 5, 8))


def test_the_binding_names_the_scales_types():
    import load_balance_planning_amd as m
    assert (m.BLOCK4, m.LINE4, m.FEW_TOKENS) == (32, 256, 64)


def cpu_layer(m, monkeypatch, T=8, E=4, k=2, H=64):
    """A Layer of host tensors without a handle: every check of its calls passes or refuses, and behind them the library
    refuses the handle."""
    torch = pytest.importorskip("torch")
    layer = object.__new__(m.Layer)
    layer.torch, layer._index, layer.device, layer.handle = torch, -1, torch.device("cpu"), None
    layer._bf16, layer._fp4, layer._e8m0 = torch.bfloat16, torch.float4_e2m1fn_x2, torch.float8_e8m0fnu
    layer._dims, layer._cap, layer._few = (T, E, k, H), E, {}
    layer._current_stream = lambda i: 0
    monkeypatch.setattr(m, "moex4_experts_work", lambda h, f: 4096)
    layer._empty = lambda shape, dtype, stream=None: torch.empty(shape, dtype=dtype)
    return torch, layer


def blocks4(m, torch, lead, cols):
    q, scale = m.Blocks4.shapes(lead, cols)
    return m.Blocks4(torch.zeros(q, dtype=torch.uint8).view(torch.float4_e2m1fn_x2),
                     torch.full(scale, 127, dtype=torch.uint8).view(torch.float8_e8m0fnu), cols)


def test_refusals_before_the_library(monkeypatch):
    import load_balance_planning_amd as m
    torch, layer = cpu_layer(m, monkeypatch)
    T, E, k, H = layer._dims
    b = lambda lead, cols: blocks4(m, torch, lead, cols)
    x, y = torch.zeros(5, 70, dtype=torch.bfloat16), torch.zeros(T, H, dtype=torch.bfloat16)
    good = [
        lambda: layer.quantize4(x), lambda: layer.quantize4(x, out=b((5,), 70)), lambda: layer.swiglu4(x),
        lambda: layer.values4(b((5,), 70)), lambda: layer.values4(b((3, 5), 300)),
        lambda: layer.quantize_weights4(x.view(1, 5, 70), transposed=True, out=(b((1, 5), 70), b((1, 70), 5))),
        lambda: layer.experts(y, torch.zeros(T, k), b((E, 64), H), b((E, H), 32), topk_idx=torch.zeros(T, k, dtype=torch.int32)),
    ]
    for call in good:
        with pytest.raises(m.MoePlanError):
            call()
    idx, weight, w1, w2 = torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k), b((E, 64), H), b((E, H), 32)
    few = lambda **kw: layer.experts(**{**dict(hidden=y, weight=weight, w1=w1, w2=w2, topk_idx=idx), **kw})
    for call, error in (
            (lambda: layer.quantize4(x.float()), TypeError), (lambda: layer.quantize4(x[:, ::2]), ValueError),
            (lambda: layer.quantize4(x, out=b((5,), 71)), ValueError), (lambda: layer.quantize4(x, out=b((4,), 70)), ValueError),
            (lambda: layer.swiglu4(x[:, :69].contiguous()), ValueError), (lambda: layer.values4(m.Blocks4(b((5,), 70).q[0], b((5,), 70).scale, 70)), ValueError),
            (lambda: layer.values4(m.Blocks4(b((5,), 70).q, b((5,), 300).scale, 70)), ValueError),
            (lambda: layer.values4(b((5,), 70), out=x[:4]), ValueError),
            (lambda: layer.quantize_weights4(x), ValueError),
            (lambda: layer.quantize_weights4(x.view(1, 5, 70), transposed=True, out=(b((1, 5), 70), b((1, 5), 70))), ValueError),
            (lambda: few(hidden=y[:4]), ValueError), (lambda: few(hidden=y.half()), TypeError),
            (lambda: few(weight=weight[:, :1]), ValueError), (lambda: few(weight=weight.bfloat16()), TypeError),
            (lambda: few(topk_idx=idx.long()), TypeError), (lambda: few(topk_idx=idx.t()), ValueError),
            (lambda: few(w1=b((E, 62), H)), ValueError), (lambda: few(w1=b((E, 64), H + 1)), ValueError),
            (lambda: few(w2=b((E, H + 1), 32)), ValueError), (lambda: few(w2=b((E + 1, H), 32)), ValueError),
            (lambda: few(out=y), ValueError), (lambda: few(out=torch.zeros(T, H)), TypeError),
            (lambda: few(w2=m.Blocks(torch.zeros(E, H, 128).to(torch.float8_e4m3fn), w2.scale, 32)), TypeError)):
        with pytest.raises(error):
            call()
