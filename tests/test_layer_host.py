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
