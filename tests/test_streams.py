"""Checks of a Layer before its calls: which stream they go to, and results that overlap what is read."""
from __future__ import annotations

from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")


def test_a_torch_without_the_private_lookup_goes_through_the_public_one():
    import load_balance_planning_amd as mp
    asked = []
    public = SimpleNamespace(current_stream=lambda i: asked.append(i) or SimpleNamespace(cuda_stream=0x1230 + i))
    bare = SimpleNamespace(_C=SimpleNamespace(), cuda=public)
    assert mp._current_stream(bare)(3) == 0x1233 and asked == [3]
    own = SimpleNamespace(_C=SimpleNamespace(_cuda_getCurrentRawStream=lambda i: 0x4560 + i), cuda=public)
    assert mp._current_stream(own)(3) == 0x4563 and asked == [3]


@pytest.mark.gpu
def test_the_lookup_names_the_current_stream():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import load_balance_planning_amd as mp
    lookup = mp._current_stream(torch)
    index = torch.cuda.current_device()
    handles = set()
    for stream in [torch.cuda.default_stream()] + [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(stream):
            assert lookup(index) == torch.cuda.current_stream(index).cuda_stream == stream.cuda_stream
            handles.add(lookup(index))
    assert len(handles) == 4


def bare_layer(mp, index=0):
    """A Layer without a device behind it, for the checks that come before any device work."""
    layer = object.__new__(mp.Layer)
    layer.torch, layer._index, layer.device, layer.handle = torch, index, torch.device("cuda", index), None
    layer._current_stream = lambda i: 0x10 + i
    return layer


def test_a_stream_of_another_device_is_refused():
    import load_balance_planning_amd as mp
    layer = bare_layer(mp)
    assert layer._stream() == 0x10
    assert layer._stream(SimpleNamespace(device_index=0, cuda_stream=0x77)) == 0x77
    other = SimpleNamespace(device_index=1, cuda_stream=0x78)
    with pytest.raises(ValueError):
        layer._stream(other)
    with pytest.raises(ValueError):
        layer._empty((4,), torch.float32, other)


@pytest.mark.gpu
def test_an_external_stream_is_taken():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import load_balance_planning_amd as mp
    layer = mp.Layer(mp.make_config(8, 4, 1, 1, 1, 8, 0), cooc=False)
    x = torch.ones(4, 8, dtype=torch.bfloat16, device=layer.device)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = layer.quantize(x, stream=torch.cuda.ExternalStream(side.cuda_stream))
    side.synchronize()
    assert (b.q[:, :8].float() * 2.0 ** (b.scale.view(torch.uint8)[:, :1].float() - 127) == 1).all()
    assert layer.status() == 0
    layer.close()


def test_results_over_the_rows_that_are_read_are_refused():
    import load_balance_planning_amd as mp
    rows = torch.zeros(8, 4, dtype=torch.bfloat16)
    for out, fine in ((rows, False), (rows[7:], False), (rows[:1], False), (torch.zeros(8, 4), True)):
        if fine:
            mp.Layer._check_apart(out, rows)
        else:
            with pytest.raises(ValueError):
                mp.Layer._check_apart(out, rows)
    mp.Layer._check_apart(rows[4:], rows[:4])
    mp.Layer._check_apart(rows[:4], rows[4:])


@pytest.mark.gpu
def test_combines_refuse_results_over_their_rows():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import load_balance_planning_amd as mp
    T, k, H = 8, 2, 16
    layer = mp.Layer(mp.make_config(T, 4, k, 1, 1, H, 0), cooc=False)
    buf = torch.ones(2 * T * k, H, dtype=torch.bfloat16, device=layer.device)
    rows, w = buf[: T * k], torch.ones(T, k, device=layer.device)
    pos = torch.arange(T * k, dtype=torch.int32, device=layer.device)
    g = torch.ones(T, H, dtype=torch.bfloat16, device=layer.device)
    with pytest.raises(ValueError):
        layer.combine_weighted(rows, w, slot_pos=pos, out=rows[T:])
    for out in (rows, buf[T: T + T * k]):
        with pytest.raises(ValueError):
            layer.combine_grad(rows, g, w, slot_pos=pos, out=(out, w.clone()))
    with pytest.raises(ValueError):
        layer.combine_grad(rows, buf[T * k + 3: T * k + 3 + T], w, slot_pos=pos, out=(buf[T * k:], w.clone()))
    assert (layer.combine_weighted(rows, w, slot_pos=pos, out=buf[T * k: T * k + T]) == 2).all()
    assert (layer.combine_grad(rows, g, w, slot_pos=pos, out=(buf[T * k:], w.clone()))[0] == 1).all()
    assert layer.status() == 0
    layer.close()
