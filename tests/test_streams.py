"""Which stream the calls of a Layer go to."""
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
