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
