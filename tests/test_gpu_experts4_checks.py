"""The 4-bit operators and the layer of few tokens at the ends of their contract: the most channels, every operand of a
backward pass, the inputs that only a conversion instruction sees."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import expert4_refs as refs4
from tests import expert_refs as refs
from tests.test_gpu_experts4 import BF, instances, layer_for, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import load_balance_planning_amd as m
    m.lib()
    return m


# ---- the most channels ------------------------------------------------------------

def test_products_of_the_most_channels(mp):
    """2^20 channels, and up to 2048 instances, of which 30 are there: they are of the first 8 of 1024 experts, and only
    those have matrices."""
    rows, E, B, n, k, used, count = 6148, 1024, 1024, 1 << 20, 256, 8, 30
    print("products4 of %d channels, %d experts" % (n, E), flush=True)
    layer = mp.Layer(mp.make_config(rows, E, 1, 4, 1, 8, B), cooc=False)
    dev = layer.device
    rng = np.random.RandomState(0)
    loads = rng.multinomial(rows, rng.dirichlet(np.full(count, 0.5)))
    plan, off, spans = instances(mp, layer, loads, rng.randint(0, used, count))
    x = layer.quantize4(normal(1, rows, k).to(dev))
    w = torch.randn(used, n, k, device=dev, dtype=BF, generator=torch.Generator(device=dev).manual_seed(2)) * 2 ** -4
    wb = layer.quantize_weights4(w)
    del w
    y = torch.full((rows, n), 7.0, dtype=BF, device=dev)
    p = lambda t: t.data_ptr()
    mp.moex4_matmul(layer.handle, plan.struct(), p(off), 4, p(x.q), p(x.scale), p(wb.q), p(wb.scale), n, k, p(y),
                    torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert layer.status() == 0
    at = torch.cat([torch.arange(300), torch.from_numpy(rng.randint(0, n, 400)), torch.arange(n - 300, n)])
    q, s = wb.q.view(torch.uint8)[:, at.to(dev)], wb.scale.view(torch.uint8)[:, :, at.to(dev)].contiguous()
    wv = refs4.values(mp.Blocks4(q.contiguous(), s.view(torch.float8_e8m0fnu), k))
    xv, got, seen = refs4.values(x), y[:, at.to(dev)].cpu().double(), 0
    for e, a, z in spans:
        want = xv[a:z] @ wv[e].t()
        assert ((got[a:z] - want).abs() <= refs4.rounded(want, refs4.added(xv[a:z], wv[e]))).all()
        seen += z - a
    assert seen == rows
    layer.close()


def test_more_tiles_than_the_limit_are_refused(mp):
    """2^26 rows by 2^20 channels: refused on the host, whatever the memory."""
    layer = mp.Layer(mp.make_config(1 << 21, 32, 32, 1, 1, 8, 0), cooc=False, topk_val=False)
    plan, off, _ = instances(mp, layer, [8], [0])
    s, p, some = plan.struct(), off.data_ptr(), torch.zeros(64, dtype=torch.uint8, device=layer.device).data_ptr()
    for bits in (4, 8):
        assert mp.lib().moex4_matmul(layer.handle, ctypes.byref(s), p, bits, some, some, some, some, 1 << 20, 256, some,
                                     None) == mp.MOE_ERR_UNSUPPORTED
    layer.close()
