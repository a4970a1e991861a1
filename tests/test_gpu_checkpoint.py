"""GPU checks of the 8-bit checkpoints (lce_pack8, lce_unpack8) against the
64-bit definition: the codes' values and the scales are exact, so equality is
asked for."""
import numpy as np
import pytest
import torch

from lm_head_linear_amd import lce
from tests import ops_plain

pytestmark = pytest.mark.gpu
TYPES = {"bf16": (torch.bfloat16, 3.3895313892515355e38, -117), "fp16": (torch.float16, 65504.0, -15)}


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _values(n, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, d, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g))
    x[torch.rand(n, d, generator=g) < 0.05] = 0.0
    if n > 2:
        x[1] = 0.0                                      # a row of zeros
    x[torch.rand(n, d, generator=g) < 0.02] *= 100.0    # wide values inside a block
    return x.to(dt)


def _same(a, b):
    return np.array_equal(a, b, equal_nan=True)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n,d", [(1, 1), (1, 31), (3, 32), (5, 33), (2, 64), (7, 511), (4, 512),
                                 (3, 513), (37, 1003), (129, 4096), (1, 20000), (4097, 8)])
def test_pack_and_unpack(n, d, dt):
    dev = _dev()
    print(f"case checkpoint {n}x{d} {dt}", flush=True)
    t, most, lowest = TYPES[dt]
    x = _values(n, d, t, 100 + n + d)
    want, e = ops_plain.checkpoint(x.double().numpy(), most, lowest)
    p = lce.pack8(x.to(dev))
    got = lce.unpack8(p)
    assert got.dtype == t and got.shape == x.shape
    assert np.array_equal(p.scales.cpu().numpy().astype(np.int64) - 127, e)
    assert _same(got.double().cpu().numpy(), want)
    # reading back and packing again changes nothing
    again = lce.unpack8(lce.pack8(got))
    assert torch.equal(again, got)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_edges_of_the_type(dt):
    """Every power of two and its neighbours, largest, smallest, infinite and
    NaN values, each alone in its block and next to ordinary ones."""
    dev = _dev()
    t, most, lowest = TYPES[dt]
    info = torch.finfo(t)
    v = [0.0, -0.0, info.max, -info.max, info.tiny, info.tiny / 8, float("inf"), -float("inf"),
         float("nan"), 448.0, 449.0, 464.0, 480.0, 0.875, 0.9375, 1.75, 1.7578125, 2.0 ** -9]
    v += [s * 2.0 ** k for k in range(-24, 16) for s in (1.0, 1.5, 1.75, 1.875, -1.96875)]
    x = torch.zeros(2 * len(v), 32)
    for i, a in enumerate(v):
        x[i, 5] = a
        x[len(v) + i] = torch.linspace(-3, 3, 32)
        x[len(v) + i, 31] = a
    x = x.to(t)
    want, e = ops_plain.checkpoint(x.double().numpy(), most, lowest)
    p = lce.pack8(x.to(dev))
    assert np.array_equal(p.scales.cpu().numpy().astype(np.int64) - 127, e)
    assert _same(lce.unpack8(p).double().cpu().numpy(), want)


def test_views_and_untouched_neighbours():
    """Bases that are not 16-byte aligned; what lies around the outputs stays."""
    dev = _dev()
    n, d = 9, 77
    x = _values(1, n * d + 5, torch.bfloat16, 3).view(-1).to(dev)
    v = x[5:].view(n, d)
    nb = -(-d // 32)
    codes = torch.full((n * d + 40,), 7, dtype=torch.uint8, device=dev)
    scales = torch.full((n * nb + 40,), 9, dtype=torch.uint8, device=dev)
    assert lce.lce_pack8(v, n, d, codes[3:3 + n * d], scales[1:1 + n * nb]) == 580
    want, e = ops_plain.checkpoint(v.double().cpu().numpy(), TYPES["bf16"][1], -117)
    out = torch.full((n * d + 40,), 5.0, dtype=torch.bfloat16, device=dev)
    assert lce.lce_unpack8(codes[3:3 + n * d], scales[1:1 + n * nb], n, d, out[7:7 + n * d]) == 580
    assert _same(out[7:7 + n * d].view(n, d).double().cpu().numpy(), want)
    assert bool((out[:7] == 5).all()) and bool((out[7 + n * d:] == 5).all())
    assert bool((codes[:3] == 7).all()) and bool((codes[3 + n * d:] == 7).all())
    assert bool((scales[:1] == 9).all()) and bool((scales[1 + n * nb:] == 9).all())
