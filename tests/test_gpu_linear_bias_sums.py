"""GPU checks of the bias gradient's sum over many tokens.  The inputs are sums
whose exact value fp32 holds, but not every partial sum of it: 64 tokens that
add up to 2^24 units and a few units in every later 64, each of which an fp32
sum past 2^24 would drop.  Groups of 64 tokens are exact in fp32 and their sum
is exact in fp64, so the result has to be equal to the exact one."""
import pytest
import torch

from lm_head_linear_amd import lce

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _grads(n, d_out, t, seed):
    """(dy, its exact column sums in units of `unit`)."""
    unit = 1.0 if t == torch.bfloat16 else 2.0 ** -6       # 2^18 units fit the type
    dy = torch.zeros(n, d_out, dtype=t)
    first = 64 * (seed % (n // 64))
    dy[first:first + 64] = 2.0 ** 18 * unit
    for group in range(n // 64):
        if 64 * group != first:
            dy[64 * group + (7 * group + seed) % 64] = unit
            dy[64 * group + (7 * group + seed) % 64, ::3] = 3 * unit
    sums = dy.double().sum(0)
    assert bool((sums == sums.float().double()).all())
    return dy, sums


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n,d_in,d_out", [(64 * 257, 64, 96),        # one launch with small tiles
                                          (64 * 129, 1032, 4100),    # with the 256 x 256 core
                                          (64 * 1025, 8, 130)])
def test_sums_over_many_tokens(n, d_in, d_out, dt):
    dev = _dev()
    t = TYPES[dt]
    print(f"case bias sums {n}x{d_in}->{d_out} {dt}", flush=True)
    x = torch.zeros(n, d_in, dtype=t, device=dev)
    w = torch.zeros(d_out, d_in, dtype=t, device=dev)
    z = torch.ones(n, d_out, dtype=t, device=dev)
    for seed in (0, 5, n // 64 - 1):
        dy, sums = _grads(n, d_out, t, seed)
        dy = dy.to(dev)
        want = sums.float().to(dev)
        for act in ("none", "relu"):
            both = lce.linear_backward(dy, x, w, z, activation=act, want_bias=True)
            assert torch.equal(both.d_bias, want)
            alone = lce.linear_backward(dy, x, w, z, activation=act, want_x=False, want_weight=False,
                                        want_bias=True)
            assert torch.equal(alone.d_bias, want)
        # added to what is there: the gradient's fp32 value, one rounding more
        b0 = torch.linspace(-3.0, 3.0, d_out, device=dev)
        got = b0.clone()
        lce.linear_backward(dy, x, w, z, want_x=False, want_weight=False, want_bias=True, d_bias=got,
                            accumulate=True)
        assert torch.equal(got, b0 + want)
        if t == torch.bfloat16:
            small = torch.empty(d_out, dtype=t, device=dev)
            lce.linear_backward(dy, x, w, z, want_x=False, want_weight=False, want_bias=True,
                                d_bias=small)
            assert torch.equal(small, want.to(t))
