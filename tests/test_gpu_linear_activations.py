"""GPU checks of the activations' own error in lce_linear and their slopes' in
lce_linear_backward, with nothing else to round: a product of one term with the
factor 1 gives z exactly, outputs are fp32, and the slope shows unrounded in
the bias gradient of a single token whose d_out is 1.

Bounds in units of u = 2^-24, from the forms that are computed.  The hardware's
exp2 and reciprocal are off by at most 2 u relatively, a rounding by 1 u.

gelu: with t = 1 / (1 + c |z|), the normal tail is t P(t) exp(-z^2 / 2), P of
degree 7 with positive and negative coefficients: its fit is off by 1.6 u, its
evaluation by 3.6 u, t by 3 u (a rounding and the reciprocal), which counts up
to 3.4-fold; the exponential's argument by 2.2 u relatively, which is 1.1 z^2 u
of the exponential, itself off by 2 u; two products 2 u: (20 + 1.2 z^2) u of
the tail.  z * tail (or z * (1 - tail)) is one rounding more:
(21 + 1.2 z^2) u |gelu(z)| on the negative side and no more on the positive
one.  Its slope, cdf + z density: the density's exponential as above, three
roundings: (24 + 1.2 z^2) u (cdf + |z| density).

silu: the exponential's argument z log2 e is off by 1.3 u relatively (the
constant and a rounding), 1.3 |z| u of the exponential, itself off by 2 u; a
sum, a reciprocal and the product: (6 + 1.3 |z|) u |silu(z)|.  Its slope
s + z s (1 - s) adds two roundings of each term and 1 - s its own: (10 + 2 |z|) u
(s + |z| s).

Below, an absolute 2^-118 stands for results whose factors leave fp32's normal
range (tails beyond |z| = 13, exponentials beyond |z| = 87)."""
import math

import pytest
import torch

from lm_head_linear_amd import lce

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _values(t):
    """Every finite value of the type up to 100 in magnitude."""
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(t)
    v = v[torch.isfinite(v.float())]
    return v[v.float().abs() <= 100.0]


def _cdf(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _density(z):
    return torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)


def _within(got, want, tol):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float((off / tol).max()))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_values(act, dt):
    dev = _dev()
    t = TYPES[dt]
    v = _values(t).to(dev)
    one = torch.ones(1, 1, dtype=t, device=dev)
    got = lce.linear(v.view(-1, 1), one, activation=act, out_dtype=torch.float32).out.view(-1)
    z = v.double()
    if act == "gelu":
        want, rel = z * _cdf(z), 21 + 1.2 * z * z
    else:
        want, rel = z * torch.sigmoid(z), 6 + 1.3 * z.abs()
    _within(got, want, rel * U * want.abs() + 2.0 ** -118)
    # few tokens, the same values along a row
    got = lce.linear(one, v.view(-1, 1), activation=act, out_dtype=torch.float32).out.view(-1)
    _within(got, want, rel * U * want.abs() + 2.0 ** -118)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_slopes(act, dt):
    dev = _dev()
    t = TYPES[dt]
    v = _values(t).to(dev).view(1, -1)
    dy = torch.ones_like(v)
    w = torch.zeros(v.shape[1], 8, dtype=t, device=dev)
    got = lce.linear_backward(dy, None, w, v, activation=act, want_x=False, want_weight=False,
                              want_bias=True).d_bias
    z = v.double().view(-1)
    if act == "gelu":
        want = _cdf(z) + z * _density(z)
        tol = (24 + 1.2 * z * z) * U * (_cdf(z) + z.abs() * _density(z))
    else:
        s = torch.sigmoid(z)
        want = s * (1 + z * torch.sigmoid(-z))
        tol = (10 + 2 * z.abs()) * U * (s + z.abs() * s)
    _within(got, want, tol + 2.0 ** -118)
