"""GPU checks of lce_linear_backward where 256 rows' byte offsets pass 31 bits,
with inputs of -1, 0 and 1: every partial sum of at most 2^22 + 100 such
products is a whole number below 2^24, exact in fp32 in any order, so results
have to equal the 64-bit form rounded once.  That a lost depth split, a lost
end or zeros would show is asserted on the expected values."""
import pytest
import torch

from lm_head_linear_amd import lce

pytestmark = pytest.mark.gpu
LONG = (1 << 22) + 100
SPLIT = -(-LONG // 16 // 64) * 64       # depths of one of 16 parts of a long sum, in steps of 64


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _signs(g, *shape):
    return torch.randint(-1, 2, shape, generator=g).to(torch.bfloat16)


def _ends(long):
    """Places where a long sum could lose something: both sides of every
    boundary of 16 parts and of the last steps of 64, and the ends."""
    at = {0, 1, 63, 64, long - 1, long - 2, long - 37, long - 63, long - 64, long - 65, long - 101}
    for part in range(1, 16):
        at |= {part * SPLIT - 1, part * SPLIT, part * SPLIT - 64, part * SPLIT + 63}
    return sorted(a for a in at if 0 <= a < long)


def _exact(dy, x, w, z):
    g = dy.double() * (z > 0)
    return g @ w.double(), g.t().contiguous() @ x.double(), g.sum(0)


def _equal(got, want):
    assert torch.equal(got.double(), want.to(got.dtype).double())


def _check(dy, x, w, z):
    dx, dw, db = _exact(dy, x, w, z)
    for x_, z_ in ((x, z), (lce.pack8(x), lce.pack8(z))):
        r = lce.linear_backward(dy, x_, w, z_, activation="relu", want_bias=True)
        _equal(r.d_x, dx)
        _equal(r.d_weight, dw)
        _equal(r.d_bias, db)


@pytest.mark.parametrize("dense", [True, False])
def test_long_rows(dense):
    """d_x sums over 2^22 + 100 outputs."""
    dev = _dev()
    n, d_in = 3, 16
    g = torch.Generator().manual_seed(31)
    x, z = _signs(g, n, d_in).to(dev), _signs(g, n, LONG).to(dev)
    w = _signs(g, LONG, d_in).to(dev)
    dy = _signs(g, n, LONG).to(dev)
    if not dense:                       # few enough that d_x is exact in 16 bits
        at = torch.tensor(_ends(LONG), device=dev)
        some = torch.zeros_like(dy)
        some[:, at] = 1
        z[:, at] = 1
        w[at] = torch.where(w[at] == 0, 1, w[at])
        dy = some
        full = _exact(dy, x, w, z)[0]
        assert bool((full.abs() <= 256).all())
        for i in at.tolist():           # any of them missing would show
            less = dy.clone()
            less[:, i] = 0
            assert bool((_exact(less[:, i:i + 1], x, w[i:i + 1], z[:, i:i + 1])[0] == 0).all())
            assert bool((w[i].double().abs() == 1).all())
    else:
        full = _exact(dy, x, w, z)[0].to(torch.bfloat16)
        less = dy.clone()
        less[:, 5 * SPLIT:6 * SPLIT] = 0
        assert not torch.equal(full, _exact(less, x, w, z)[0].to(torch.bfloat16))
        assert bool(full.any())
    _check(dy, x, w, z)


@pytest.mark.parametrize("dense", [True, False])
def test_many_tokens(dense):
    """d_weight and d_bias sum over 2^22 + 100 tokens."""
    dev = _dev()
    d_in, d_out = 8, 24
    g = torch.Generator().manual_seed(32)
    x, z = _signs(g, LONG, d_in).to(dev), _signs(g, LONG, d_out).to(dev)
    w = _signs(g, d_out, d_in).to(dev)
    dy = _signs(g, LONG, d_out).to(dev)
    at = torch.tensor(_ends(LONG), device=dev)
    if not dense:
        some = torch.zeros_like(dy)
        some[at] = 1
        dy = some
    z[at] = 1
    x[at] = torch.where(x[at] == 0, 1, x[at])
    dy[at] = torch.where(dy[at] == 0, 1, dy[at])
    _, dw, db = _exact(dy, x, w, z)
    assert bool((dw.abs() < 2 ** 24).all()) and bool(dw.any()) and bool(db.any())
    # every place adds a whole number that is not 0 to every sum, and fp32 holds
    # the sums: any place missing would show
    assert bool((dy[at].double().abs() == 1).all()) and bool((x[at].double().abs() == 1).all())
    _check(dy, x, w, z)
