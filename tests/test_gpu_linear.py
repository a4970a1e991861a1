"""GPU checks of lce_linear and lce_linear_backward against the 64-bit forms.

Bounds, element by element.  A product summed in fp32 in any order over K
terms errs by at most K 2^-23 sum |a b| (each addition rounds, possibly by
truncation, within 2^-23 of a partial sum that sum |a b| bounds; the products
of 16-bit factors are exact).  An activation passes that on at most 1.13-fold
(the largest slope of gelu; silu's is 1.10) and adds at most 2^-20 max(1, |z|)
of its own (fp32 erf, exp and division, a few ulp each).  A 16-bit result adds
half a step, eps/2 relatively, or for fp16 2^-25 absolutely; an fp32 result
2^-24.  In the backward g = dy act'(z): the slope errs by at most
2^-20 max(1, |z|) and g is rounded to 16 bits once, so a product with g errs by
the sum over |g's error| |b| besides its own summation."""
import pytest
import torch

from lm_head_linear_amd import lce
from tests import ops_plain

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _half(dt):
    return torch.finfo(dt).eps / 2, (2.0 ** -25 if dt == torch.float16 else 0.0)


def _round(y, err, dt):
    """The error of rounding a value that is y but for err to dt."""
    if dt == torch.float32:
        return err + 2.0 ** -24 * (y.abs() + err)
    rel, small = _half(dt)
    return err + rel * (y.abs() + err) + small


def _within(got, want, tol):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist(), float(off[bad].max()))


def _d(a):
    return None if a is None else a.double()


def _inputs(n, d_in, d_out, dt, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return (r(n, d_in).to(dt), (r(d_out, d_in) / d_in ** 0.5).to(dt), r(d_out), r(n, d_out).to(dt),
            (0.1 * r(n, d_out)).to(dt))


def _check_forward(x, w, b, r, act, preact, out_dt, result=None):
    X, W, B, R = _d(x), _d(w), _d(b), _d(r)
    y, z = ops_plain.linear(X, W, B, R, act)
    res = result or lce.linear(x, w, b, r, activation=act, want_preact=preact, out_dtype=out_dt)
    size = X.abs() @ W.abs().T + (0 if B is None else B.abs())
    e = (x.shape[1] + 1) * 2.0 ** -23 * size
    if preact:
        _within(res.preact, z, _round(z, e, x.dtype))
    ey = 1.13 * e
    if act in ("gelu", "silu"):
        ey = ey + 2.0 ** -20 * z.abs().clamp(min=1.0)
    if R is not None:
        ey = ey + 2.0 ** -23 * (y.abs() + R.abs())
    _within(res.out, y, _round(y, ey, out_dt))
    return res


SIZES = [(1, 1, 1), (1, 1024, 1024), (2, 7, 5), (3, 8, 16), (5, 64, 260), (16, 72, 129),
         (17, 128, 64), (33, 100, 300), (64, 1000, 513), (65, 256, 40), (130, 1003, 77),
         (257, 192, 130), (300, 520, 264), (513, 65, 520), (31, 4104, 24), (4, 8200, 96)]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n,d_in,d_out", SIZES)
def test_forward(n, d_in, d_out, dt):
    dev = _dev()
    t = TYPES[dt]
    x, w, b, r, _ = (a.to(dev) for a in _inputs(n, d_in, d_out, t, n + d_in + d_out))
    for i, act in enumerate(ops_plain.ACTS):
        print(f"case linear {n}x{d_in}->{d_out} {dt} {act}", flush=True)
        _check_forward(x, w, b if i != 1 else None, r if i % 2 else None, act, i in (0, 2),
                       torch.float32 if i >= 2 else t)
    _check_forward(x, w, b.to(t), r, "gelu", True, t)


def _check_backward(dy, x, w, z, act, grads, x_values=None, z_values=None):
    DY, W = _d(dy), _d(w)
    X, Z = _d(x_values if x_values is not None else x), None
    if act != "none":
        Z = _d(z_values if z_values is not None else z)
    dx, dw, db, g = ops_plain.linear_backward(DY, X, W, Z, act)
    eg = torch.zeros_like(g)
    if act in ("gelu", "silu"):
        eg = DY.abs() * 2.0 ** -20 * Z.abs().clamp(min=1.0) + 2.0 ** -24 * g.abs()
    er = eg if act == "none" else _round(g, eg, dy.dtype)
    n, m = g.shape
    size = g.abs() + er
    if grads.d_x is not None:
        _within(grads.d_x, dx, _round(dx, er @ W.abs() + m * 2.0 ** -23 * (size @ W.abs()),
                                      dy.dtype))
    if grads.d_weight is not None:
        _within(grads.d_weight, dw,
                _round(dw, er.T @ X.abs() + n * 2.0 ** -23 * (size.T @ X.abs()),
                       grads.d_weight.dtype))
    if grads.d_bias is not None:
        _within(grads.d_bias, db, _round(db, eg.sum(0) + n * 2.0 ** -23 * size.sum(0),
                                         grads.d_bias.dtype))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n,d_in,d_out", SIZES)
def test_backward(n, d_in, d_out, dt):
    dev = _dev()
    t = TYPES[dt]
    x, w, _, z, dy = (a.to(dev) for a in _inputs(n, d_in, d_out, t, n + d_in + d_out))
    for i, act in enumerate(ops_plain.ACTS):
        print(f"case linear backward {n}x{d_in}->{d_out} {dt} {act}", flush=True)
        g = lce.linear_backward(dy, x, w, z, activation=act, want_bias=i != 1,
                                weight_grad_dtype=t if i % 2 else None)
        assert g.d_weight.dtype == (t if i % 2 else torch.float32)
        _check_backward(dy, x, w, z, act, g)
        x8, z8 = lce.pack8(x), lce.pack8(z)
        g = lce.linear_backward(dy, x8, w, z8 if i != 3 else z, activation=act, want_bias=True)
        _check_backward(dy, x, w, z, act, g, lce.unpack8(x8), lce.unpack8(z8) if i != 3 else z)


def test_some_gradients_only():
    dev = _dev()
    t = torch.bfloat16
    x, w, _, z, dy = (a.to(dev) for a in _inputs(70, 96, 130, t, 5))
    full = lce.linear_backward(dy, x, w, z, activation="gelu", want_bias=True)
    a = lce.linear_backward(dy, None, w, z, activation="gelu", want_weight=False)
    b = lce.linear_backward(dy, x, None, z, activation="gelu", want_x=False)
    c = lce.linear_backward(dy, x, w, z, activation="gelu", want_x=False, want_weight=False,
                            want_bias=True)
    assert torch.equal(a.d_x, full.d_x) and a.d_weight is None and a.d_bias is None
    assert torch.equal(b.d_weight, full.d_weight) and b.d_x is None
    assert c.d_x is None and c.d_weight is None       # (its sums may run in another order)
    _check_backward(dy, x, w, z, "gelu", c)


@pytest.mark.parametrize("wdt", ["f32", "bf16"])
@pytest.mark.parametrize("n,d_in,d_out", [(40, 64, 100), (300, 520, 264), (33, 77, 19)])
def test_accumulation(n, d_in, d_out, wdt):
    """accumulate adds the gradient to what is there: one rounding of the sum
    (fp32: 2^-24, bf16: 2^-8 relatively) on top of the fresh gradient."""
    dev = _dev()
    t = torch.bfloat16
    wt = torch.float32 if wdt == "f32" else t
    x, w, _, z, dy = (a.to(dev) for a in _inputs(n, d_in, d_out, t, 6))
    g = torch.Generator().manual_seed(7)
    w0 = torch.randn(d_out, d_in, generator=g).to(wt).to(dev)
    b0 = torch.randn(d_out, generator=g).to(dev)
    fresh = lce.linear_backward(dy, x, w, z, activation="silu", want_bias=True)   # fp32
    dw, db = w0.clone(), b0.clone()
    lce.linear_backward(dy, x, w, z, activation="silu", want_bias=True, d_weight=dw, d_bias=db,
                        accumulate=True)
    half = 2.0 ** -24 if wdt == "f32" else 2.0 ** -8
    want = w0.double() + fresh.d_weight.double()
    assert bool(((dw.double() - want).abs() <= half * want.abs() * (1 + half)).all())
    want = b0.double() + fresh.d_bias.double()
    assert bool(((db.double() - want).abs() <= 2.0 ** -24 * want.abs() * 1.001).all())


@pytest.mark.parametrize("act", ["gelu", "silu", "none"])
def test_gradients_against_differences(act):
    """d/dh of sum(c * linear) along random directions, by central differences
    of the 64-bit form (step 1e-4: truncation about 1e-8 of the third
    derivative), against the kernel's gradients dotted with the direction.
    The kernel's gradients err by their rounding (2^-8 of each term for bf16:
    g, and the 16-bit d_x), summed over |direction|."""
    dev = _dev()
    n, d_in, d_out = 37, 72, 50
    t = torch.bfloat16
    x, w, b, _, c = _inputs(n, d_in, d_out, t, 11)
    X, W, B, C = (a.double() for a in (x, w, b, c))
    z = lce.linear(x.to(dev), w.to(dev), b.to(dev), activation=act, out_dtype=torch.float32,
                   want_preact=True).preact
    # the slope is taken at the stored (rounded) z: shift the bias to match it
    shift = z.double().cpu() - (X @ W.T + B)
    g = lce.linear_backward(c.to(dev), x.to(dev), w.to(dev), z, activation=act, want_bias=True)
    f = lambda X_, W_, B_: float((C * ops_plain.act(X_ @ W_.T + B_ + shift, act)).sum())
    G = C.abs() * 1.2
    gen = torch.Generator().manual_seed(12)
    h = 1e-4
    for _ in range(3):
        for got, at, size in ((g.d_x, 0, G @ W.abs()), (g.d_weight, 1, G.T @ X.abs()),
                              (g.d_bias, 2, G.sum(0))):
            args = [X, W, B]
            v = torch.randn(args[at].shape, generator=gen, dtype=torch.float64)
            hi, lo = list(args), list(args)
            hi[at], lo[at] = args[at] + h * v, args[at] - h * v
            want = (f(*hi) - f(*lo)) / (2 * h)
            tol = 2 * 2.0 ** -8 * float((size * v.abs()).sum()) + 1e-5
            assert abs(float((got.double().cpu() * v).sum()) - want) <= tol


def test_non_finite_values_stay_in_their_rows():
    dev = _dev()
    t = torch.bfloat16
    for n, d_in, d_out in ((20, 72, 96), (300, 264, 136)):
        x, w, b, r, _ = (a.to(dev) for a in _inputs(n, d_in, d_out, t, 13))
        clean = lce.linear(x, w, b, r, activation="gelu").out
        x2 = x.clone()
        x2[3, 5], x2[7, d_in - 1] = float("nan"), float("inf")
        got = lce.linear(x2, w, b, r, activation="gelu").out
        keep = torch.ones(n, dtype=torch.bool, device=dev)
        keep[3] = keep[7] = False
        assert torch.equal(got[keep], clean[keep])
        assert bool(got[3].isnan().all())


def test_views_in_place_residual_and_neighbours():
    """Bases at odd offsets; the residual may be the output; what lies around
    the outputs stays."""
    dev = _dev()
    n, d_in, d_out = 45, 104, 88
    t = torch.float16
    x, w, b, r, dy = (a.to(dev) for a in _inputs(n, d_in, d_out, t, 15))
    off = lambda a, k: torch.cat([a.new_zeros(k), a.reshape(-1)])[k:].view(a.shape)
    ws = torch.empty(lce.lce_linear_workspace_bytes(n, d_in, d_out, t), dtype=torch.uint8, device=dev)
    for k in (0, 1, 3, 4):
        xo, wo, bo, ro = off(x, k), off(w, k + 1), off(b, k), off(r, k)
        buf = torch.full((n * d_out + 16,), 2.0, dtype=t, device=dev)
        out = buf[k + 2: k + 2 + n * d_out].view(n, d_out)
        assert lce.lce_linear(xo, wo, bo, ro, n, d_in, d_out, 2, None, out, ws) == 580
        _check_forward(xo, wo, bo, ro, "gelu", False, t, lce.LinearResult(out, None))
        assert bool((buf[:k + 2] == 2).all()) and bool((buf[k + 2 + n * d_out:] == 2).all())
        same = ro.clone()
        assert lce.lce_linear(xo, wo, bo, same, n, d_in, d_out, 2, None, same, ws) == 580
        assert torch.equal(same, out)
        g = lce.linear_backward(off(dy, k), xo, wo, ro, activation="silu", want_bias=True)
        _check_backward(dy, x, w, r, "silu", g)


def test_same_bits_every_time():
    dev = _dev()
    for n, d_in, d_out in ((2, 4096, 96), (200, 2048, 136), (600, 520, 1000)):
        x, w, b, r, dy = (a.to(dev) for a in _inputs(n, d_in, d_out, torch.bfloat16, 17))
        first = lce.linear(x, w, b, r, activation="gelu", want_preact=True)
        g1 = lce.linear_backward(dy, x, w, r, activation="gelu", want_bias=True)
        for _ in range(3):
            again = lce.linear(x, w, b, r, activation="gelu", want_preact=True)
            g2 = lce.linear_backward(dy, x, w, r, activation="gelu", want_bias=True)
            assert torch.equal(again.out, first.out) and torch.equal(again.preact, first.preact)
            for k in ("d_x", "d_weight", "d_bias"):
                assert torch.equal(getattr(g1, k), getattr(g2, k)), k


@pytest.mark.parametrize("n,d_in,d_out,act,dt", [
    (20, 1024, 40000, "none", "bf16"),      # 128 x 32 tiles
    (60, 1000, 40000, "silu", "fp16"),      # 128 x 64 tiles, an odd depth
    (100, 8192, 72, "gelu", "bf16"),        # 64 x 64 tiles, the depth in 16 parts
    (700, 512, 3000, "relu", "fp16"),       # 128 x 128 tiles
    (777, 1003, 1531, "silu", "fp16"),      # padded copies of odd rows
    (515, 1002, 777, "gelu", "bf16"),       # odd rows read as they lie
    (4096, 512, 4096, "gelu", "bf16"),      # 256 x 256 tiles
    (3000, 2601, 5300, "gelu", "fp16"),     # 256 x 256 tiles of padded copies
    (130, 40, 20001, "none", "bf16")])
def test_forward_on_every_core(n, d_in, d_out, act, dt):
    dev = _dev()
    t = TYPES[dt]
    print(f"case linear {n}x{d_in}->{d_out} {dt} {act}", flush=True)
    x, w, b, r, _ = (a.to(dev) for a in _inputs(n, d_in, d_out, t, 21))
    _check_forward(x, w, b, r, act, True, t)
    _check_forward(x, w, None, None, act, False, torch.float32)


@pytest.mark.parametrize("n,d_in,d_out,act,dt", [
    (5000, 72, 120, "silu", "bf16"),        # d_weight's depth in 16 parts
    (515, 1003, 777, "silu", "fp16"),       # both products in one launch
    (2100, 512, 1900, "gelu", "bf16"),
    (8200, 1032, 4100, "gelu", "bf16"),     # 256 x 256 tiles, d_weight in 2 parts
    (4100, 2056, 4224, "none", "fp16"),     # the same without copies of d_out_grad
    (250, 65536, 1000, "relu", "bf16")])    # d_x from the weight as it lies
def test_backward_on_every_core(n, d_in, d_out, act, dt):
    dev = _dev()
    t = TYPES[dt]
    print(f"case linear backward {n}x{d_in}->{d_out} {dt} {act}", flush=True)
    x, w, _, z, dy = (a.to(dev) for a in _inputs(n, d_in, d_out, t, 22))
    g = lce.linear_backward(dy, x, w, z, activation=act, want_bias=True)
    _check_backward(dy, x, w, z, act, g)
    x8, z8 = lce.pack8(x), lce.pack8(z)
    g = lce.linear_backward(dy, x8, w, z8, activation=act, weight_grad_dtype=t)
    _check_backward(dy, x, w, z, act, g, lce.unpack8(x8), lce.unpack8(z8))
    g = lce.linear_backward(dy, None, w, z, activation=act, want_weight=False)
    _check_backward(dy, x, w, z, act, g)


@pytest.mark.parametrize("n,d_in,d_out", [(3, 16, (1 << 22) + 100), ((1 << 22) + 100, 8, 24)])
def test_backward_of_very_long_dimensions(n, d_in, d_out):
    """Rows and depths whose 256-fold byte offsets pass 31 bits."""
    dev = _dev()
    t = torch.bfloat16
    x, w, _, z, dy = (a.to(dev) for a in _inputs(n, d_in, d_out, t, 26))
    g = lce.linear_backward(dy, x, w, z, activation="relu", want_bias=True)
    _check_backward(dy, x, w, z, "relu", g)


def test_more_than_32_bits_of_outputs():
    """2^32 outputs and more: the last rows and columns are where they belong."""
    dev = _dev()
    n, d_in, d_out = 8200, 16, 1 << 19
    x, w, b, _, _ = (a.to(dev) for a in _inputs(1, d_in, d_out, torch.bfloat16, 23))
    x = torch.randn(n, d_in, generator=torch.Generator().manual_seed(24)).bfloat16().to(dev)
    out = lce.linear(x, w, b, activation="relu").out
    for rows in (slice(0, 2), slice(4095, 4098), slice(n - 2, n)):
        _check_forward(x[rows], w, b, None, "relu", False, torch.bfloat16,
                       lce.LinearResult(out[rows], None))


def test_views_that_are_not_aligned_on_the_large_cores():
    dev = _dev()
    t = torch.bfloat16
    off = lambda a, k: torch.cat([a.new_zeros(k), a.reshape(-1)])[k:].view(a.shape)
    for n, d_in, d_out in ((4096, 512, 4096), (700, 512, 3000), (20, 1024, 40000)):
        x, w, b, r, dy = (a.to(dev) for a in _inputs(n, d_in, d_out, t, 25))
        _check_forward(off(x, 1), off(w, 3), b, off(r, 1), "gelu", True, t)
        g = lce.linear_backward(off(dy, 1), off(x, 1), off(w, 1), off(r, 3), activation="gelu",
                                want_bias=True)
        _check_backward(dy, x, w, r, "gelu", g)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_activations_at_the_ends(dt):
    """Large, tiny and infinite pre-activations: what the formulas give in fp32."""
    dev = _dev()
    t = TYPES[dt]
    v = torch.tensor([0.0, -0.0, 1e-4, -1e-4, 0.5, -0.5, 3.0, -3.0, 6.0, -6.0, 12.0, -12.0, 80.0,
                      -80.0, 1e4, -1e4, 6e4, -6e4]).to(t)
    x = v.view(-1, 1).to(dev)
    w = torch.ones(1, 1, dtype=t, device=dev)
    for act in ops_plain.ACTS:
        _check_forward(x, w, None, None, act, True, t)
        dy = torch.full_like(x, 0.5)
        _check_backward(dy, x, w, x, act, lce.linear_backward(dy, x, w, x, activation=act))
    inf = torch.tensor([[float("inf")], [-float("inf")], [float("nan")]], dtype=t, device=dev)
    got = lce.linear(inf, w, activation="relu").out.view(-1)
    assert got[0] == float("inf") and got[1] == 0 and bool(got[2].isnan())
    got = lce.linear(inf, w, activation="gelu").out.view(-1)
    assert got[0] == float("inf") and bool(got[2].isnan())
