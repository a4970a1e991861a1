"""Shapes that the allocating calls of the operators refuse, decided before the
device is looked at (CPU buffers): a tensor with enough elements in another
order would be read or written wrongly without a word."""
import pytest
import torch

from lm_head_linear_amd import lce

U8 = torch.uint8
N, D_IN, D_OUT = 6, 70, 40
T = torch.bfloat16


def _backward(**kw):
    x8 = lce.Packed8(torch.zeros(N, D_IN, dtype=U8), torch.zeros(N, 3, dtype=U8), T)
    z8 = lce.Packed8(torch.zeros(N, D_OUT, dtype=U8), torch.zeros(N, 2, dtype=U8), T)
    base = dict(d_out=torch.zeros(N, D_OUT, dtype=T), x=x8, weight=torch.zeros(D_OUT, D_IN, dtype=T),
                preact=z8, activation="gelu", want_bias=True)
    return lce.linear_backward(**{**base, **kw})


def test_backward_shapes_that_fit_reach_the_device_check():
    """What fits is only refused for not being on a GPU."""
    z = torch.zeros(N, D_OUT, dtype=T)
    for kw in ({}, {"preact": z}, {"x": torch.zeros(N, D_IN, dtype=T)},
               {"d_weight": torch.zeros(D_OUT, D_IN), "d_bias": torch.zeros(D_OUT)},
               {"d_bias": torch.zeros(1, D_OUT)},                       # one order only
               {"activation": "none", "preact": torch.zeros(1, 1, dtype=T)},   # not read
               {"want_weight": False, "d_weight": torch.zeros(1, 1)},   # not written
               {"want_bias": False, "d_bias": torch.zeros(1)}):
        with pytest.raises(ValueError, match="GPU"):
            _backward(**kw)


@pytest.mark.parametrize("shape", [(D_OUT, N), (N * D_OUT,), (N, D_OUT, 1), (N + 1, D_OUT),
                                   (N, D_OUT + 1), (1, N, D_OUT)])
def test_backward_preact_shape(shape):
    with pytest.raises(ValueError, match="preact"):
        _backward(preact=torch.zeros(shape, dtype=T))
    if len(shape) == 2:
        with pytest.raises(ValueError, match="preact"):
            _backward(preact=lce.Packed8(torch.zeros(shape, dtype=U8),
                                         torch.zeros(shape[0], (shape[1] + 31) // 32, dtype=U8), T))


@pytest.mark.parametrize("x_scales,z_scales", [((3, N), (N, 2)), ((N * 3,), (N, 2)), ((N, 4), (N, 2)),
                                               ((N + 1, 3), (N, 2)), ((N, 3), (2, N)),
                                               ((N, 3), (N, 3)), ((N, 3), (N * 2,))])
def test_backward_scales_shape(x_scales, z_scales):
    x8 = lce.Packed8(torch.zeros(N, D_IN, dtype=U8), torch.zeros(x_scales, dtype=U8), T)
    z8 = lce.Packed8(torch.zeros(N, D_OUT, dtype=U8), torch.zeros(z_scales, dtype=U8), T)
    with pytest.raises(ValueError, match="scales"):
        _backward(x=x8, preact=z8)


def test_backward_scales_that_are_not_read():
    """x without d_weight and preact without an activation take no part."""
    x8 = lce.Packed8(torch.zeros(N, D_IN, dtype=U8), torch.zeros(1, dtype=U8), T)
    with pytest.raises(ValueError, match="GPU"):
        _backward(x=x8, want_weight=False)
    z8 = lce.Packed8(torch.zeros(1, 1, dtype=U8), torch.zeros(1, dtype=U8), T)
    with pytest.raises(ValueError, match="GPU"):
        _backward(preact=z8, activation="none")


@pytest.mark.parametrize("shape", [(D_IN, D_OUT), (D_OUT * D_IN,), (D_OUT + 1, D_IN),
                                   (D_OUT, D_IN, 1)])
def test_backward_given_d_weight_shape(shape):
    for add in (False, True):
        with pytest.raises(ValueError, match="d_weight"):
            _backward(d_weight=torch.zeros(shape), d_bias=torch.zeros(D_OUT), accumulate=add)


@pytest.mark.parametrize("numel", [D_OUT - 1, D_OUT + 1, 2 * D_OUT])
def test_backward_given_d_bias_shape(numel):
    with pytest.raises(ValueError, match="d_bias"):
        _backward(d_bias=torch.zeros(numel))


def _select(**kw):
    base = dict(logits=torch.zeros(6, 50), scores=torch.zeros(2, 3), n_out=3, eos=1)
    return lce.beam_select(**{**base, **kw})


def test_select_shapes_that_fit_reach_the_device_check():
    for kw in ({"finished": torch.zeros(2, 3, dtype=U8)}, {"finished": torch.zeros(6, dtype=U8)},
               {"allowed": torch.ones(6, 50, dtype=U8)}, {"allowed": torch.ones(2, 3, 50, dtype=U8)}):
        with pytest.raises(ValueError, match="GPU"):
            _select(**kw)


@pytest.mark.parametrize("shape", [(3, 2), (5,), (7,), (6, 1), (1, 6), (2, 4), (2, 3, 1)])
def test_select_finished_shape(shape):
    with pytest.raises(ValueError, match="finished"):
        _select(finished=torch.zeros(shape, dtype=U8))


@pytest.mark.parametrize("shape", [(50, 6), (300,), (6, 51), (7, 50), (3, 2, 50), (2, 3, 51),
                                   (50, 2, 3), (2, 150), (50,)])
def test_select_allowed_shape(shape):
    with pytest.raises(ValueError, match="allowed"):
        _select(allowed=torch.ones(shape, dtype=U8))


@pytest.mark.parametrize("shape,fits", [((N, 3), True), ((3, N), False), ((N * 3,), False),
                                        ((N, 4), False), ((N + 1, 3), False), ((N, 3, 1), False)])
def test_unpack_scales_shape(shape, fits):
    p = lce.Packed8(torch.zeros(N, D_IN, dtype=U8), torch.zeros(shape, dtype=U8), T)
    with pytest.raises(ValueError, match="GPU" if fits else "scales"):
        lce.unpack8(p)


def test_backward_of_a_checkpoint_of_another_type():
    """A checkpoint of the other 16-bit type would be rounded and saturated to
    d_out's; the unpacked tensor of that type is refused, so it is too."""
    other = torch.float16
    x8 = lce.Packed8(torch.zeros(N, D_IN, dtype=U8), torch.zeros(N, 3, dtype=U8), other)
    z8 = lce.Packed8(torch.zeros(N, D_OUT, dtype=U8), torch.zeros(N, 2, dtype=U8), other)
    for kw in ({"x": x8}, {"preact": z8}, {"x": x8, "preact": z8, "activation": "relu"},
               {"d_out": torch.zeros(N, D_OUT, dtype=other), "weight": torch.zeros(D_OUT, D_IN, dtype=other)}):
        with pytest.raises(ValueError, match="checkpoint"):
            _backward(**kw)
    # not read: neither type matters
    for kw in ({"x": x8, "want_weight": False}, {"preact": z8, "activation": "none"}):
        with pytest.raises(ValueError, match="GPU"):
            _backward(**kw)
    with pytest.raises(ValueError, match="GPU"):
        _backward(x=x8, preact=z8, d_out=torch.zeros(N, D_OUT, dtype=other),
                  weight=torch.zeros(D_OUT, D_IN, dtype=other))
