"""GPU checks of beam selection (lce_beam_select) over logits of any finite
size: tokens masked by value (the type's lowest number, -1e30, -1e10) that fill
whole pieces of a row, rows of nothing else, and large positive maxima.

The 64-bit form takes x - max first and then the logarithm of the sum, so that
the logarithm is not lost beside a large maximum: a row of V equal logits has
totals score - log V whatever the logits are.

Bounds: a score is one rounding to fp32 (2^-24 relatively) of score + (x - max)
- log(sum), where sum, at least 1, errs by less than 2^-18 relatively: a thread
adds 32 positive fp32 exponentials at most (31 roundings of 2^-24); each is off
by at most 2^-22 (the instruction) and by its argument, (x - max) log2 e, at
distance t = max - x: the difference's rounding, the constant's and the
product's, 3 times 2^-24 t at most, which is 3 2^-24 t exp(-t) <= 1.2 2^-24 of
the sum.  Together less than 2^-24 (31 + 4 + 2) < 2^-18; the rest is fp64."""
import numpy as np
import pytest
import torch

from lm_head_linear_amd import lce

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _want(x, scores, n_out, allowed=None):
    """(scores, parents, tokens) of the n_out best, in fp64."""
    n_seq, beams = scores.shape
    V = x.shape[1]
    S = np.full((n_seq, n_out), -np.inf)
    P = np.full((n_seq, n_out), -1, dtype=np.int64)
    T = np.full((n_seq, n_out), -1, dtype=np.int64)
    for q in range(n_seq):
        cands = []
        for k in range(beams):
            row = x[q * beams + k].copy()
            if allowed is not None:
                row[allowed[q * beams + k] == 0] = -np.inf
            top = row.max()
            if not np.isfinite(top):
                continue
            rest = row - top
            log_sum = np.log(np.exp(rest).sum())
            for i in np.argsort(-rest, kind="stable")[:n_out]:
                if rest[i] > -np.inf:
                    cands.append((-(float(scores[q, k]) + (rest[i] - log_sum)), k * V + int(i)))
        cands.sort()
        for j, (s, place) in enumerate(cands[:n_out]):
            S[q, j], P[q, j], T[q, j] = -s, place // V, place % V
    return S, P, T


def _check(x, scores, n_out, allowed=None):
    dev = _dev()
    S, P, T = _want(x.double().numpy(), scores.numpy(), n_out + 1,
                    None if allowed is None else allowed.numpy())
    with np.errstate(invalid="ignore"):
        gap = S[:, :-1] - S[:, 1:]
    assert ((P[:, :-1] == P[:, 1:]) | (gap == 0) | (gap > 2.0 ** -17) | ~np.isfinite(gap)).all()
    S, P, T = (a[:, :n_out] for a in (S, P, T))
    r = lce.beam_select(x.to(dev), scores.to(dev), n_out,
                        allowed=None if allowed is None else allowed.to(dev))
    got = r.scores.cpu().double().numpy()
    assert np.array_equal(r.parents.cpu().numpy(), P)
    assert np.array_equal(r.tokens.cpu().numpy(), T)
    fin = np.isfinite(S)
    assert np.array_equal(fin, np.isfinite(got))
    assert (np.abs(got[fin] - S[fin]) <= 2.0 ** -24 * np.abs(S[fin]) + 2.0 ** -18).all()


def _value(name, t):
    return torch.finfo(t).min if name == "lowest" else float(name)


MASKS = [("bf16", "-1e10"), ("bf16", "-5e9"), ("bf16", "-1e30"), ("bf16", "lowest"),
         ("f32", "-5e9"), ("f32", "-1e10"), ("f32", "-1e12"), ("f32", "-1e30"),
         ("f32", str(torch.finfo(torch.bfloat16).min)), ("f32", "lowest"), ("fp16", "lowest")]


@pytest.mark.parametrize("dt,mask", MASKS)
def test_pieces_masked_by_value(dt, mask):
    """Pieces in the middle and at the end of a row that hold the mask alone,
    a row masked to 1 % of its tokens, and ordinary rows beside them."""
    t = TYPES[dt]
    V, n_out = 13000, 12
    g = torch.Generator().manual_seed(V)
    x = (3 * torch.randn(8, V, generator=g)).to(t)
    v = _value(mask, t)
    x[0, 4096:8192] = v                                 # a piece of 4096
    x[1, 12288:] = v                                    # the row's tail
    x[2, :12500] = v                                    # all but the last tokens
    x[3, torch.rand(V, generator=g) < 0.99] = v
    x[5, :8192] = v
    x[5, 12288:] = v
    scores = -torch.rand(2, 4, generator=g)
    _check(x, scores, n_out)
    allowed = torch.rand(8, V, generator=g) < 0.5       # masked both ways
    allowed[0, 4096:8192] = True
    _check(x, scores, n_out, allowed)


@pytest.mark.parametrize("dt,mask", MASKS)
def test_rows_of_one_value(dt, mask):
    """Equal logits, whatever they are: every token has -log V, the lowest
    tokens are the best; with one token above them it is alone, and the masked
    ones follow in their order."""
    t = TYPES[dt]
    v = _value(mask, t)
    for V in (7, 4096, 9001, 40000):
        x = torch.full((3, V), v, dtype=t)
        x[1] = torch.linspace(-2.0, 2.0, V).to(t)
        _check(x, torch.tensor([[0.0], [-1.0], [-2.0]]), 5)
        _check(x, torch.tensor([[-0.5, 0.0, -1.0]]), 4)
        if mask != "-5e9":
            x[2, V - 2] = 1.5
            _check(x, torch.tensor([[0.0], [0.0], [-2.0]]), 6)


@pytest.mark.parametrize("dt,top", [("f32", 1e10), ("f32", 1e12), ("f32", 3e38), ("bf16", 1e12),
                                    ("bf16", 3e38), ("fp16", 65504.0)])
def test_large_positive_logits(dt, top):
    """A large maximum takes its beam's whole probability; rows of large equal
    values spread it."""
    t = TYPES[dt]
    V = 9000
    g = torch.Generator().manual_seed(3)
    x = (2 * torch.randn(6, V, generator=g)).to(t)
    x[1, 8500] = top
    x[2] = top
    x[4] = -top
    x[4, 5000:5003] = top
    _check(x, torch.tensor([[0.0, -1.0, -0.25], [-0.5, -0.75, -3.0]]), 3)


def test_long_rows_masked_by_value():
    """Pieces of 16384 tokens (many rows): 99 % of each row at the lowest
    number, some rows with whole pieces of it."""
    n_seq, beams, V, n_out = 105, 4, 40000, 8
    g = torch.Generator().manual_seed(9)
    for t in (torch.bfloat16, torch.float32):
        x = (3 * torch.randn(n_seq * beams, V, generator=g)).to(t)
        x[torch.rand(n_seq * beams, V, generator=g) < 0.99] = torch.finfo(t).min
        x[::3, 16384:] = torch.finfo(t).min
        x[1::7, :32768] = torch.finfo(t).min
        _check(x, -torch.rand(n_seq, beams, generator=g), n_out)


def test_totals_below_the_range_of_fp32():
    """A masked token chosen twice in a row passes fp32's range: its score is
    -inf, with the parent and the token it belongs to."""
    dev = _dev()
    lowest = torch.finfo(torch.float32).min
    x = torch.full((1, 9), lowest)
    x[0, 4] = 1.0
    r = lce.beam_select(x.to(dev), torch.tensor([[lowest]], device=dev), 3)
    assert r.tokens.tolist() == [[4, 0, 1]] and r.parents.tolist() == [[0, 0, 0]]
    assert r.scores.tolist() == [[lowest, -float("inf"), -float("inf")]]
