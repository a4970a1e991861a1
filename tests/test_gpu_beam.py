"""GPU checks of the beam step (lce_beam_select, lce_beam_reorder).

Parents, tokens and flags are whole numbers and have to equal the 64-bit
form's; a score is one rounding to fp32 of score + logit - lse.  The kernel's
lse: a thread adds 32 positive fp32 exponentials (31 roundings of 2^-24), each
off by at most 2^-22 (the instruction) and by its argument's two roundings
(2^-23 t exp(-t) <= 2^-24 at distance t from the maximum); the rest is fp64.
Together less than 2^-24 (31 + 4 + 1) < 2^-18 relatively in the sum, so
absolutely in lse.  The order across beams is only asked for where the 64-bit
totals differ by more than twice that, or are equal."""
import numpy as np
import pytest
import torch

from lm_head_linear_amd import lce
from tests import ops_plain

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _run(x, scores, n_out, finished=None, allowed=None, eos=None):
    dev = _dev()
    to = lambda a: None if a is None else a.to(dev)
    return lce.beam_select(to(x), to(scores), n_out, to(finished), to(allowed), eos)


def _check(x, scores, n_out, finished=None, allowed=None, eos=None):
    np_ = lambda a: None if a is None else a.numpy()
    S, P, T, F = ops_plain.beam_select(x.double().numpy(), scores.numpy(), n_out + 1,
                                       np_(finished), np_(allowed), -1 if eos is None else eos)
    with np.errstate(invalid="ignore"):
        gap = S[:, :-1] - S[:, 1:]
    assert ((P[:, :-1] == P[:, 1:]) | (gap == 0) | (gap > 2.0 ** -17) | ~np.isfinite(gap)).all()
    S, P, T, F = (a[:, :n_out] for a in (S, P, T, F))
    r = _run(x, scores, n_out, finished, allowed, eos)
    got = r.scores.cpu().double().numpy()
    assert np.array_equal(r.parents.cpu().numpy(), P)
    assert np.array_equal(r.tokens.cpu().numpy(), T)
    assert np.array_equal(r.finished.cpu().numpy(), F)
    fin = np.isfinite(S)
    assert np.array_equal(fin, np.isfinite(got))
    assert (np.abs(got[fin] - S[fin]) <= 2.0 ** -24 * np.abs(S[fin]) + 2.0 ** -18).all()
    return r


@pytest.mark.parametrize("dt", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("n_seq,beams,V,n_out", [(1, 1, 1, 1), (1, 1, 7, 4), (2, 3, 5, 6),
                                                 (1, 4, 1000, 8), (3, 8, 8192, 16),
                                                 (2, 5, 8193, 10), (1, 16, 20011, 32),
                                                 (1, 32, 8190, 64), (2, 2, 100003, 1),
                                                 (5, 1, 333, 64)])
def test_select(n_seq, beams, V, n_out, dt):
    print(f"case select {n_seq}x{beams}x{V} -> {n_out} {dt}", flush=True)
    g = torch.Generator().manual_seed(n_seq * 1000 + beams + V)
    x = (3 * torch.randn(n_seq * beams, V, generator=g)).to(TYPES[dt])
    scores = -5 * torch.rand(n_seq, beams, generator=g)
    _check(x, scores, n_out)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [50, 9001])
def test_finished_beams_and_masks(V, dt):
    g = torch.Generator().manual_seed(V)
    n_seq, beams, n_out = 4, 6, 12
    x = (2 * torch.randn(n_seq * beams, V, generator=g)).to(TYPES[dt])
    scores = -5 * torch.rand(n_seq, beams, generator=g)
    finished = torch.rand(n_seq, beams, generator=g) < 0.4
    finished[3] = True                                  # a sequence that is done
    share = torch.rand(n_seq * beams, 1, generator=g) ** 3
    share[::5] = 0.0                                    # rows without any token
    allowed = torch.rand(n_seq * beams, V, generator=g) < share
    # what is masked does not count, whatever it is
    x = torch.where(allowed | (torch.rand(x.shape, generator=g) < 0.5), x,
                    torch.full((), float("nan"), dtype=x.dtype))
    x[7][~allowed[7]] = float("inf")
    _check(x, scores, n_out, finished, allowed.to(torch.uint8), eos=V - 1)
    _check(x, scores, n_out, finished.to(torch.uint8), allowed, eos=0)


def test_ties_go_to_the_lowest_place():
    V = 9000
    x = torch.zeros(6, V)
    scores = torch.tensor([[0.0, 0.0, 0.0], [-1.0, 0.0, 0.0]])
    _check(x, scores, 7)                                # all equal: long ties in every piece
    x[:, 100:130] = 1.0
    _check(x, scores, 40)
    x[1, 5], x[1, 6] = -0.0, 0.0
    _check(x.half(), scores, 64)
    same = torch.randn(1, V, generator=torch.Generator().manual_seed(1)).repeat(6, 1).bfloat16()
    _check(same, torch.zeros(2, 3), 9)                  # equal beams


def test_many_values_at_the_cut():
    """One thread's values fill the list: the cut is found by bisection."""
    V = 8192
    x = torch.full((2, V), -50.0)
    x[0] = 4.0                                          # 8192 equal values
    x[1, : V // 2] = 3.0
    x[1, V // 2:] = torch.linspace(3.0, 3.5, V // 2)
    for n_out in (1, 5, 64):
        _check(x, torch.tensor([[0.0, -0.25]]), n_out)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_offer_nothing(value):
    V = 12000
    x = torch.randn(4, V, generator=torch.Generator().manual_seed(2))
    if value == -float("inf"):
        x[1] = value
        x[2, 1:] = value                                # one token left
    else:
        x[1, 8500] = value
    _check(x, torch.tensor([[0.0, 0.0, -0.5, 0.0]]), 8)
    # scores that are not finite
    for bad in (float("nan"), float("inf"), -float("inf")):
        _check(torch.randn(4, 40, generator=torch.Generator().manual_seed(3)),
               torch.tensor([[0.0, bad], [bad, bad]]), 5, torch.tensor([[0, 0], [0, 1]]).bool(),
               eos=3)


def test_first_step_has_one_live_beam():
    x = torch.randn(1, 500, generator=torch.Generator().manual_seed(4)).repeat(4, 1).half()
    _check(x, torch.tensor([[0.0] + [-float("inf")] * 3]), 4)


def test_views_and_repeats():
    """An unaligned base, one workspace for calls in a row, every call the same."""
    dev = _dev()
    V, rows = 4099, 6
    flat = (3 * torch.randn(rows * V + 3, generator=torch.Generator().manual_seed(6))).bfloat16()
    x = flat[3:].view(rows, V)
    scores = -torch.rand(2, 3, generator=torch.Generator().manual_seed(7))
    want = _check(x.clone(), scores, 6)
    ws = torch.empty(lce.lce_beam_workspace_bytes(2, 3, V, 64), dtype=torch.uint8, device=dev)
    xd = flat.to(dev)[3:].view(rows, V)
    for _ in range(3):
        r = lce.beam_select(xd, scores.to(dev), 6, workspace=ws)
        for a in ("scores", "parents", "tokens"):
            assert torch.equal(getattr(r, a), getattr(want, a))
        lce.beam_select(xd * 2, scores.to(dev), 64, workspace=ws)


# ---------------------------------------------------------------- reordering

def _reordered(x, parents, beams):
    n_seq, n_out = parents.shape
    out = torch.zeros(n_seq * n_out, *x.shape[1:], dtype=x.dtype)
    for q in range(n_seq):
        for j in range(n_out):
            k = int(parents[q, j])
            if 0 <= k < beams:
                out[q * n_out + j] = x[q * beams + k]
    return out


@pytest.mark.parametrize("n_seq,beams,n_out", [(1, 1, 1), (3, 4, 4), (2, 8, 3), (1, 3, 20),
                                               (2, 32, 32), (5, 2, 9)])
@pytest.mark.parametrize("shape,dt", [((7,), torch.int64), ((3, 5, 8), torch.bfloat16),
                                      ((2, 9, 5), torch.float16), ((1, 1, 1), torch.uint8),
                                      ((2, 300, 16), torch.float32), ((3, 11, 7), torch.uint8)])
def test_reorder(n_seq, beams, n_out, shape, dt):
    dev = _dev()
    g = torch.Generator().manual_seed(beams * 100 + n_out)
    xs = [torch.randint(0, 200, (n_seq * beams, *shape), generator=g).to(dt) for _ in range(3)]
    parents = torch.randint(0, beams, (n_seq, n_out), generator=g)
    if n_out > 1:
        parents[0, 1] = -1
    into = [torch.full((n_seq * n_out, *shape), 3, dtype=dt, device=dev) for _ in xs]
    got = lce.beam_reorder([x.to(dev) for x in xs], parents.to(dev), beams, out=into)
    for x, y in zip(xs, got):
        assert torch.equal(y.cpu(), _reordered(x, parents, beams))
    if n_out == beams:
        own = [x.to(dev) for x in xs]
        lce.beam_reorder(own, parents.to(dev), beams)
        for x, y in zip(xs, own):
            assert torch.equal(y.cpu(), _reordered(x, parents, beams))


@pytest.mark.parametrize("length", [0, 1, 13, 64])
@pytest.mark.parametrize("in_place", [False, True])
def test_reorder_of_filled_caches(length, in_place):
    """Only the filled part moves; the room behind it stays as it was."""
    dev = _dev()
    g = torch.Generator().manual_seed(length)
    n_seq, beams = 2, 5
    x = torch.randn(n_seq * beams, 3, 64, 10, generator=g).half()
    parents = torch.randint(0, beams, (n_seq, beams), generator=g)
    parents[1, 2] = 99                                  # no beam: zeros
    src = x.to(dev)
    dst = src if in_place else torch.full_like(src, 4.0)
    lce.beam_reorder([src], parents.to(dev), beams, out=None if in_place else [dst], length=length)
    want = (x if in_place else torch.full_like(x, 4.0)).clone()
    want[:, :, :length] = _reordered(x, parents, beams)[:, :, :length]
    assert torch.equal(dst.cpu(), want)


def test_reorder_many_states_and_views():
    """More states than one launch takes, at bases of every alignment."""
    dev = _dev()
    flat = torch.arange(70 * 400, dtype=torch.int32).to(torch.uint8)
    parents = torch.tensor([[2, 0, 1, 1]])
    src = [flat[i * 400 + i % 16: i * 400 + i % 16 + 4 * 83].view(4, 83) for i in range(70)]
    big = torch.zeros(70 * 400, dtype=torch.uint8, device=dev)
    dst = [big[i * 400 + (i * 7) % 16: i * 400 + (i * 7) % 16 + 4 * 83].view(4, 83) for i in range(70)]
    on = flat.to(dev)
    lce.beam_reorder([on[i * 400 + i % 16: i * 400 + i % 16 + 4 * 83].view(4, 83) for i in range(70)],
                     parents.to(dev), 4, out=dst)
    for a, b in zip(src, dst):
        assert torch.equal(b.cpu(), a[[2, 0, 1, 1]])
    covered = torch.zeros_like(big, dtype=torch.bool)
    for i in range(70):
        covered[i * 400 + (i * 7) % 16: i * 400 + (i * 7) % 16 + 4 * 83] = True
    assert bool((big[~covered] == 0).all())
