"""The operators next to the losses, used together: a head's transform trained
through the fused loss with 8-bit checkpoints, and steps of beam search from
hidden states to reordered caches; eagerly, on other streams, and captured in
HIP graphs that are replayed between eager work.  Each stage is checked
against its 64-bit form on the stage's own inputs, so that the bounds are
those of the single operators."""
import numpy as np
import pytest
import torch

import oracle
from lm_head_linear_amd import lce
from tests import ops_plain
from tests.test_gpu_linear import _check_backward, _check_forward

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


class Train:
    """x -> transform (gelu, residual) -> fused head loss -> gradients."""

    def __init__(self, n, d, vocab, seed, dev, t=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)
        self.n, self.d, self.vocab, self.chunk = n, d, vocab, 64
        self.x = r(n, d).to(t).to(dev)
        self.w = (r(d, d) / d ** 0.5).to(t).to(dev)
        self.b = (0.1 * r(d)).to(dev)
        self.head = (r(vocab, d) / d ** 0.5).to(t).to(dev)
        self.y = torch.randint(0, vocab, (n,), generator=g).to(dev)
        new = lambda *s, dtype=t: torch.empty(*s, dtype=dtype, device=dev)
        nb = -(-d // 32)
        self.h, self.z, self.dh, self.dx = (new(n, d) for _ in range(4))
        self.x8 = lce.Packed8(new(n, d, dtype=torch.uint8), new(n, nb, dtype=torch.uint8), t)
        self.z8 = lce.Packed8(new(n, d, dtype=torch.uint8), new(n, nb, dtype=torch.uint8), t)
        self.lse = new(n, dtype=torch.float32)
        self.dhead = new(vocab, d, dtype=torch.float32)
        self.dw = new(d, d, dtype=torch.float32)
        self.db = new(d, dtype=torch.float32)
        self.ws = lce.workspace_for(n, d, vocab, self.chunk, t, dev)
        self.lws = new(max(lce.lce_linear_workspace_bytes(n, d, d, t),
                           lce.lce_linear_backward_workspace_bytes(n, d, d, t)), dtype=torch.uint8)

    def step(self):
        n, d, V, c = self.n, self.d, self.vocab, self.chunk
        ok = []
        ok.append(lce.lce_linear(self.x, self.w, self.b, self.x, n, d, d, 2, self.z, self.h, self.lws))
        ok.append(lce.lce_pack8(self.x, n, d, self.x8.codes, self.x8.scales))
        ok.append(lce.lce_pack8(self.z, n, d, self.z8.codes, self.z8.scales))
        ok.append(lce.lce_forward(self.h, self.head, self.y, None, n, d, V, c, 1e-4, self.lse,
                                  self.ws, sync=False)[0])
        ok.append(lce.lce_backward(self.h, self.head, self.y, None, self.lse, n, d, V, c, 1e-4, 1.0,
                                   self.dh, self.dhead, False, self.ws))
        ok.append(lce.lce_linear_backward(self.dh, self.x8.codes, self.x8.scales, self.w,
                                          self.z8.codes, self.z8.scales, n, d, d, 2, self.dx, self.dw,
                                          self.db, 0, self.lws))
        assert ok == [580] * len(ok), ok

    def results(self):
        return [a.clone() for a in (self.h, self.z, self.x8.codes, self.z8.codes, self.lse, self.dh,
                                    self.dhead, self.dx, self.dw, self.db)]


def test_training_step():
    dev = _dev()
    s = Train(150, 96, 700, 1, dev)
    s.step()
    _check_forward(s.x, s.w, s.b, s.x, "gelu", True, torch.bfloat16, lce.LinearResult(s.h, s.z))
    st, loss = lce.lce_loss_fetch(s.ws)
    assert st == 580
    H, W = s.h.double().cpu().numpy(), s.head.double().cpu().numpy()
    y = s.y.cpu().numpy()
    ref = oracle.fused_forward(H, W, y, chunk=64, z_coef=1e-4)
    assert abs(loss.loss_mean - ref["loss_mean"]) <= 2e-3 * abs(ref["loss_mean"])
    rdh, rdw = oracle.backward(H, W, y, ref["lse"], z_coef=1e-4)
    assert np.abs(s.dh.double().cpu().numpy() - rdh).max() <= 1e-2 * np.abs(rdh).max()
    assert np.abs(s.dhead.double().cpu().numpy() - rdw).max() <= 1e-2 * np.abs(rdw).max()
    for full, packed in ((s.x, s.x8), (s.z, s.z8)):
        back = lce.unpack8(packed)
        want, _ = ops_plain.checkpoint(full.double().cpu().numpy(), 3.3895313892515355e38, -117)
        assert np.array_equal(back.double().cpu().numpy(), want)
    _check_backward(s.dh, s.x, s.w, s.z, "gelu", lce.LinearGrads(s.dx, s.dw, s.db),
                    lce.unpack8(s.x8), lce.unpack8(s.z8))


class Beams:
    """One step of beam search: logits, selection, caches and histories."""

    def __init__(self, n_seq, beams, d, vocab, seed, dev, t=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)
        rows = n_seq * beams
        self.n_seq, self.beams, self.vocab, self.length = n_seq, beams, vocab, 5
        self.h = r(rows, d).to(t).to(dev)
        self.head = (2 * r(vocab, d) / d ** 0.5).to(t).to(dev)
        self.b = r(vocab).to(dev)
        self.scores = (-torch.rand(n_seq, beams, generator=g)).to(dev)
        self.done = (torch.rand(n_seq, beams, generator=g) < 0.2).to(dev)
        self.caches0 = [r(rows, 3, 9, 16).to(t).to(dev) for _ in range(4)]
        self.caches = [c.clone() for c in self.caches0]
        self.history = torch.randint(0, vocab, (rows, 9), generator=g).to(dev)

    def step(self):
        self.logits = lce.linear(self.h, self.head, self.b).out
        self.choice = lce.beam_select(self.logits, self.scores, self.beams, finished=self.done, eos=7)
        for c, c0 in zip(self.caches, self.caches0):
            c.copy_(c0)
        lce.beam_reorder(self.caches, self.choice.parents, self.beams, length=self.length)
        (self.moved,) = lce.beam_reorder([self.history], self.choice.parents, self.beams,
                                         out=[torch.empty_like(self.history)])

    def results(self):
        c = self.choice
        return [a.clone() for a in (self.logits, c.scores, c.parents, c.tokens, c.finished, self.moved,
                                    *self.caches)]

    def check(self):
        _check_forward(self.h, self.head, self.b, None, "none", False, torch.bfloat16,
                       lce.LinearResult(self.logits, None))
        S, P, T, F = ops_plain.beam_select(self.logits.double().cpu().numpy(),
                                           self.scores.cpu().numpy(), self.beams,
                                           self.done.cpu().numpy(), None, 7)
        c = self.choice
        assert np.array_equal(c.parents.cpu().numpy(), P) and np.array_equal(c.tokens.cpu().numpy(), T)
        assert np.array_equal(c.finished.cpu().numpy(), F)
        assert np.abs(c.scores.cpu().double().numpy() - S).max() <= 2.0 ** -18 + 2.0 ** -24 * np.abs(S).max()
        rows = (torch.arange(self.n_seq).view(-1, 1) * self.beams + c.parents.cpu()).view(-1)
        assert torch.equal(self.moved.cpu(), self.history.cpu()[rows])
        for a, a0 in zip(self.caches, self.caches0):
            want = a0.cpu().clone()
            want[:, :, :self.length] = a0.cpu()[rows][:, :, :self.length]
            assert torch.equal(a.cpu(), want)


@pytest.mark.parametrize("n_seq,beams,d,vocab", [(1, 4, 64, 900), (3, 5, 72, 4001), (8, 16, 128, 9000)])
def test_beam_search_step(n_seq, beams, d, vocab):
    s = Beams(n_seq, beams, d, vocab, 3, _dev())
    s.step()
    s.check()


@pytest.mark.parametrize("what", ["train", "train large", "beams"])
def test_captured_and_replayed(what):
    """Every replay gives the eager bits, with eager work and new inputs between."""
    dev = _dev()
    make = {"train": lambda seed: Train(150, 96, 700, seed, dev),
            "train large": lambda seed: Train(2100, 520, 900, seed, dev),
            "beams": lambda seed: Beams(3, 5, 72, 4001, seed, dev)}[what]
    s, other = make(5), make(6)

    def inputs(q):
        if what == "beams":
            return [q.h, q.head, q.b, q.scores, q.done, q.history, *q.caches0]
        return [q.x, q.w, q.b, q.head, q.y]

    eager = []
    for q in (s, other):
        q.step()
        eager.append(q.results())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    kept = [a.clone() for a in inputs(s)]
    for i in range(5):
        for a, b in zip(inputs(s), inputs(other) if i % 2 else kept):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for j, (got, want) in enumerate(zip(s.results(), eager[i % 2])):
            assert torch.equal(got, want), (i, j)
        make(7).step()                                   # eager work between
        torch.cuda.synchronize()


def test_two_graphs_share_a_workspace():
    dev = _dev()
    n, d = 300, 264
    a, b = Train(n, d, 400, 8, dev), Train(n, d, 400, 9, dev)
    b.lws, b.ws = a.lws, a.ws
    a.step(), b.step()
    want_a, want_b = a.results(), b.results()
    graphs = []
    for s in (a, b):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step()
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for got, want in ((a.results(), want_a), (b.results(), want_b)):
            assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_other_streams():
    """Calls on a stream of their own, and on two at once with workspaces of
    their own."""
    dev = _dev()
    s = [Train(200, 136, 500, 10 + i, dev) for i in range(2)]
    q = [Beams(2, 4, 64, 3000, 20 + i, dev) for i in range(2)]
    for t in (*s, *q):
        t.step()
    want = [t.results() for t in (*s, *q)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                s[i].step()
                q[i].step()
        torch.cuda.synchronize()
        for got, w in zip([t.results() for t in (*s, *q)], want):
            assert all(torch.equal(x, y) for x, y in zip(got, w))


def test_offsets_beyond_32_bits():
    """Caches, logits and checkpoints of more than 2^32 bytes (2^31 elements):
    the far ends are read and written where they lie."""
    dev = _dev()
    row = 1_200_000_007                                  # bytes of a row: 4.8 GB in all
    cache = torch.zeros(4, row, dtype=torch.uint8, device=dev)
    for k in range(4):
        cache[k, :3] = 10 + k
        cache[k, -3:] = 20 + k
        cache[k, row // 2] = 30 + k
    parents = torch.tensor([[3, 2, 1, 3]], device=dev)
    (moved,) = lce.beam_reorder([cache], parents, 4, out=[torch.empty_like(cache)])
    for j, k in enumerate((3, 2, 1, 3)):
        assert torch.equal(moved[j, :3], cache[k, :3]) and torch.equal(moved[j, -3:], cache[k, -3:])
        assert int(moved[j, row // 2]) == 30 + k
    lce.beam_reorder([cache], parents, 4)
    assert torch.equal(cache, moved)
    del cache, moved

    V, n_seq, beams = 1 << 24, 5, 26
    logits = torch.full((n_seq * beams, V), -8.0, dtype=torch.bfloat16, device=dev)
    logits[-1, V - 2], logits[-1, 5] = 12.0, 11.0
    logits[0, V - 1], logits[0, 4] = 10.0, 9.5
    r = lce.beam_select(logits, torch.zeros(n_seq, beams, device=dev), 2)
    assert r.parents[-1].tolist() == [beams - 1] * 2 and r.tokens[-1].tolist() == [V - 2, 5]
    assert r.parents[0].tolist() == [0, 0] and r.tokens[0].tolist() == [V - 1, 4]
    assert r.tokens[1].tolist() == [0, 1] and r.parents[1].tolist() == [0, 0]
    del logits

    n, d = 65600, 65537
    x = torch.ones(n, d, dtype=torch.bfloat16, device=dev)
    x[-1, -40:] = 3.0
    p = lce.pack8(x)
    back = lce.unpack8(p)
    assert torch.equal(back[-2:], x[-2:]) and torch.equal(back[:2], x[:2])
    assert int(p.scales[-1, -1]) == 127 - 7                # 3 = 384 / 2^7


def test_a_tensor_on_another_device_or_the_host_is_refused():
    dev = _dev()
    x = torch.zeros(2, 8, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(3, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lce.linear(x, w)
    with pytest.raises(ValueError):
        lce.beam_select(x, torch.zeros(1, 2), 2)
    with pytest.raises(ValueError):
        lce.pack8(x[:, :4])                                # not contiguous
    with pytest.raises(lce.LceError) as e:
        lce.linear(x, w.to(dev), activation="tanh")
    assert e.value.status == 588
    with pytest.raises(lce.LceError) as e:
        lce.linear(x.float(), w.to(dev).float())
    assert e.value.status == 590
