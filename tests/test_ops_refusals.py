"""Refusals of the operators next to the losses: decided on the host before
any device call, so they are checked without a GPU (CPU buffers)."""
import pytest
import torch

from lm_head_linear_amd import lce

U8 = torch.uint8


def test_checkpoint_refusals():
    x = torch.zeros(4, 40, dtype=torch.bfloat16)
    codes, scales = torch.zeros(4, 40, dtype=U8), torch.zeros(4, 2, dtype=U8)
    call = lambda **kw: lce.lce_pack8(**{**dict(x=x, n=4, d=40, codes=codes, scales=scales,
                                                stream=0), **kw})
    back = lambda **kw: lce.lce_unpack8(**{**dict(codes=codes, scales=scales, n=4, d=40, out=x,
                                                  stream=0), **kw})
    for f in (call, back):
        assert f(n=0) == 581
        assert f(d=0) == 581
        assert f(d=-3) == 581
        assert f(n=2 ** 24 + 1) == 583
        assert f(d=2 ** 24 + 1) == 583
        assert f(n=2 ** 24, d=2 ** 23) == 584
        assert f(codes=codes.int()) == 590
        assert f(scales=scales.float()) == 590
        assert f(codes=codes[:3]) == 582
        assert f(scales=scales[:, :1].contiguous()) == 582
    assert call(x=x.float()) == 590
    assert back(out=x.float()) == 590
    assert call(x=x[:3]) == 582
    assert back(out=x[:3]) == 582
    with pytest.raises(ValueError):
        lce.pack8(x)                                    # not on a GPU


def test_beam_select_refusals():
    n_seq, beams, V, n_out = 2, 3, 50, 4
    rows = n_seq * beams
    ws = lce.lce_beam_workspace_bytes(n_seq, beams, V, n_out)
    assert ws > 0
    w = lce.lce_beam_workspace_bytes
    assert w(0, 3, 50, 4) == -581 and w(2, 0, 50, 4) == -581
    assert w(2, 3, 0, 4) == -581 and w(2, 3, 50, 0) == -581
    assert w(2, 33, 50, 4) == -583 and w(2, 3, 50, 65) == -583
    assert w(2 ** 24 + 1, 3, 50, 4) == -583 and w(2, 3, 2 ** 24 + 1, 4) == -583
    assert w(2 ** 20, 32, 50, 4) == -584
    base = dict(logits=torch.zeros(rows, V), scores=torch.zeros(rows), finished=None, allowed=None,
                n_seq=n_seq, beams=beams, vocab=V, n_out=n_out, eos=-1,
                out_scores=torch.zeros(n_seq * n_out),
                out_parents=torch.zeros(n_seq * n_out, dtype=torch.int64),
                out_tokens=torch.zeros(n_seq * n_out, dtype=torch.int64), out_finished=None,
                workspace=torch.zeros(ws, dtype=U8), stream=0)
    call = lambda **kw: lce.lce_beam_select(**{**base, **kw})
    assert call(n_seq=0) == 581
    assert call(beams=33) == 583
    assert call(n_out=65) == 583
    assert call(logits=torch.zeros(rows, V, dtype=torch.float64)) == 590
    assert call(scores=torch.zeros(rows, dtype=torch.float16)) == 590
    assert call(out_tokens=torch.zeros(n_seq * n_out, dtype=torch.int32)) == 590
    assert call(finished=torch.zeros(rows), eos=1) == 590
    assert call(allowed=torch.zeros(rows, V)) == 590
    assert call(out_finished=torch.zeros(n_seq * n_out)) == 590
    assert call(workspace=torch.zeros(ws)) == 590
    assert call(logits=torch.zeros(rows, V - 1)) == 582
    assert call(scores=torch.zeros(rows - 1)) == 582
    assert call(out_parents=torch.zeros(n_seq * n_out - 1, dtype=torch.int64)) == 582
    assert call(finished=torch.zeros(rows - 1, dtype=U8), eos=1) == 582
    assert call(allowed=torch.zeros(rows, V - 1, dtype=U8)) == 582
    assert call(out_finished=torch.zeros(n_seq * n_out - 1, dtype=U8)) == 582
    assert call(workspace=torch.zeros(ws - 1, dtype=U8)) == 582
    assert call(eos=V) == 586
    assert call(eos=-2) == 586
    assert call(finished=torch.zeros(rows, dtype=U8)) == 586
    with pytest.raises(ValueError):
        lce.beam_select(torch.zeros(rows, V), torch.zeros(n_seq, beams), 4)
    with pytest.raises(ValueError):
        lce.beam_select(torch.zeros(rows + 1, V), torch.zeros(n_seq, beams), 4)


def test_beam_reorder_refusals():
    n_seq, beams = 2, 3
    src, dst = [torch.zeros(6, 20)], [torch.zeros(6, 20)]
    p = torch.zeros(n_seq, beams, dtype=torch.int64)
    base = dict(src=src, dst=dst, parents=p, n_seq=n_seq, beams=beams, n_out=beams, segs=4,
                seg_elems=5, seg_stride=5, stream=0)
    call = lambda **kw: lce.lce_beam_reorder(**{**base, **kw})
    assert call(src=[], dst=[]) == 581
    for k in ("n_seq", "beams", "n_out", "segs", "seg_stride"):
        assert call(**{k: 0}) == 581
    assert call(seg_elems=-1) == 581
    assert call(beams=33) == 583
    assert call(n_out=33) == 583
    assert call(n_seq=2 ** 24 + 1) == 583
    assert call(segs=2 ** 40, seg_stride=2 ** 10) == 584
    assert call(parents=p.int()) == 590
    assert call(dst=[torch.zeros(6, 20, dtype=torch.int64)]) == 590
    assert call(src=src * 2, dst=dst + [torch.zeros(6, 20, dtype=torch.float16)]) == 590
    assert call(seg_elems=6) == 582
    assert call(parents=p[:1]) == 582
    assert call(src=[torch.zeros(5, 20)]) == 582
    assert call(dst=[torch.zeros(5, 20)]) == 582
    # an overlap, some in place and some not, in place with another row count
    room = torch.zeros(7, 20)
    assert call(src=[room[:6]], dst=[room[1:]]) == 582
    assert call(src=[src[0], room[:6]], dst=[src[0], torch.zeros(6, 20)]) == 582
    assert call(src=[room[:6]], dst=[room[:6]], n_out=2, parents=p) == 582
    # one state twice, states that change places, a destination in the parents
    assert call(src=[src[0]] * 2, dst=[src[0]] * 2) == 582
    assert call(src=src * 2, dst=dst * 2) == 582
    a, b, c = (torch.zeros(6, 20) for _ in range(3))
    assert call(src=[a, b], dst=[b, a]) == 582
    assert call(src=[a, b], dst=[c, a]) == 582
    words = torch.zeros(6, 20, dtype=torch.int64)
    assert call(src=[torch.zeros_like(words)], dst=[words], parents=words.view(-1)[30:36]) == 582
    assert call(src=[torch.zeros(6, 20) for _ in range(1025)],
                dst=[torch.zeros(6, 20) for _ in range(1025)]) == 583
    assert call(seg_elems=0) == 580                     # nothing to carry over
    with pytest.raises(ValueError):
        lce.beam_reorder(src, p, beams)
    with pytest.raises(ValueError):
        lce.lce_beam_reorder(src, dst * 2, p, 2, 3, 3, 4, 5, 5, 0)


def test_linear_refusals():
    n, d_in, d_out = 70, 8200, 12           # (the depth in parts: a workspace)
    t = torch.bfloat16
    w = lce.lce_linear_workspace_bytes
    v = lce.lce_linear_backward_workspace_bytes
    for f in (w, v):
        assert f(n, d_in, d_out, t) == f(n, d_in, d_out, torch.float16) >= 0
        assert f(0, d_in, d_out, t) == -581 and f(n, 0, d_out, t) == -581
        assert f(n, d_in, 0, t) == -581
        assert f(n, 2 ** 16 + 1, d_out, t) == -583 and f(2 ** 24, 2 ** 12, 2 ** 12, t) == -584
        assert f(n, d_in, d_out, torch.float32) == -590
    base = dict(x=torch.zeros(n, d_in, dtype=t), weight=torch.zeros(d_out, d_in, dtype=t),
                bias=torch.zeros(d_out), residual=torch.zeros(n, d_out, dtype=t), n_tok=n,
                d_in=d_in, d_out=d_out, activation=2, preact=torch.zeros(n, d_out, dtype=t),
                out=torch.zeros(n, d_out, dtype=t),
                workspace=torch.zeros(w(n, d_in, d_out, t), dtype=U8), stream=0)
    call = lambda **kw: lce.lce_linear(**{**base, **kw})
    assert call(n_tok=0) == 581 and call(d_in=0) == 581 and call(d_out=-1) == 581
    assert call(d_in=2 ** 16 + 1) == 583
    assert call(n_tok=2 ** 24, d_in=2 ** 12, d_out=2 ** 12) == 584
    assert call(x=base["x"].float()) == 590
    for k in ("weight", "residual", "preact", "out"):
        assert call(**{k: base[k].half()}) == 590, k
    assert call(bias=torch.zeros(d_out, dtype=torch.float64)) == 590
    assert call(workspace=base["workspace"].float()) == 590
    for k in ("x", "weight", "bias", "residual", "preact", "out", "workspace"):
        assert call(**{k: base[k][:-1]}) == 582, k
    assert call(x=None) in (582, 590)
    assert call(out=None) in (582, 590)
    assert call(activation=4) == 588 and call(activation=-1) == 588
    with pytest.raises(ValueError):
        lce.linear(base["x"], base["weight"])               # not on a GPU
    with pytest.raises(ValueError):
        lce.linear(base["x"], base["weight"][:, :9].contiguous())

    bw = dict(d_out_grad=torch.zeros(n, d_out, dtype=t), x=base["x"], x_scales=None,
              weight=base["weight"], preact=base["preact"], preact_scales=None, n_tok=n, d_in=d_in,
              d_out=d_out, activation=2, d_x=torch.zeros(n, d_in, dtype=t),
              d_weight=torch.zeros(d_out, d_in), d_bias=torch.zeros(d_out), accumulate=0,
              workspace=torch.zeros(v(n, d_in, d_out, t), dtype=U8), stream=0)
    call = lambda **kw: lce.lce_linear_backward(**{**bw, **kw})
    codes, zcodes = torch.zeros(n, d_in, dtype=U8), torch.zeros(n, d_out, dtype=U8)
    scales, zscales = torch.zeros(n, 257, dtype=U8), torch.zeros(n, 1, dtype=U8)
    assert w(n, d_in, d_out, t) > 0 and w(3, d_in, d_out, t) == 0
    assert call(n_tok=0) == 581 and call(d_in=0) == 581 and call(d_out=0) == 581
    assert call(d_in=2 ** 16 + 1) == 583
    assert call(d_x=None, d_weight=None, d_bias=None) == 582
    assert call(weight=None) == 582 and call(x=None) == 582 and call(preact=None) == 582
    assert call(d_out_grad=bw["d_out_grad"].float()) == 590
    for k in ("x", "weight", "preact", "d_x", "d_weight", "d_bias"):
        assert call(**{k: bw[k].half()}) == 590, k
    assert call(x=codes) == 590 and call(x_scales=scales) == 590
    assert call(x=codes, x_scales=scales.float()) == 590
    assert call(preact=zcodes) == 590 and call(preact_scales=zscales) == 590
    assert call(x=codes, x_scales=scales[:2]) == 582
    assert call(preact=zcodes, preact_scales=zscales[:2]) == 582
    for k in ("d_out_grad", "x", "weight", "preact", "d_x", "d_weight", "d_bias", "workspace"):
        assert call(**{k: bw[k][:-1]}) == 582, k
    assert call(activation=7) == 588
    with pytest.raises(ValueError):
        lce.linear_backward(bw["d_out_grad"], base["x"], base["weight"], base["preact"])
    with pytest.raises(ValueError):
        lce.linear_backward(bw["d_out_grad"], base["x"], base["weight"][:5], base["preact"])
    with pytest.raises(ValueError):
        lce.linear_backward(bw["d_out_grad"], base["x"], base["weight"], accumulate=True)
