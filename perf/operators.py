"""Timing cases of the operators around the head: the linear layer with its
epilogue, its backward, 8-bit activation checkpoints, beam selection and the
reordering of beam states.  `own` False computes them in elementary torch
operations, True through lm_head_linear_amd."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
BLOCK = 32          # values that share one scale of an 8-bit checkpoint
MOST_FLOPS = 2 * 8192 * 4096 * 4096


def listed():
    return [
        # one token through a decoder's head transform: latency
        {"name": "linear one token", "op": "linear", "n": 1, "d_in": 1024, "d_out": 1024, "type": "bf16",
         "out": "bf16", "act": "gelu", "bias": True, "residual": True, "preact": False},
        # the logits of 8 sequences x 4 beams: one read of the head
        {"name": "linear beam logits", "op": "linear", "n": 32, "d_in": 1024, "d_out": 151936, "type": "bf16",
         "out": "bf16", "act": "none", "bias": True, "residual": False, "preact": False},
        # a training batch, pre-activation kept for the backward
        {"name": "linear training batch", "op": "linear", "n": 8192, "d_in": 4096, "d_out": 4096, "type": "bf16",
         "out": "bf16", "act": "gelu", "bias": True, "residual": True, "preact": True},
        # a ragged batch with rows that are not 16-byte aligned
        {"name": "linear odd", "op": "linear", "n": 777, "d_in": 1003, "d_out": 1531, "type": "fp16",
         "out": "f32", "act": "silu", "bias": True, "residual": False, "preact": True},
        # the training batch's backward with input and pre-activation kept in 8 bits
        {"name": "backward training batch", "op": "backward", "n": 8192, "d_in": 4096, "d_out": 4096,
         "type": "bf16", "act": "gelu", "bias": True, "saved8": True},
        # the ragged batch's backward from 16-bit saved tensors
        {"name": "backward odd", "op": "backward", "n": 515, "d_in": 1003, "d_out": 777, "type": "fp16",
         "act": "silu", "bias": True, "saved8": False},
        # the checkpoint of a training batch, written and read back
        {"name": "checkpoint training batch", "op": "checkpoint", "n": 8192, "d": 4096, "type": "bf16"},
        # a small ragged checkpoint
        {"name": "checkpoint odd", "op": "checkpoint", "n": 37, "d": 1003, "type": "fp16"},
        # a serving batch: 64 sequences x 8 beams over a large vocabulary, two candidates a beam
        {"name": "select serving batch", "op": "select", "n_seq": 64, "beams": 8, "vocab": 151936,
         "n_out": 16, "type": "bf16", "finished": False, "allowed": False},
        # one sequence with finished beams and a grammar's mask, odd vocabulary
        {"name": "select one sequence", "op": "select", "n_seq": 1, "beams": 4, "vocab": 32003,
         "n_out": 4, "type": "f32", "finished": True, "allowed": True},
        # caches of 16 layers, filled to a ragged length
        {"name": "reorder serving batch", "op": "reorder", "n_seq": 8, "beams": 8, "states": 16, "heads": 8,
         "room": 1024, "length": 777, "d_head": 128, "type": "bf16"},
        # one sequence's small caches
        {"name": "reorder one sequence", "op": "reorder", "n_seq": 1, "beams": 4, "states": 4, "heads": 2,
         "room": 64, "length": 33, "d_head": 64, "type": "fp16"},
    ]


def _span(rng, lo, hi):
    """A whole number from lo to hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "backward", "checkpoint", "select", "reorder"])
    kind = rng.choice(["bf16", "fp16"])
    if op in ("linear", "backward"):
        n, d_in = _span(rng, 1, 8192), _span(rng, 16, 4096)
        even = rng.random() < 0.6                   # most layers have round widths, some do not
        d_in = d_in // 16 * 16 if even else d_in
        most = 151936 if op == "linear" and n <= 64 else 8192
        d_out = _span(rng, 16, max(16, min(most, MOST_FLOPS // (2 * n * d_in))))
        d_out = d_out // 16 * 16 if even else d_out
        c = {"op": op, "n": n, "d_in": d_in, "d_out": d_out, "type": kind,
             "act": rng.choice(["none", "relu", "gelu", "silu"]), "bias": rng.random() < 0.8}
        if op == "backward":
            return {**c, "saved8": rng.random() < 0.5}
        return {**c, "out": rng.choice([kind, "f32"]), "residual": rng.random() < 0.5,
                "preact": rng.random() < 0.5}
    if op == "checkpoint":
        return {"op": op, "n": _span(rng, 1, 8192), "d": _span(rng, 1, 4096), "type": kind}
    beams = rng.randint(1, 16)
    if op == "select":
        n_seq = _span(rng, 1, 512 // beams)
        return {"op": op, "n_seq": n_seq, "beams": beams, "vocab": _span(rng, 500, 151936),
                "n_out": rng.randint(1, 2 * beams), "type": rng.choice(["bf16", "fp16", "f32"]),
                "finished": rng.random() < 0.5, "allowed": rng.random() < 0.3}
    n_seq = _span(rng, 1, 64 // beams)
    room = _span(rng, 1, 1024)
    return {"op": op, "n_seq": n_seq, "beams": beams, "states": rng.randint(1, 16),
            "heads": rng.randint(1, 8), "room": room, "length": rng.randint(1, room),
            "d_head": rng.choice([40, 64, 80, 96, 128]), "type": kind}


# --------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, t=torch.float32):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(t)

    s = {"case": case}
    op = case["op"]
    t = TYPES[case["type"]]
    if op == "linear":
        n, d_in, d_out = case["n"], case["d_in"], case["d_out"]
        s["x"] = normal(n, d_in, t=t)
        s["weight"] = normal(d_out, d_in, std=d_in ** -0.5, t=t)
        s["bias"] = normal(d_out, std=0.1) if case["bias"] else None
        s["residual"] = normal(n, d_out, t=t) if case["residual"] else None
    elif op == "backward":
        n, d_in, d_out = case["n"], case["d_in"], case["d_out"]
        s["d_out"] = normal(n, d_out, std=0.01, t=t)
        s["x"] = normal(n, d_in, t=t)
        s["weight"] = normal(d_out, d_in, std=d_in ** -0.5, t=t)
        s["preact"] = normal(n, d_out, t=t) if case["act"] != "none" else None
        if case["saved8"]:
            s["x"] = _pack8(s["x"])
            s["preact"] = None if s["preact"] is None else _pack8(s["preact"])
    elif op == "checkpoint":
        n, d = case["n"], case["d"]
        # hidden states: a few wide columns, a spread of row sizes, rows of zeros
        rows = torch.exp(normal(n, 1))
        cols = torch.where(torch.rand(1, d, generator=g, device=DEV) < 0.02, 20.0, 1.0)
        keep = (torch.rand(n, 1, generator=g, device=DEV) > 0.01).float()
        s["x"] = (normal(n, d) * rows * cols * keep).to(t)
    elif op == "select":
        n_seq, beams, vocab = case["n_seq"], case["beams"], case["vocab"]
        rows = n_seq * beams
        s["logits"] = normal(rows, vocab, std=3.0, t=t)
        s["scores"] = -20.0 - 3.0 * torch.rand(n_seq, beams, generator=g, device=DEV)
        if case["finished"]:
            s["finished"] = torch.rand(n_seq, beams, generator=g, device=DEV) < 0.25
        if case["allowed"]:
            # a grammar leaves some beams many tokens, some few, some none
            share = torch.rand(rows, 1, generator=g, device=DEV) ** 3
            share[torch.rand(rows, 1, generator=g, device=DEV) < 0.1] = 0.0
            s["allowed"] = torch.rand(rows, vocab, generator=g, device=DEV) < share
    else:
        rows = case["n_seq"] * case["beams"]
        shape = (rows, case["heads"], case["room"], case["d_head"])
        s["states"] = [normal(*shape, t=t) for _ in range(case["states"])]
        s["into"] = [torch.zeros_like(x) for x in s["states"]]
        s["parents"] = torch.randint(0, case["beams"], (case["n_seq"], case["beams"]), generator=g, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _plain_linear(s, case):
    z = s["x"].float() @ s["weight"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"out": y.to(TYPES[case["out"]])}
    if case["preact"]:
        out["preact"] = z.to(s["x"].dtype)
    return out


def _pack8(x):
    """Codes [n][d] and exponents [n][d / 32, rounded up]: x is about code * 2^exponent,
    the exponent the smallest that keeps every magnitude of the block within 448 (and at
    least -117, for fp16 -15, so that code * 2^exponent is a number of x's type)."""
    n, d = x.shape
    blocks = (d + BLOCK - 1) // BLOCK
    f = torch.zeros(n, blocks * BLOCK, device=x.device)
    f[:, :d] = x.float()
    f = f.view(n, blocks, BLOCK)
    part, power = torch.frexp(f.abs().amax(2))      # amax = part * 2^power, part in [0.5, 1)
    e = torch.where(part <= 0.875, power - 9, power - 8)
    e = torch.where(part == 0, -127, e).clamp(min=-15 if x.dtype == torch.float16 else -117)
    codes = torch.ldexp(f, -e[:, :, None]).to(torch.float8_e4m3fn)
    return {"codes": codes.view(n, -1)[:, :d].contiguous().view(torch.uint8), "scales": (e + 127).to(torch.uint8),
            "type": x.dtype}


def _unpack8(p):
    n, d = p["codes"].shape
    e = (p["scales"].int() - 127).repeat_interleave(BLOCK, 1)[:, :d]
    most = torch.finfo(p["type"]).max
    return torch.ldexp(p["codes"].view(torch.float8_e4m3fn).float(), e).clamp(-most, most).to(p["type"])


def _plain_backward(s, case):
    x, z = s["x"], s["preact"]
    if case["saved8"]:
        x, z = _unpack8(x), None if z is None else _unpack8(z)
    g = s["d_out"].float()
    if z is not None:
        g = g * _act_slope(z.float(), case["act"])
    t = s["d_out"].dtype
    out = {"d_x": (g @ s["weight"].float()).to(t), "d_weight": (g.t() @ x.float()).to(t)}
    if case["bias"]:
        out["d_bias"] = g.sum(0)
    return out


def _plain_select(s, case):
    """In 64 bits: the order of candidates is decided by small differences."""
    n_seq, beams, vocab, n_out = case["n_seq"], case["beams"], case["vocab"], case["n_out"]
    x = s["logits"].double()
    none = torch.full((), -math.inf, dtype=torch.float64, device=x.device)
    if "allowed" in s:
        x = torch.where(s["allowed"], x, none)
    top = x.amax(1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    lse = top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
    total = s["scores"].double().view(-1, 1) + (x - lse)
    total = torch.where(torch.isfinite(total), total, none).view(n_seq, beams, vocab)
    token = torch.arange(vocab, device=x.device)
    done = s.get("finished")
    if done is not None:
        kept = torch.where(token == _eos(case), s["scores"].double()[:, :, None], none)
        total = torch.where(done[:, :, None], kept, total)
    total = total.view(n_seq, beams * vocab)
    last = torch.topk(total, n_out, 1).values[:, -1:]
    above, level = total > last, total == last
    room = n_out - above.sum(1, keepdim=True)
    pick = above | (level & (torch.cumsum(level, 1) <= room))      # ties: the lowest places
    place = torch.arange(beams * vocab, device=x.device)
    place = -torch.topk(torch.where(pick, -place, -beams * vocab), n_out, 1).values
    best, order = torch.sort(total.gather(1, place), dim=1, descending=True, stable=True)
    place = place.gather(1, order)
    real = best > none
    parents = torch.where(real, place // vocab, -1)
    tokens = torch.where(real, place % vocab, -1)
    out = {"scores": best.float(), "parents": parents, "tokens": tokens}
    if done is not None:
        out["finished"] = real & (tokens == _eos(case))
    return out


def _eos(case):
    return case["vocab"] // 3


def _plain_reorder(s, case):
    rows = s["parents"] + torch.arange(case["n_seq"], device=DEV)[:, None] * case["beams"]
    rows, n = rows.view(-1), case["length"]
    for src, dst in zip(s["states"], s["into"]):
        dst[:, :, :n] = src[:, :, :n][rows]
    return s["into"]


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "linear":
            return _plain_linear(state, case)
        if op == "backward":
            return _plain_backward(state, case)
        if op == "checkpoint":
            return _unpack8(_pack8(state["x"]))
        if op == "select":
            return _plain_select(state, case)
        return _plain_reorder(state, case)

    from lm_head_linear_amd import lce
    if op == "linear":
        r = lce.linear(state["x"], state["weight"], state["bias"], state["residual"], activation=case["act"],
                       want_preact=case["preact"], out_dtype=TYPES[case["out"]])
        return {"out": r.out, "preact": r.preact} if case["preact"] else {"out": r.out}
    if op == "backward":
        x, z = state["x"], state["preact"]
        if case["saved8"]:
            x, z = (None if p is None else lce.Packed8(p["codes"], p["scales"], p["type"]) for p in (x, z))
        g = lce.linear_backward(state["d_out"], x, state["weight"], z, activation=case["act"],
                                want_bias=case["bias"], weight_grad_dtype=state["d_out"].dtype)
        out = {"d_x": g.d_x, "d_weight": g.d_weight}
        if case["bias"]:
            out["d_bias"] = g.d_bias
        return out
    if op == "checkpoint":
        return lce.unpack8(lce.pack8(state["x"]))
    if op == "select":
        done = state.get("finished")
        r = lce.beam_select(state["logits"], state["scores"], case["n_out"], finished=done,
                            allowed=state.get("allowed"), eos=None if done is None else _eos(case))
        out = {"scores": r.scores, "parents": r.parents, "tokens": r.tokens}
        if done is not None:
            out["finished"] = r.finished
        return out
    return lce.beam_reorder(state["states"], state["parents"], case["beams"], out=state["into"],
                            length=case["length"])


# ----------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    size = 4 if case["type"] == "f32" else 2
    if op in ("linear", "backward"):
        n, k, m = case["n"], case["d_in"], case["d_out"]
        if op == "linear":
            b = 2 * (n * k + m * k) + (4 if case["out"] == "f32" else 2) * n * m
            b += 4 * m * case["bias"] + 2 * n * m * (case["residual"] + case["preact"])
            return {"bytes": b, "flops": 2 * n * k * m}
        saved = 1 + 1 / BLOCK if case["saved8"] else 2
        b = 2 * (n * m + m * k) + saved * (n * k + n * m * (case["act"] != "none"))
        return {"bytes": b + 2 * (n * k + m * k) + 4 * m * case["bias"], "flops": 4 * n * k * m}
    if op == "checkpoint":
        n, d = case["n"], case["d"]
        return {"bytes": 2 * (2 * n * d + n * d + n * ((d + BLOCK - 1) // BLOCK)), "flops": 4 * n * d}
    if op == "select":
        rows, v = case["n_seq"] * case["beams"], case["vocab"]
        return {"bytes": rows * v * (size + case["allowed"]) + rows * 4 + case["n_seq"] * case["n_out"] * 20,
                "flops": 4 * rows * v}
    cells = case["n_seq"] * case["beams"] * case["heads"] * case["length"] * case["d_head"] * case["states"]
    read = 1 - (1 - 1 / case["beams"]) ** case["beams"]     # the share of rows that some beam continues
    return {"bytes": (1 + read) * size * cells, "flops": 0}


# -------------------------------------------------------------- 64-bit values

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        z = torch.matmul(s["weight"].double(), s["x"].double().mT).mT
        if case["bias"]:
            z = z + s["bias"].double()
        y = z
        if case["act"] == "relu":
            y = torch.maximum(z, torch.zeros_like(z))
        elif case["act"] == "gelu":                 # z times the normal distribution function
            y = z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        elif case["act"] == "silu":
            y = z * torch.sigmoid(z)
        if case["residual"]:
            y = y + s["residual"].double()
        return {"out": y, "preact": z} if case["preact"] else {"out": y}
    if op == "backward":
        x, z = s["x"], s["preact"]
        if case["saved8"]:
            x, z = _value8(x), None if z is None else _value8(z)
        g = s["d_out"].double()
        if z is not None:
            z = z.double().requires_grad_(True)     # the slope from differentiation
            if case["act"] == "relu":
                y = torch.maximum(z, torch.zeros_like(z))
                slope = (z.detach() > 0).double()
            else:
                y = z * (0.5 * torch.special.erfc(-z / math.sqrt(2.0)) if case["act"] == "gelu" else torch.sigmoid(z))
                (slope,) = torch.autograd.grad(y.sum(), z)
            g = g * slope.detach()
        out = {"d_x": torch.matmul(s["weight"].double().mT.contiguous(), g.mT.contiguous()).mT,
               "d_weight": torch.matmul(x.double().mT.contiguous(), g).mT}
        if case["bias"]:
            out["d_bias"] = torch.matmul(torch.ones(1, case["n"], dtype=torch.float64, device=DEV), g).view(-1)
        return out
    if op == "checkpoint":
        x = s["x"].double()
        n, d = x.shape
        short = -d % BLOCK
        x = torch.cat([x, x.new_zeros(n, short)], 1).view(n, -1, BLOCK)
        most = x.abs().amax(2, keepdim=True)
        # the smallest power of two that brings the block within 448
        unit = torch.exp2(torch.ceil(torch.log2(most / 448)).clamp(min=-15 if case["type"] == "fp16" else -117))
        v = x / unit
        # numbers with 4 significant bits, at least 2^-9 apart; a tie goes to the even one
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        v = torch.round(v / step) * step * unit
        lim = torch.finfo(TYPES[case["type"]]).max
        return v.reshape(n, -1)[:, :d].clamp(-lim, lim)
    if op == "select":
        return _exact_select(s, case)
    out = []
    at = (torch.arange(case["n_seq"], device=DEV).view(-1, 1) * case["beams"] + s["parents"]).flatten()
    for src in s["states"]:
        dst = torch.zeros(src.shape, dtype=torch.float64, device=DEV)
        dst.narrow(2, 0, case["length"]).copy_(src.index_select(0, at).narrow(2, 0, case["length"]))
        out.append(dst)
    return out


def _value8(p):
    """What the codes stand for, from their bits: 1 sign, 4 exponent (bias 7), 3 fraction."""
    c = p["codes"].long()
    field, frac = (c >> 3) & 15, (c & 7).double()
    v = torch.where(field == 0, frac * 2.0 ** -9, (8 + frac) * torch.exp2(field.double() - 10))
    v = torch.where(c >= 128, -v, v)
    block = torch.arange(c.shape[1], device=DEV) // BLOCK
    v = v * torch.exp2(p["scales"].double() - 127)[:, block]
    most = torch.finfo(p["type"]).max
    return v.clamp(-most, most)


def _exact_select(s, case):
    """Row by row: the candidates of a sequence in order, the first n_out of them."""
    n_seq, beams, vocab, n_out = case["n_seq"], case["beams"], case["vocab"], case["n_out"]
    out = {"scores": [], "parents": [], "tokens": []}
    if case["finished"]:
        out["finished"] = []
    for q in range(n_seq):
        score, place = [], []
        for k in range(beams):
            base = s["scores"][q, k].double()
            if case["finished"] and bool(s["finished"][q, k]):
                score.append(base.view(1))
                place.append(torch.tensor([k * vocab + _eos(case)], device=DEV))
                continue
            x = s["logits"][q * beams + k].double()
            ids = torch.arange(vocab, device=DEV)
            if case["allowed"]:
                ids = ids[s["allowed"][q * beams + k]]
                x = x[ids]
            if x.numel() == 0:
                continue
            logp = x - torch.logsumexp(x, 0)
            # a beam gives n_out candidates at most: its best logits, equal ones by token
            order = torch.sort(logp, dim=0, descending=True, stable=True).indices[:n_out]
            score.append(base + logp[order])
            place.append(k * vocab + ids[order])
        score = torch.cat(score) if score else torch.zeros(0, dtype=torch.float64, device=DEV)
        place = torch.cat(place) if place else torch.zeros(0, dtype=torch.int64, device=DEV)
        order = torch.sort(score, dim=0, descending=True, stable=True).indices[:n_out]
        score, place = score[order], place[order]
        short = n_out - score.numel()
        parents = torch.cat([place // vocab, place.new_full((short,), -1)])
        tokens = torch.cat([place % vocab, place.new_full((short,), -1)])
        out["scores"].append(torch.cat([score, score.new_full((short,), -math.inf)]))
        out["parents"].append(parents)
        out["tokens"].append(tokens)
        if case["finished"]:
            out["finished"].append(tokens == _eos(case))
    return {k: torch.stack(v) for k, v in out.items()}
