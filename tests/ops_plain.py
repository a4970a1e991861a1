"""Plain 64-bit forms of the operators next to the losses: torch float64 for
the linear layer (on whatever device its inputs are), numpy for the others."""
import math

import numpy as np
import torch

ACTS = ("none", "relu", "gelu", "silu")


def act(z, name):
    if name == "relu":
        return z.clamp(min=0.0)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z / math.sqrt(2.0)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return (0.5 * (1.0 + torch.erf(z / math.sqrt(2.0)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def linear(x, w, b=None, r=None, name="none"):
    z = x @ w.T
    if b is not None:
        z = z + b
    y = act(z, name)
    return (y if r is None else y + r), z


def linear_backward(dy, x, w, z, name):
    g = dy if name == "none" else dy * act_slope(z, name)
    return g @ w, g.T @ x, g.sum(0), g


def round_e4m3(v):
    """Nearest number with 4 significant bits, at least 2^-9 apart (|v| <= 448)."""
    a = np.maximum(np.abs(v), 2.0 ** -6)
    step = 2.0 ** (np.floor(np.log2(a)) - 3)
    return np.rint(v / step) * step


def checkpoint(x, most, lowest):
    """(values a checkpoint of x stands for, exponents of its scales)."""
    n, d = x.shape
    nb = -(-d // 32)
    p = np.zeros((n, nb * 32))
    p[:, :d] = x
    p = p.reshape(n, nb, 32)
    fin = np.where(np.isfinite(p), np.abs(p), 0.0)
    amax = fin.max(2)
    e = np.full((n, nb), lowest, dtype=np.int64)
    nz = amax > 0
    m, k = np.frexp(amax)          # amax = m 2^k, m in [1/2, 1): 448 = 7/8 2^9
    e[nz] = np.maximum(k[nz] - 9 + (m[nz] > 0.875), lowest)
    unit = 2.0 ** e[:, :, None].astype(np.float64)
    v = np.where(np.isfinite(p), round_e4m3(np.where(np.isfinite(p), p, 0.0) / unit) * unit, np.nan)
    v = np.clip(v, -most, most)
    return v.reshape(n, -1)[:, :d], e


def beam_select(x, scores, n_out, finished=None, allowed=None, eos=-1):
    """x [n_seq*beams][vocab] in fp64: (scores, parents, tokens, finished)."""
    n_seq, beams = scores.shape
    V = x.shape[1]
    S = np.full((n_seq, n_out), -np.inf)
    P = np.full((n_seq, n_out), -1, dtype=np.int64)
    T = np.full((n_seq, n_out), -1, dtype=np.int64)
    for q in range(n_seq):
        cands = []
        for k in range(beams):
            s = float(scores[q, k])
            if not math.isfinite(s):
                continue
            if finished is not None and finished[q, k]:
                cands.append((-s, k * V + eos))
                continue
            ids = np.arange(V)
            row = x[q * beams + k]
            if allowed is not None:
                ids = ids[allowed[q * beams + k] != 0]
            row = row[ids]
            if row.size == 0 or np.isnan(row).any() or row.max() in (np.inf, -np.inf):
                continue
            m = row.max()
            logp = row - (m + math.log(math.fsum(np.exp(row - m))))
            order = np.lexsort((ids, -row))[:n_out]
            cands += [(-(s + logp[i]), k * V + int(ids[i])) for i in order if row[i] > -np.inf]
        cands.sort()
        for j, (s, place) in enumerate(cands[:n_out]):
            S[q, j], P[q, j], T[q, j] = -s, place // V, place % V
    return S, P, T, (T == eos) & (T >= 0)
