"""Plain 64-bit forms of the operators around token IDs, in numpy, written
from the formulas of include/toktier.h, and the error bounds the tests use."""
import math
from fractions import Fraction

import numpy as np

EPS = 2.0**-24                                             # unit roundoff of float
UNIT = {"float32": 2.0**-24, "float16": 2.0**-11, "bfloat16": 2.0**-8}
TINY = {"float32": 2.0**-140, "float16": 2.0**-24, "bfloat16": 2.0**-130}   # spacing of the least values


def embed(ids, table, scale):
    out = np.zeros((len(ids), table.shape[1]))
    there = ids >= 0
    out[there] = table[ids[there]] * scale
    return out


def embed_grad(ids, dout, n_vocab, scale):
    """(sums, sums of absolute terms, number of terms a row)."""
    g, m, c = np.zeros((n_vocab, dout.shape[1])), np.zeros((n_vocab, dout.shape[1])), np.zeros(n_vocab)
    for i, v in enumerate(ids):
        if 0 <= v < n_vocab:
            g[v] += dout[i]
            m[v] += np.abs(dout[i])
            c[v] += 1
    return g * scale, m * abs(scale), c


def token_loss(x, targets, g):
    """(loss, lse, dlogits) of finite or -inf logits."""
    with np.errstate(all="ignore"):
        m = x.max(1)
        lse = np.where(m == -np.inf, -np.inf, m + np.log(np.exp(x - np.where(m == -np.inf, 0, m)[:, None]).sum(1)))
        n, v = x.shape
        there = (targets >= 0) & (targets < v)
        t = np.where(there, targets, 0)
        loss = np.where(lse == -np.inf, np.inf, lse - x[np.arange(n), t])
        loss = np.where(there, loss, 0.0)
        d = np.exp(x - lse[:, None])
        d[np.arange(n), t] -= 1
        d *= g[:, None]
        d[~there | (lse == -np.inf)] = 0
    return loss, lse, d


def lse_bound(x, lse):
    """A float's error in lse: its own rounding and the maximum's; exp and its
    argument a few roundings (the argument's error is at most |l - M| EPS, and
    |l - M| exp(l - M) < 0.4); a sum of 512 or more interleaved parts."""
    return EPS * (2 * np.abs(lse) + 2 * np.abs(x.max(1)) + 16 + x.shape[1] / 128)


def sample_weights(x, t, exp2):
    """The weights as header states them: the exponent in floats, the power by
    `exp2` (float array to float array), whole numbers of 2^-40."""
    x = np.where(np.isnan(x), -np.inf, x).astype(np.float32)
    with np.errstate(all="ignore"):
        m = x.max()
        c = np.minimum(np.float32(1.4426950408889634) / np.float32(t), np.float32(3.4028234663852886e38))
        y = np.where(x == m, np.float32(0), (m - x) * c).astype(np.float32)
        w = np.rint(exp2(-y).astype(np.float64) * 2.0**40)
    return np.where(x == -np.inf, 0, w).astype(np.int64)


def sample(w, u, t=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(ID, logprob) from a row's whole-number weights."""
    if not w.any():
        return -1, -math.inf
    order = np.argsort(-w, kind="stable")
    order = order[: 1 if t == 0 else top_k if top_k > 0 else len(w)]
    order = order[(w[order] > 0) & (w[order] >= float(np.float32(min_p)) * 2.0**40)]
    c = np.cumsum(w[order])
    least = max(1, math.ceil(Fraction(float(np.float32(top_p))) * int(c[-1])))
    order = np.sort(order[: 1 + int(np.searchsorted(c, least, side="left"))])
    c = np.cumsum(w[order])
    r = math.floor(Fraction(float(np.float32(u))) * int(c[-1]))
    i = int(np.searchsorted(c, r, side="right"))
    return int(order[i]), math.log(int(w[order[i]]) / int(c[-1]))
