"""Plain 64-bit forms of the losses of a model's head (tt_linear_loss, tt_distill_loss),
written from the formulas of include/toktier.h in torch doubles, with the error bounds
that the tests use.  They run where their tensors are."""
import torch

EPS = 2.0**-24                                             # unit roundoff of float
UNIT = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
# half the spacing of the least values
TINY = {torch.float32: 2.0**-149, torch.float16: 2.0**-25, torch.bfloat16: 2.0**-134}


def product_bound(absolute, k, kind):
    """The error of a tensor core's product over k, given the sum of its terms'
    absolute values.  Sixteen terms are added to the sum at a time; each such step is
    taken to keep 22 bits of the largest value that meets in it, which the sum of
    absolute values is not below.  32-bit operands: three parts each, products of
    parts below 2^-24 left out (three of those, and the parts' own remainder)."""
    steps = (k + 15) // 16 + 2
    if kind == torch.float32:
        # six products, five of them 2^-8 of the first or less, added first
        return absolute * (steps * 2.0**-22 * (1 + 5 * 2.0**-8) + 5 * 2.0**-24)
    return absolute * (steps * 2.0**-22)


def linear(h, w, targets, g):
    """(loss, lse, dhidden, dweight) and what the bounds need."""
    kind = h.dtype
    h, w, g = h.double(), w.double(), g.double()
    logits = h @ w.T
    lse = torch.logsumexp(logits, 1)
    there = (targets >= 0) & (targets < w.shape[0])
    t = torch.where(there, targets, 0).long()[:, None]
    lt = logits.gather(1, t)[:, 0]
    loss = torch.where(there, lse - lt, 0.0)
    p = torch.exp(logits - lse[:, None])
    one = torch.zeros_like(p).scatter_(1, t, 1.0)
    G = (p - one) * torch.where(there, g, 0.0)[:, None]
    return dict(kind=kind, h=h, w=w, g=torch.where(there, g, 0.0), logits=logits, p=p, G=G,
                loss=loss, lse=lse, dh=G @ w, dw=G.T @ h)


def linear_bounds(r):
    """Bounds of the errors of loss, lse, dhidden and dweight (in 32 bits, before the
    gradients are rounded to their type)."""
    kind, h, w = r["kind"], r["h"], r["w"]
    (n, dim), vocab = h.shape, w.shape[0]
    logit = product_bound(h.abs() @ w.abs().T, dim, kind)  # of each logit
    worst = logit.amax(1)
    # lse: the logits' errors, its own rounding and the maximum's, exp and its argument a
    # few roundings, a sum of interleaved parts
    lse = worst + EPS * (2 * r["lse"].abs() + 4 * r["logits"].abs().amax(1) + 24 + vocab / 64)
    loss = 2 * worst + lse
    # a probability: its logit's error and lse's, exp's argument; what rounds G, a row's factor
    # (which may make up for its target's rounding, of as much), and for dweight the factor's
    # product with hidden
    p = r["p"] * torch.expm1(logit + (lse + 2 * worst + EPS * (4 * r["logits"].abs().amax(1) + 8))[:, None])
    dG = p * r["g"].abs()[:, None] + r["G"].abs() * (4 * EPS)
    unit = UNIT[kind] if kind != torch.float32 else 0.0
    # scaled 16-bit floats: what lies below their least values
    low = r["g"].abs().max() * 2.0**-37 if kind == torch.float16 else 0.0
    over_h = dG + r["G"].abs() * (2 * unit + unit * unit) + low
    over_w = dG + r["G"].abs() * (3 * unit + 4 * unit * unit) + low
    dh = over_h @ w.abs() + product_bound(r["G"].abs() @ w.abs(), vocab, kind) * 1.01
    dw = over_w.T @ h.abs() + product_bound(r["G"].abs().T @ h.abs(), n, kind) * 1.01
    return loss, lse, dh, dw


def rounded(bound, want, kind):
    """A bound once the value is rounded to a type."""
    return bound * 1.01 + UNIT[kind] * want.abs() * 1.01 + TINY[kind]


def distill(x, ids, values, temperature, g):
    """(loss, lse, dlogits), bounds of their errors in 32 bits; finite or -inf logits,
    a row of which is not -inf throughout."""
    y, v = x.double() / temperature, values.double() / temperature
    n, vocab = y.shape
    lse = torch.logsumexp(y, 1)
    there = (ids >= 0) & (ids < vocab)
    v = torch.where(there, v, -torch.inf)
    some = (v > -torch.inf).any(1)
    v = torch.where(some[:, None], v, 0.0)
    logq = torch.log_softmax(v, 1)
    q = torch.where(there & some[:, None], logq.exp(), 0.0)
    at = torch.where(there, ids, 0).long()
    yt = y.gather(1, at)
    loss = torch.where(q > 0, q * (logq - yt + lse[:, None]), 0.0).sum(1)
    p = torch.exp(y - lse[:, None])
    share = torch.zeros_like(y).scatter_add_(1, at, q)
    gt = torch.where(some, g.double() / temperature, 0.0)[:, None]
    d = (p - share) * gt
    top = y.amax(1)
    far = torch.where(y > -torch.inf, (y - top[:, None]).abs(), 0.0)
    # exp's argument is off by a few roundings of itself (|a| exp(-|a|) < 0.4), sums of
    # interleaved parts
    sums = EPS * (24 + vocab / 64)
    e_lse = sums + EPS * (2 * lse.abs() + 2 * top.abs())
    vf = torch.where(v > -torch.inf, (v - v.amax(1, keepdim=True)).abs(), 0.0)
    e_q = q * EPS * (4 * vf + 24 + ids.shape[1] / 8)
    term = torch.where(q > 0, (logq - yt + lse[:, None]).abs(), 0.0)
    away = torch.where(q > 0, (yt - top[:, None]).abs() + vf, 0.0)
    e_loss = (e_q * term + q * (EPS * (4 * away + 8) + sums)).sum(1) + EPS * (q * term).sum(1) * (4 + ids.shape[1] / 8)
    e_share = torch.zeros_like(y).scatter_add_(1, at, e_q) + share * EPS * ids.shape[1]
    e_d = (p * (EPS * (4 * far + 8) + sums) + e_share) * gt.abs() + d.abs() * 4 * EPS
    return (loss, lse, d), (e_loss, e_lse, e_d)
