"""The losses of a language model's head: what is timed, on which inputs, and their plain forms.

  linear   next-token loss of hidden states through the head's weight, the logits not kept;
           with the gradients of both, or the loss and lse alone
  distill  Kullback-Leibler divergence from a teacher's top logits of each row of logits;
           with the logits' gradient, or the loss and lse alone

`run` calls exact_bpe_tokenization_gb300.binding where `own` is true, else the plain forms below.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    """Vocabularies of 4,352, 100,256 and 200,256 IDs (256 bytes and 4,096, 100,000 or 200,000 merges) and
    the token count of a 64 KB request (16,400) are the workloads'."""
    return [
        # a step of the example's model: latency
        dict(name="linear_small_64", op="linear", n=64, vocab=4352, dim=64, type="f32", grad=True),
        # the log-probability of one given token: the head's weight is read once
        dict(name="linear_score_1", op="linear", n=1, vocab=100256, dim=2048, type="bf16", grad=False),
        # a 64 KB request scored (perplexity, reranking)
        dict(name="linear_score_64k_request", op="linear", n=16400, vocab=100256, dim=2048, type="bf16", grad=False),
        # a ragged pack against a large vocabulary of odd size; rows whose width fits no vector
        dict(name="linear_odd_1023x641", op="linear", n=1023, vocab=200255, dim=641, type="f16", grad=True),
        # a small model's step with everything in 32 bits
        dict(name="linear_f32_2047", op="linear", n=2047, vocab=4352, dim=1024, type="f32", grad=True),
        # a training micro-batch
        dict(name="linear_batch_4096", op="linear", n=4096, vocab=100256, dim=2048, type="bf16", grad=True),
        # a training step on a 64 KB request
        dict(name="linear_train_64k_request", op="linear", n=16400, vocab=100256, dim=2048, type="bf16", grad=True),
        # a small student's step: latency
        dict(name="distill_small_64", op="distill", n=64, vocab=4352, k=8, type="f32", teacher="f32", grad=True),
        # a training micro-batch, the teacher's answers stored in 16 bits
        dict(name="distill_batch_4096", op="distill", n=4096, vocab=100256, k=64, type="bf16", teacher="bf16", grad=True),
        # a large vocabulary of odd size, 32-bit logits
        dict(name="distill_odd_1023", op="distill", n=1023, vocab=200255, k=37, type="f32", teacher="f16", grad=True),
        # a student scored against many of the teacher's logits
        dict(name="distill_score_2048", op="distill", n=2048, vocab=100256, k=256, type="f16", teacher="f32", grad=False),
    ]


def log_int(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "distill"])
    vocab = rng.choice([4352, 100256, 200256, log_int(rng, 300, 200256)])
    kind = rng.choice(["f32", "f16", "bf16", "bf16"])
    grad = rng.random() < 0.6
    if op == "linear":
        dim = rng.choice([8 * log_int(rng, 8, 512), log_int(rng, 64, 4096)])
        dim = min(dim, 420_000_000 // vocab)
        # no more products than the largest listed case has, a sixth of them in 32 bits
        most = (500_000_000_000 if kind == "f32" else 3_000_000_000_000) // (vocab * dim)
        return dict(op=op, n=log_int(rng, 1, min(16400, max(1, most))), vocab=vocab, dim=dim, type=kind, grad=grad)
    return dict(op=op, n=log_int(rng, 1, min(8192, 400_000_000 // vocab)), vocab=vocab, k=log_int(rng, 1, 256), type=kind,
                teacher=rng.choice(["f32", kind]), grad=grad)


def zipf_ids(n, vocab, g):
    """IDs with Zipf(1.1) frequencies over a random order of the vocabulary; one in 64 is padding (-1)."""
    p = torch.arange(1, vocab + 1, device="cuda", dtype=torch.float64).pow(-1.1).cumsum(0)
    at = torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * p[-1]
    rank = torch.searchsorted(p, at).clamp_(max=vocab - 1)
    ids = torch.randperm(vocab, generator=g, device="cuda")[rank]
    ids[torch.rand(n, generator=g, device="cuda") < 1 / 64] = -1
    return ids.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n, vocab, t = case["n"], case["vocab"], TYPES[case["type"]]
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = {"op": case["op"], "grad": case["grad"]}
    if s["op"] == "linear":
        # logits with a spread of 2, and the target's up to 16 above, as a trained model gives
        dim = case["dim"]
        w = torch.empty(vocab, dim, device="cuda", dtype=t)
        for a in range(0, vocab, 65536):
            w[a:a + 65536] = randn(min(65536, vocab - a), dim) * (2 / math.sqrt(dim))
        s["targets"] = zipf_ids(n, vocab, g)
        h = torch.empty(n, dim, device="cuda", dtype=t)
        for a in range(0, n, 4096):
            to = s["targets"][a:a + 4096].long().clamp(min=0)
            h[a:a + 4096] = randn(len(to), dim) + w[to].float() * (4 * rand(len(to), 1))
        s["hidden"], s["weight"] = h, w
    else:
        # logits: a spread bulk, and a few dozen tokens above it; the teacher's are near the student's
        k, x = case["k"], torch.empty(n, vocab, device="cuda", dtype=t)
        s["ids"] = torch.empty(n, k, device="cuda", dtype=torch.int32)
        s["values"] = torch.empty(n, k, device="cuda", dtype=TYPES[case["teacher"]])
        for a in range(0, n, 256):
            m, top = min(256, n - a), max(48, k)
            y = randn(m, vocab) * 2
            at = (torch.arange(top, device="cuda") + 0.999 * rand(m, top)).mul_(vocab // top).long()  # all different
            high = 6 + 8 * rand(m, top)
            x[a:a + m] = y.scatter(1, at, high)
            best, order = torch.topk(high + randn(m, top), k, 1)
            s["values"][a:a + m] = best
            s["ids"][a:a + m] = at.gather(1, order).int()
        # answers cut short, and rows without one
        s["ids"][torch.arange(k, device="cuda")[None] >= torch.where(rand(n, 1) < 1 / 16, rand(n, 1) * k, k)] = -1
        s["ids"][rand(n) < 1 / 64] = -1
        s["logits"], s["temperature"] = x, 2.0
    s["grads"] = torch.full((n,), 1.0 / n, device="cuda")
    return s


def linear_plain(h, w, targets, grads, grad):
    n, vocab = h.shape[0], w.shape[0]
    w32 = w.float()
    loss, lse, dh = torch.empty_like(grads), torch.empty_like(grads), torch.empty_like(h)
    dw = torch.zeros_like(w32) if grad else None
    for a in range(0, n, 4096):
        h32, there = h[a:a + 4096].float(), targets[a:a + 4096] >= 0
        t = targets[a:a + 4096].long().clamp(min=0)[:, None]
        v = h32 @ w32.T
        m = v.amax(1, keepdim=True)
        vt = v.gather(1, t)
        e = v.sub_(m).exp_()
        z = e.sum(1, keepdim=True)
        lse[a:a + 4096] = (m + torch.log(z))[:, 0]
        loss[a:a + 4096] = torch.where(there, (m - vt + torch.log(z))[:, 0], 0.0)
        if grad:
            d = e.div_(z)
            d.scatter_add_(1, t, torch.full_like(t, -1, dtype=torch.float32))
            d *= torch.where(there, grads[a:a + 4096], 0.0)[:, None]
            dh[a:a + 4096] = (d @ w32).to(h.dtype)
            dw.addmm_(d.T, h32)
    return (loss, lse, dh, dw.to(w.dtype)) if grad else (loss, lse)


def distill_plain(x, ids, values, temperature, grads, grad):
    there = ids >= 0
    some = there.any(1)
    at = ids.long().clamp(min=0)
    tv = torch.where(there, values.float() / temperature, -math.inf)
    tv = torch.where(some[:, None], tv, 0.0)
    q = torch.softmax(tv, 1) * there
    logq = torch.log_softmax(tv, 1)
    v = x.float() / temperature
    m = v.amax(1, keepdim=True)
    vt = v.gather(1, at) - m
    e = v.sub_(m).exp_()
    z = e.sum(1, keepdim=True)
    lse = (m + torch.log(z))[:, 0]
    loss = torch.where(q > 0, q * (logq - vt + torch.log(z)), 0.0).sum(1)
    if not grad:
        return loss, lse
    d = e.div_(z)
    d.scatter_add_(1, at, -q)
    d *= torch.where(some, grads / temperature, 0.0)[:, None]
    return loss, lse, d.to(x.dtype)


def run(s):
    if own:
        from exact_bpe_tokenization_gb300 import binding as tt
        if s["op"] == "linear":
            return tt.linear_loss(s["hidden"], s["weight"], s["targets"], row_grads=s["grads"], want_grad=s["grad"])
        return tt.distill_loss(s["logits"], s["ids"], s["values"], temperature=s["temperature"], row_grads=s["grads"],
                               want_grad=s["grad"])
    if s["op"] == "linear":
        return linear_plain(s["hidden"], s["weight"], s["targets"], s["grads"], s["grad"])
    return distill_plain(s["logits"], s["ids"], s["values"], s["temperature"], s["grads"], s["grad"])


def work(case):
    n, vocab, e = case["n"], case["vocab"], SIZE[case["type"]]
    times = 1 + case["grad"]
    if case["op"] == "linear":
        # the logits, and with gradients one product for each of the two
        return {"bytes": times * (n + vocab) * case["dim"] * e + 16 * n, "flops": (1 + 2 * case["grad"]) * 2 * n * vocab * case["dim"]}
    return {"bytes": times * n * vocab * e + n * case["k"] * (4 + SIZE[case["teacher"]]) + 12 * n, "flops": 7 * n * vocab}


def exact(case, seed):
    if case["op"] == "linear" and work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    n, vocab = case["n"], case["vocab"]
    rows = max(1, 200_000_000 // vocab)
    parts = []
    if case["op"] == "linear":
        h, w = s["hidden"].double(), s["weight"].double()
        dw = torch.zeros_like(w) if s["grad"] else None
        for a in range(0, n, rows):
            x, t, g = h[a:a + rows], s["targets"][a:a + rows].long(), s["grads"][a:a + rows].double()
            y = torch.mm(x, w.t())
            z = torch.logsumexp(y, 1)
            i = (t >= 0).nonzero()[:, 0]
            one = torch.zeros_like(z)
            one[i] = z[i] - y[i, t[i]]
            part = [one, z]
            if s["grad"]:
                p = torch.zeros_like(y)
                p[i] = torch.exp(y[i] - z[i, None]) * g[i, None]
                p[i, t[i]] -= g[i]
                part.append(torch.mm(p, w))
                dw += torch.mm(p.t(), x)
            parts.append(part)
        out = [torch.cat(c) for c in zip(*parts)]
        return tuple(out + [dw] if s["grad"] else out)
    for a in range(0, n, rows):
        x = s["logits"][a:a + rows].double() / s["temperature"]
        z = torch.logsumexp(x, 1)
        ids, tv = s["ids"][a:a + rows].long(), s["values"][a:a + rows].double() / s["temperature"]
        loss, q = torch.zeros_like(z), torch.zeros_like(x)
        scale = torch.zeros_like(z)
        for j in range(len(ids)):
            at = ids[j][ids[j] >= 0]
            if len(at):
                logq = tv[j][ids[j] >= 0] - torch.logsumexp(tv[j][ids[j] >= 0], 0)
                loss[j] = torch.sum(torch.exp(logq) * (logq - x[j, at] + z[j]))
                q[j, at] = torch.exp(logq)
                scale[j] = s["grads"][a + j].double() / s["temperature"]
        part = [loss, z]
        if s["grad"]:
            part.append((torch.exp(x - z[:, None]) - q) * scale[:, None])
        parts.append(part)
    return tuple(torch.cat(c) for c in zip(*parts))
