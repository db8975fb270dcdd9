"""The operators around token IDs: what is timed, on which inputs, and their plain forms.

  embed       rows of an embedding table gathered by token ID and scaled
  embed_grad  its gradient: the rows of dout summed by token ID into a dense table
  loss        next-token loss of each row of logits, with the logits' gradient
  sample      one token ID a row of logits: temperature, top-k, min-p, top-p, drawn with a given random number

`run` calls exact_bpe_tokenization_gb300.binding where `own` is true, else the plain forms below.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
LOG2E = 1.4426950408889634
FLT_MAX = 3.4028234663852886e38


def listed():
    """Vocabularies of 4,352, 100,256 and 200,256 IDs (256 bytes and 4,096, 100,000 or 200,000 merges) and
    the token counts of a 64 KB request (16,400) and of a 1M-character request (304,824) are the workloads'."""
    return [
        # the new tokens of a decoding batch: latency
        dict(name="embed_decode_64", op="embed", n=64, vocab=100256, dim=2048, type="bf16", out="bf16"),
        # a ragged pack of rows whose width fits no vector, 32-bit table into a 16-bit activation
        dict(name="embed_odd_8191x641", op="embed", n=8191, vocab=200256, dim=641, type="f32", out="bf16"),
        # the prefill of one 1M-character request
        dict(name="embed_1m_request", op="embed", n=304824, vocab=100256, dim=4096, type="bf16", out="bf16"),
        # a training step on one 64 KB request, everything in 32 bits
        dict(name="embed_grad_64k_request", op="embed_grad", n=16400, vocab=4352, dim=1024, type="f32", out="f32"),
        # few tokens into a large table: most rows are zero; a width that fits no vector
        dict(name="embed_grad_odd_8191x641", op="embed_grad", n=8191, vocab=200256, dim=641, type="bf16", out="bf16"),
        # a training step on a 1M-character request, 16-bit gradients into a 32-bit table
        dict(name="embed_grad_1m_request", op="embed_grad", n=304824, vocab=100256, dim=2048, type="bf16", out="f32"),
        # a small model's step
        dict(name="loss_small_64", op="loss", n=64, vocab=4352, type="f32"),
        # a training micro-batch
        dict(name="loss_batch_4096", op="loss", n=4096, vocab=100256, type="bf16"),
        # a large vocabulary of odd size, 32-bit logits (scoring, distillation)
        dict(name="loss_odd_1023", op="loss", n=1023, vocab=200255, type="f32"),
        # one request decoding: latency
        dict(name="sample_single", op="sample", n=1, vocab=100256, type="bf16"),
        # a serving batch, 32-bit logits of odd size
        dict(name="sample_odd_37", op="sample", n=37, vocab=200255, type="f32"),
        # a full serving batch
        dict(name="sample_batch_256", op="sample", n=256, vocab=100256, type="bf16"),
    ]


def log_int(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "loss", "sample"])
    vocab = rng.choice([4352, 100256, 200256, log_int(rng, 300, 200256)])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op in ("embed", "embed_grad"):
        dim = rng.choice([8 * log_int(rng, 8, 512), log_int(rng, 64, 4096)])
        if dim == 3 * 1024:
            dim -= 8
        if op == "embed_grad":  # no more than 1.6 GB for the whole table
            dim = min(dim, 400_000_000 // vocab)
        n = log_int(rng, 1, min(304824, (300_000_000 if op == "embed" else 120_000_000) // dim))
        return dict(op=op, n=n, vocab=vocab, dim=dim, type=kind, out=rng.choice([kind, "f32"]))
    if op == "loss":
        return dict(op=op, n=log_int(rng, 1, min(8192, 100_000_000 // vocab)), vocab=vocab, type=kind)
    return dict(op=op, n=log_int(rng, 1, 256), vocab=vocab, type=kind)


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
    s = {"op": case["op"]}
    if case["op"] in ("embed", "embed_grad"):
        s["ids"] = zipf_ids(n, vocab, g)
        rows = vocab if case["op"] == "embed" else n
        x = torch.empty(rows, case["dim"], device="cuda", dtype=t)
        for a in range(0, rows, 65536):
            x[a:a + 65536] = torch.randn(min(65536, rows - a), case["dim"], generator=g, device="cuda") * 0.02
        return {**s, "x": x, "vocab": vocab, "scale": math.sqrt(case["dim"]), "out": TYPES[case["out"]]}
    # logits: a spread bulk, and a few dozen tokens above it, as a trained model gives
    x = torch.empty(n, vocab, device="cuda", dtype=t)
    for a in range(0, n, 256):
        m = min(256, n - a)
        y = torch.randn(m, vocab, generator=g, device="cuda") * 2
        top = (torch.arange(48, device="cuda") + 0.999 * rand(m, 48)).mul_(vocab // 48).long()  # all different
        x[a:a + m] = y.scatter(1, top, 6 + 8 * rand(m, 48))
    s["x"] = x
    if case["op"] == "loss":
        s["targets"] = (rand(n) * vocab).to(torch.int32).clamp_(max=vocab - 1)
        s["targets"][rand(n) < 1 / 64] = -1
        s["grads"] = torch.full((n,), 1.0 / n, device="cuda")
        return s
    # sampling parameters as requests carry them: some greedy, some with filters off, some under a grammar's mask
    pick = lambda values, dt: torch.tensor(values, device="cuda", dtype=dt)[(rand(n) * len(values)).long().clamp_(max=len(values) - 1)]  # noqa: E731
    s["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.3], torch.float32)
    s["top_k"] = pick([0, 0, 1, 20, 50, 1000], torch.int32)
    s["top_p"] = pick([1.0, 0.8, 0.9, 0.95], torch.float32)
    s["min_p"] = pick([0.0, 0.0, 0.0, 0.05], torch.float32)
    s["uniform"] = rand(n)
    allowed = (rand(n, 24) * vocab).long().clamp_(max=vocab - 1)
    masked = torch.arange(n, device="cuda") % 16 == 7
    x[masked] = torch.full_like(x[masked], -math.inf).scatter(1, allowed[masked], x[masked].gather(1, allowed[masked]))
    return s


def embed_plain(ids, table, scale, out):
    there = (ids >= 0)[:, None]
    return torch.where(there, table[ids.long().clamp(min=0)].float() * scale, 0.0).to(out)


def embed_grad_plain(ids, dout, vocab, scale, out):
    there = ids >= 0
    g = torch.zeros(vocab, dout.shape[1], device=dout.device)
    g.index_add_(0, ids.long().clamp(min=0), torch.where(there[:, None], dout.float(), 0.0))
    return (g * scale).to(out)


def loss_plain(x, targets, grads):
    there = targets >= 0
    t = targets.long().clamp(min=0)[:, None]
    v = x.float()
    m = v.amax(1, keepdim=True)
    e = torch.exp(v - m)
    z = e.sum(1, keepdim=True)
    lse = (m + torch.log(z))[:, 0]
    loss = torch.where(there, lse - v.gather(1, t)[:, 0], 0.0)
    d = e / z
    d.scatter_add_(1, t, torch.full_like(t, -1, dtype=torch.float32))
    d *= torch.where(there, grads, 0.0)[:, None]
    return loss, lse, d.to(x.dtype)


def sample_plain(x, uniform, temperature, top_k, top_p, min_p):
    """Weights are whole numbers of 2^-40 of the largest, so that their sums are the same in every order."""
    v = torch.where(torch.isnan(x), -math.inf, x.float())
    m = v.amax(1, keepdim=True)
    c = (torch.full_like(temperature, LOG2E) / temperature).clamp(max=FLT_MAX)[:, None]
    y = torch.where(v == m, 0.0, (m - v) * c)
    w = torch.round(torch.exp2(-y) * 2.0**40)
    w = torch.where(v == -math.inf, 0.0, w).to(torch.int64)
    ws, order = torch.sort(w, dim=1, descending=True, stable=True)
    at = torch.arange(x.shape[1], device=x.device)[None]
    k = torch.where(temperature == 0, 1, torch.where(top_k > 0, top_k, x.shape[1])).long()[:, None]
    ws = torch.where((at < k) & (ws >= torch.ceil(min_p.double() * 2.0**40).long()[:, None]), ws, 0)
    cum = ws.cumsum(1)
    least = torch.ceil(top_p.double() * cum[:, -1].double()).long().clamp(min=1)[:, None]
    ws = torch.where(cum - ws < least, ws, 0)
    kept = torch.zeros_like(w).scatter_(1, order, ws)
    cum = kept.cumsum(1)
    total = cum[:, -1]
    r = torch.floor(uniform.double() * total.double()).long()
    ids = (cum <= r[:, None]).sum(1)
    one = kept.gather(1, ids.clamp(max=x.shape[1] - 1)[:, None])[:, 0]
    logp = torch.log((one.double() / total.double()).float())
    empty = total == 0
    return torch.where(empty, -1, ids).to(torch.int32), torch.where(empty, -math.inf, logp)


def run(s):
    if own:
        from exact_bpe_tokenization_gb300 import binding as tt
        if s["op"] == "embed":
            return tt.embed(s["ids"], s["x"], scale=s["scale"], dtype=s["out"])
        if s["op"] == "embed_grad":
            return tt.embed_grad(s["ids"], s["x"], s["vocab"], scale=s["scale"], dtype=s["out"])
        if s["op"] == "loss":
            return tt.token_loss(s["x"], s["targets"], row_grads=s["grads"], want_grad=True)
        return tt.sample(s["x"], s["uniform"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    if s["op"] == "embed":
        return embed_plain(s["ids"], s["x"], s["scale"], s["out"])
    if s["op"] == "embed_grad":
        return embed_grad_plain(s["ids"], s["x"], s["vocab"], s["scale"], s["out"])
    if s["op"] == "loss":
        return loss_plain(s["x"], s["targets"], s["grads"])
    return sample_plain(s["x"], s["uniform"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])


def work(case):
    n, vocab, e = case["n"], case["vocab"], SIZE[case["type"]]
    if case["op"] in ("embed", "embed_grad"):
        dim, o = case["dim"], SIZE[case["out"]]
        if case["op"] == "embed":  # the distinct rows that n draws touch, on average
            p = np.arange(1, vocab + 1, dtype=np.float64) ** -1.1
            rows = float(np.sum(-np.expm1(n * 63 / 64 * np.log1p(-p / p.sum()))))
            return {"bytes": 4 * n + rows * dim * e + n * dim * o, "flops": n * dim}
        return {"bytes": 4 * n + n * dim * e + vocab * dim * o, "flops": n * dim + vocab * dim}
    if case["op"] == "loss":
        return {"bytes": 2 * n * vocab * e + 16 * n, "flops": 7 * n * vocab}
    return {"bytes": n * vocab * e + 28 * n, "flops": 8 * n * vocab}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "embed":
        x = s["x"].double() if s["x"].numel() < 1 << 28 else None
        rows = []
        for a in range(0, len(s["ids"]), 65536):
            i = s["ids"][a:a + 65536].long()
            r = (x[i] if x is not None else s["x"][i].double()).mul_(s["scale"])
            r[i < 0] = 0
            rows.append(r)
        return torch.cat(rows)
    if s["op"] == "embed_grad":
        # differences of running sums over the tokens in the order of their IDs
        ids, order = torch.sort(s["ids"].long())
        ends = torch.searchsorted(ids, torch.arange(-1, s["vocab"], device="cuda"), right=True)
        out = torch.empty(s["vocab"], s["x"].shape[1], device="cuda", dtype=torch.float64)
        for a in range(0, out.shape[1], 128):
            c = torch.zeros(len(ids) + 1, min(128, out.shape[1] - a), device="cuda", dtype=torch.float64)
            c[1:] = s["x"][:, a:a + 128][order].double().cumsum(0)
            out[:, a:a + 128] = (c[ends[1:]] - c[ends[:-1]]) * s["scale"]
        return out
    if s["op"] == "loss":
        loss, lse, grads = [], [], []
        for a in range(0, case["n"], 1024):
            x, t = s["x"][a:a + 1024].double(), s["targets"][a:a + 1024].long()
            z = torch.logsumexp(x, 1)
            i = torch.arange(len(t), device="cuda")[t >= 0]
            one = torch.zeros_like(z)
            one[i] = z[i] - x[i, t[i]]
            p = x.sub_(z[:, None]).exp_()
            p[i, t[i]] -= 1
            p *= s["grads"][a:a + 1024].double()[:, None]
            p[t < 0] = 0
            loss.append(one)
            lse.append(z)
            grads.append(p)
        return torch.cat(loss), torch.cat(lse), torch.cat(grads)
    ids, logps = [], []
    x, t, k, p, mp, u = (s[n].double().cpu().numpy() for n in ("x", "temperature", "top_k", "top_p", "min_p", "uniform"))
    for r in range(case["n"]):
        w = 2.0**40 * (x[r] == x[r].max()) if t[r] == 0 else np.rint(np.exp((x[r] - x[r].max()) / t[r]) * 2.0**40)
        order = np.argsort(-w, kind="stable")
        order = order[:1 if t[r] == 0 else int(k[r]) if k[r] > 0 else len(order)]
        order = order[w[order] >= max(1, mp[r] * 2.0**40)]
        c = np.cumsum(w[order])
        order = np.sort(order[:1 + int(np.searchsorted(c, p[r] * c[-1]))])
        c = np.cumsum(w[order])
        i = int(np.searchsorted(c, math.floor(u[r] * c[-1]), side="right"))
        ids.append(order[i])
        logps.append(math.log(w[order[i]] / c[-1]))
    return np.array(ids, dtype=np.int32), np.array(logps)
