"""Text to a small trained model and back, all on the GPU.

A bigram model (a vector a token, a projection to the vocabulary) is trained on
the token IDs of synthetic transcripts and then continues them:

  Tokenizer.encode   text -> IDs, their count on the device
  embed              IDs -> vectors, by the count that the encode left
  token_loss         logits and the next IDs -> losses, and the logits' gradient in place
  embed_grad         the vectors' gradient -> the table's
  sample             logits -> new IDs, from given random numbers

The two matrix products between them are torch's.

  python examples/bigram.py [--steps 60] [--tokens 64]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from exact_bpe_tokenization_gb300 import binding as tt  # noqa: E402
from exact_bpe_tokenization_gb300 import synth  # noqa: E402


def encode(tok, requests):
    """(ids, targets): the IDs of all requests, and each one's successor, with
    padding (-1) at the requests' ends."""
    data, offsets = synth.batch(requests)
    ids, io = tok.encode(torch.from_numpy(data).cuda(), torch.from_numpy(offsets).cuda())
    io = io.cpu()
    n = int(io[-1])
    targets = torch.empty(n, dtype=torch.int32, device="cuda")
    targets[:-1] = ids[1:n]
    ends = io[1:][io[1:] > io[:-1]] - 1
    targets[ends.cuda()] = -1
    return ids[:n], targets


def train(ids, targets, vocab, dim=64, steps=60, rate=20.0, seed=0):
    """(table, projection, losses)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    table = torch.randn(vocab, dim, generator=g, device="cuda") * 0.1
    proj = torch.randn(dim, vocab, generator=g, device="cuda") * 0.1
    count = int((targets >= 0).sum())
    row_grads = torch.full((len(ids),), 1.0 / count, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    losses = []
    for _ in range(steps):
        x = tt.embed(ids, table, status=status)
        logits = x @ proj
        loss, _, dlogits = tt.token_loss(logits, targets, row_grads=row_grads, dlogits=logits, status=status)
        dx = dlogits @ proj.T
        proj -= rate * (x.T @ dlogits)
        tt.embed_grad(ids, dx, vocab, scale=-rate, out=table, accumulate=True, status=status)   # the step itself
        losses.append(loss.sum() / count)
    if status.item() != tt.TT_OK:
        raise tt.TokTierError(status.item(), "training")
    return table, proj, torch.stack(losses).cpu()


def generate(table, proj, start, tokens, seed=1, temperature=0.8, top_k=40, top_p=0.95):
    """`tokens` IDs after each of `start`: [len(start), tokens]."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = len(start)
    full = lambda v, t: torch.full((n,), v, dtype=t, device="cuda")  # noqa: E731
    t, k, p = full(temperature, torch.float32), full(top_k, torch.int32), full(top_p, torch.float32)
    out = []
    ids = start
    for _ in range(tokens):
        ids, _ = tt.sample(tt.embed(ids, table) @ proj, torch.rand(n, generator=g, device="cuda"), t, k, p)
        out.append(ids)
    return torch.stack(out, 1)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args(argv)
    merges, vb, vo = synth.make_vocab(synth.PROFILE_ASCII, 1 << 20, 1000)
    vocab = len(vo) - 1
    tok = tt.Tokenizer(merges, vb, vo, tt.TT_FAMILY_CL100K_STYLE)
    ids, targets = encode(tok, [synth.transcript(1 + i, 20000, synth.PROFILE_ASCII) for i in range(4)])
    table, proj, losses = train(ids, targets, vocab, steps=a.steps)
    print("%d tokens, %d IDs; loss %.3f at first, %.3f after %d steps (uniform: %.3f)" % (
        len(ids), vocab, losses[0], losses[-1], a.steps, np.log(vocab)))
    drawn = generate(table, proj, ids[:2], a.tokens).cpu().numpy()
    for row in drawn:
        print(b"".join(bytes(vb[vo[i]:vo[i + 1]]) for i in row).decode("utf-8", "replace"))
    tok.close()
    return losses, drawn


if __name__ == "__main__":
    main()
