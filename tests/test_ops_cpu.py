"""The operators around token IDs without a GPU: what their C entry points
refuse (before any device call), and the scratch that tt_embed_grad asks for.
Addresses are stand-ins: a refused call never uses them."""
import pytest

from exact_bpe_tokenization_gb300 import binding as tt
from exact_bpe_tokenization_gb300 import build

A, B, C, D = 1 << 20, 2 << 20, 3 << 20, 4 << 20       # aligned stand-in addresses


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def refused(call, status):
    with pytest.raises(tt.TokTierError) as e:
        call()
    assert e.value.status == status


EMBED = dict(ids=A, n=4, n_ids=None, table=B, tt_=tt.TT_BF16, vocab=300, dim=16, ts=16, scale=1.0, out=C, to=tt.TT_F32,
             os=16, status=None)


def embed(**kw):
    a = {**EMBED, **kw}
    tt.tt_embed(a["ids"], a["n"], a["n_ids"], a["table"], a["tt_"], a["vocab"], a["dim"], a["ts"], a["scale"], a["out"],
                a["to"], a["os"], a["status"], 0)


@pytest.mark.parametrize("bad", [
    dict(ids=None), dict(ids=A + 2), dict(n=-1), dict(n_ids=A + 4), dict(table=None), dict(table=B + 1), dict(tt_=3),
    dict(tt_=-1), dict(vocab=0), dict(vocab=(1 << 20) + 1), dict(dim=0), dict(ts=15), dict(out=None), dict(out=C + 2),
    dict(to=7), dict(os=15), dict(status=A + 2), dict(dim=1 << 31, ts=1 << 31, os=1 << 31),
])
def test_embed_refuses(bad):
    refused(lambda: embed(**bad), tt.TT_ERR_INVALID_ARG)


def test_too_many_rows_are_refused():
    more = tt.TT_MAX_IDS + 1
    refused(lambda: embed(n=more), tt.TT_ERR_CAPACITY)
    refused(lambda: grad(n=more), tt.TT_ERR_CAPACITY)
    refused(lambda: loss(n=more), tt.TT_ERR_CAPACITY)
    refused(lambda: loss_grad(n=more), tt.TT_ERR_CAPACITY)
    refused(lambda: sample(n=more), tt.TT_ERR_CAPACITY)


def test_calls_without_rows_do_nothing():
    embed(n=0, ids=None, table=None, out=None)
    loss(n=0, logits=None, targets=None, loss=None)
    loss_grad(n=0, logits=None, targets=None, lse=None, dlogits=None)
    sample(n=0, logits=None, uniform=None, ids=None)


GRAD = dict(ids=A, n=4, n_ids=None, dout=B, td=tt.TT_BF16, dim=16, ds=16, scale=1.0, dtable=C, tt_=tt.TT_F32, vocab=300,
            ts=16, acc=0, ws=D, wb=1 << 24, status=None)


def grad(**kw):
    a = {**GRAD, **kw}
    tt.tt_embed_grad(a["ids"], a["n"], a["n_ids"], a["dout"], a["td"], a["dim"], a["ds"], a["scale"], a["dtable"],
                     a["tt_"], a["vocab"], a["ts"], a["acc"], a["ws"], a["wb"], a["status"], 0)


@pytest.mark.parametrize("bad", [
    dict(ids=None), dict(ids=A + 1), dict(n=-1), dict(n_ids=A + 4), dict(dout=None), dict(dout=B + 1), dict(td=9),
    dict(dim=0), dict(ds=15), dict(dtable=None), dict(dtable=C + 2), dict(tt_=9), dict(vocab=0),
    dict(vocab=(1 << 20) + 1), dict(ts=15), dict(ws=None), dict(ws=D + 8), dict(status=A + 1),
])
def test_embed_grad_refuses(bad):
    refused(lambda: grad(**bad), tt.TT_ERR_INVALID_ARG)


def test_embed_grad_scratch():
    need = tt.tt_embed_grad_workspace(4, 300, 16)
    assert need > 0
    refused(lambda: grad(wb=need - 1), tt.TT_ERR_CAPACITY)
    for bad in ((-1, 300, 16), (tt.TT_MAX_IDS + 1, 300, 16), (4, 0, 16), (4, (1 << 20) + 1, 16), (4, 300, 0)):
        assert tt.tt_embed_grad_workspace(*bad) == -1
    # IDs twice over, with their places, and what a row shared by two groups of blocks needs; never more than a few times that
    for n, v, d in ((1, 1, 1), (16400, 4352, 1024), (304824, 100256, 2048), (1 << 24, 1 << 20, 8192)):
        assert 16 * n <= tt.tt_embed_grad_workspace(n, v, d) < 20 * n + 8 * v + (1 << 24) + 16384 * 4 * d


LOSS = dict(logits=A, t=tt.TT_F32, n=4, vocab=300, ls=300, targets=B, loss=C, lse=None, g=None, dlogits=None, ds=300,
            status=None)


def loss(**kw):
    a = {**LOSS, **kw}
    tt.tt_token_loss(a["logits"], a["t"], a["n"], a["vocab"], a["ls"], a["targets"], a["loss"], a["lse"], a["g"],
                     a["dlogits"], a["ds"], a["status"], 0)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(logits=A + 2), dict(t=3), dict(n=-1), dict(vocab=0), dict(vocab=(1 << 20) + 1),
    dict(ls=299), dict(targets=None), dict(targets=B + 2), dict(loss=None), dict(loss=C + 1), dict(lse=C + 1),
    dict(g=C + 2), dict(dlogits=D + 2), dict(dlogits=D, ds=299), dict(dlogits=A, ds=304, ls=300), dict(status=A + 3),
])
def test_token_loss_refuses(bad):
    refused(lambda: loss(**bad), tt.TT_ERR_INVALID_ARG)


def loss_grad(**kw):
    a = {**LOSS, "lse": C, "dlogits": D, **kw}
    tt.tt_token_loss_grad(a["logits"], a["t"], a["n"], a["vocab"], a["ls"], a["targets"], a["lse"], a["g"],
                          a["dlogits"], a["ds"], a["status"], 0)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(lse=None), dict(lse=C + 2), dict(dlogits=None), dict(dlogits=D + 2), dict(ds=299),
    dict(targets=None), dict(t=4), dict(n=-1), dict(vocab=0), dict(ls=299), dict(g=C + 1), dict(status=A + 1),
])
def test_token_loss_grad_refuses(bad):
    refused(lambda: loss_grad(**bad), tt.TT_ERR_INVALID_ARG)


SAMPLE = dict(logits=A, t=tt.TT_F16, n=4, vocab=300, ls=300, uniform=B, temp=None, k=None, p=None, mp=None, ids=C,
              lp=None, status=None)


def sample(**kw):
    a = {**SAMPLE, **kw}
    tt.tt_sample(a["logits"], a["t"], a["n"], a["vocab"], a["ls"], a["uniform"], a["temp"], a["k"], a["p"], a["mp"],
                 a["ids"], a["lp"], a["status"], 0)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(logits=A + 1), dict(t=3), dict(n=-1), dict(vocab=0), dict(vocab=(1 << 20) + 1),
    dict(ls=299), dict(uniform=None), dict(uniform=B + 2), dict(temp=B + 1), dict(k=B + 1), dict(p=B + 1),
    dict(mp=B + 1), dict(ids=None), dict(ids=C + 2), dict(lp=C + 2), dict(status=C + 2),
])
def test_sample_refuses(bad):
    refused(lambda: sample(**bad), tt.TT_ERR_INVALID_ARG)


def test_binding_refuses_tensors_that_do_not_fit():
    """Types, shapes and places are checked before the C call."""
    import torch
    ids, m, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 8), torch.zeros(4)
    for call in (lambda: tt.embed(ids, m), lambda: tt.embed_grad(ids, m, 8), lambda: tt.token_loss(m, ids),
                 lambda: tt.token_loss_grad(m, ids, f), lambda: tt.sample(m, f)):
        with pytest.raises(ValueError):      # CPU tensors
            call()
    with pytest.raises(ValueError):
        tt._matrix(torch.zeros(4, 8, dtype=torch.float64), "x")
    for call in (lambda: tt.embed(None, m), lambda: tt.token_loss(m, None), lambda: tt.sample(m, None)):
        with pytest.raises(ValueError):      # what is not optional
            call()
    with pytest.raises(ValueError):
        tt.embed_grad(ids, m, 8, accumulate=True)
