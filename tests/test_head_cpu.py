"""The losses of a model's head without a GPU: what their C entry points and torch
helpers refuse (before any device call), and the scratch that tt_linear_loss asks for.
Addresses are stand-ins: a refused call never uses them."""
import pytest

from exact_bpe_tokenization_gb300 import binding as tt
from exact_bpe_tokenization_gb300 import build
from test_ops_binding_cpu import Standin, library  # noqa: F401  (a fixture)

A, B, C, D, E, F, W = (k << 20 for k in range(1, 8))      # aligned stand-in addresses


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def refused(call, status):
    with pytest.raises(tt.TokTierError) as e:
        call()
    assert e.value.status == status


LINEAR = dict(h=A, w=B, t=tt.TT_BF16, n=4, vocab=300, dim=16, hs=16, ws=16, targets=C, loss=D, lse=None, g=None, dh=None, dhs=16,
              dw=None, dwt=tt.TT_BF16, dws=16, acc=0, space=W, bytes=1 << 30, status=None)


def linear(**kw):
    a = {**LINEAR, **kw}
    tt.tt_linear_loss(a["h"], a["w"], a["t"], a["n"], a["vocab"], a["dim"], a["hs"], a["ws"], a["targets"], a["loss"], a["lse"],
                      a["g"], a["dh"], a["dhs"], a["dw"], a["dwt"], a["dws"], a["acc"], a["space"], a["bytes"], a["status"], 0)


def linear_grad(**kw):
    a = {**LINEAR, "lse": D, "dh": E, "dw": F, **kw}
    tt.tt_linear_loss_grad(a["h"], a["w"], a["t"], a["n"], a["vocab"], a["dim"], a["hs"], a["ws"], a["targets"], a["lse"], a["g"],
                           a["dh"], a["dhs"], a["dw"], a["dwt"], a["dws"], a["acc"], a["space"], a["bytes"], a["status"], 0)


BAD = [
    dict(h=None), dict(h=A + 1), dict(w=None), dict(w=B + 1), dict(t=3), dict(t=-1), dict(n=-1), dict(vocab=0),
    dict(vocab=(1 << 20) + 1), dict(dim=0), dict(dim=(1 << 16) + 1, hs=1 << 17, ws=1 << 17, dhs=1 << 17, dws=1 << 17), dict(hs=15),
    dict(ws=15), dict(targets=None), dict(targets=C + 2), dict(g=C + 2), dict(status=C + 1), dict(space=None), dict(space=W + 128),
    dict(dh=E + 1), dict(dh=E, dhs=15), dict(dw=F + 1), dict(dw=F, dws=15), dict(dw=F, dwt=tt.TT_F16), dict(dw=F, dwt=7),
    dict(dw=F + 2, dwt=tt.TT_F32),
]


@pytest.mark.parametrize("bad", BAD + [dict(loss=None), dict(loss=D + 2), dict(lse=D + 2)])
def test_linear_loss_refuses(bad):
    refused(lambda: linear(**bad), tt.TT_ERR_INVALID_ARG)


@pytest.mark.parametrize("bad", BAD + [dict(lse=None), dict(lse=D + 2), dict(dh=None, dw=None)])
def test_linear_loss_grad_refuses(bad):
    refused(lambda: linear_grad(**bad), tt.TT_ERR_INVALID_ARG)


@pytest.mark.parametrize("call", [linear, linear_grad])
def test_linear_loss_refuses_sizes(call):
    refused(lambda: call(n=tt.TT_MAX_IDS + 1), tt.TT_ERR_CAPACITY)
    for t in (tt.TT_F32, tt.TT_F16, tt.TT_BF16):
        grad = call is linear_grad
        need = tt.tt_linear_loss_workspace(4, 300, 16, t, True, t, grad)
        refused(lambda: call(t=t, dwt=t, bytes=need - 1), tt.TT_ERR_CAPACITY)
        assert tt.tt_linear_loss_workspace(4, 300, 16, t, False, t, grad) >= need


def test_linear_loss_without_rows_does_nothing():
    linear(n=0, h=None, targets=None, loss=None)
    linear(n=0, h=None, targets=None, loss=None, dh=E)


def test_linear_loss_workspace():
    f = tt.tt_linear_loss_workspace
    for bad in ((-1, 300, 16, 2, 1, 2, 1), (tt.TT_MAX_IDS + 1, 300, 16, 2, 1, 2, 1), (4, 0, 16, 2, 1, 2, 1),
                (4, (1 << 20) + 1, 16, 2, 1, 2, 1), (4, 300, 0, 2, 1, 2, 1), (4, 300, (1 << 16) + 1, 2, 1, 2, 1),
                (4, 300, 16, 3, 1, 3, 1), (4, 300, 16, 2, 1, 1, 1)):
        assert f(*bad) == -1
    # bounded, however many the rows: a chunk of G, and the weight's sums in 32 bits between chunks
    g, acc = 2 << 30, 100256 * 2048 * 4
    assert f(1 << 20, 100256, 2048, tt.TT_BF16, 1, tt.TT_F32, 1) < 3 * g
    assert acc < f(1 << 20, 100256, 2048, tt.TT_BF16, 1, tt.TT_BF16, 1) < 3 * g + acc
    assert f(1 << 20, 100256, 2048, tt.TT_BF16, 1, tt.TT_BF16, 0) < 1 << 29
    assert f(1 << 28, 300, 2048, tt.TT_BF16, 1, tt.TT_F32, 1) < 4 * g      # (copies of hidden too)
    assert f(1 << 28, 300, 2048, tt.TT_F32, 1, tt.TT_F32, 0) < 2 * g
    assert f(0, 300, 16, tt.TT_BF16, 1, tt.TT_BF16, 1) > 0


DISTILL = dict(x=A, t=tt.TT_BF16, n=4, vocab=300, xs=300, ids=B, ids_s=5, v=C, vt=tt.TT_F32, vs=5, k=5, T=2.0, loss=D, lse=None, g=None,
               dx=None, dxs=300, status=None)


def distill(**kw):
    a = {**DISTILL, **kw}
    tt.tt_distill_loss(a["x"], a["t"], a["n"], a["vocab"], a["xs"], a["ids"], a["ids_s"], a["v"], a["vt"], a["vs"], a["k"], a["T"],
                       a["loss"], a["lse"], a["g"], a["dx"], a["dxs"], a["status"], 0)


def distill_grad(**kw):
    a = {**DISTILL, "lse": D, "dx": E, **kw}
    tt.tt_distill_loss_grad(a["x"], a["t"], a["n"], a["vocab"], a["xs"], a["ids"], a["ids_s"], a["v"], a["vt"], a["vs"], a["k"], a["T"],
                            a["lse"], a["g"], a["dx"], a["dxs"], a["status"], 0)


BAD = [
    dict(x=None), dict(x=A + 1), dict(t=3), dict(n=-1), dict(vocab=0), dict(vocab=(1 << 20) + 1, xs=1 << 21, dxs=1 << 21), dict(xs=299),
    dict(ids=None), dict(ids=B + 2), dict(ids_s=4), dict(v=None), dict(v=C + 2), dict(vt=3), dict(vs=4), dict(k=0),
    dict(k=tt.TT_MAX_TEACHER + 1, ids_s=2000, vs=2000), dict(T=0.0), dict(T=-1.0), dict(T=float("inf")), dict(T=float("nan")),
    dict(T=2.0**-65), dict(T=2.0**65), dict(g=C + 2), dict(status=C + 1), dict(dx=E + 1), dict(dx=E, dxs=299),
    dict(dx=A, xs=301, dxs=300),
]


@pytest.mark.parametrize("bad", BAD + [dict(loss=None), dict(loss=D + 1), dict(lse=D + 2)])
def test_distill_loss_refuses(bad):
    refused(lambda: distill(**bad), tt.TT_ERR_INVALID_ARG)


@pytest.mark.parametrize("bad", BAD + [dict(lse=None), dict(lse=D + 2), dict(dx=None)])
def test_distill_loss_grad_refuses(bad):
    refused(lambda: distill_grad(**bad), tt.TT_ERR_INVALID_ARG)


def test_distill_loss_sizes():
    for call in (distill, distill_grad):
        refused(lambda: call(n=tt.TT_MAX_IDS + 1), tt.TT_ERR_CAPACITY)
    distill(n=0, x=None, ids=None, v=None, loss=None)
    distill_grad(n=0, x=None, ids=None, v=None, lse=None, dx=None)


def test_chained_kernels_read_nothing_as_constant():
    """tt_linear.cu's kernels start while the one before still writes, which may be the
    caller's own: what they read goes by plain loads and copies, never by the read-only path."""
    import os
    csrc = os.path.join(os.path.dirname(tt.__file__), "csrc")
    for name in ("tt_linear.cu", "tt_gemm.cuh"):
        with open(os.path.join(csrc, name), encoding="utf-8") as f:
            text = f.read()
        for word in ("__ldg", "load_raw", "ld.global.nc", "__restrict__"):
            assert word not in text, (name, word)


# ------------------------------------------------------------ the torch helpers

torch = pytest.importorskip("torch")
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def lin(L, grad=False, **kw):
    a = dict(hidden=Standin(4, 16, dtype=BF), weight=Standin(300, 16, dtype=BF), targets=Standin(4, dtype=I32))
    if grad:
        a["lse"] = Standin(4)
    return (tt.linear_loss_grad if grad else tt.linear_loss)(**{**a, **kw})


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("bad", [
    dict(hidden=Standin(4, 16, dtype=torch.float64)), dict(hidden=Standin(4, 16, dtype=BF, on=-1)), dict(hidden=Standin(4, dtype=BF)),
    dict(hidden=Standin(4, 16, dtype=BF, stride=(1, 4))), dict(weight=Standin(300, 15, dtype=BF)), dict(weight=Standin(300, 16)),
    dict(weight=Standin(300, 16, dtype=BF, on=1)), dict(targets=None), dict(targets=Standin(5, dtype=I32)),
    dict(targets=Standin(4, dtype=torch.int64)), dict(targets=Standin(4, dtype=I32, on=1)), dict(row_grads=Standin(3)),
    dict(row_grads=Standin(4, dtype=BF)), dict(status=Standin(2, dtype=I32)), dict(dhidden=Standin(4, 16)),
    dict(dhidden=Standin(3, 16, dtype=BF)), dict(dhidden=Standin(4, 16, dtype=BF, on=1)), dict(dweight=Standin(300, 16, dtype=torch.float16)),
    dict(dweight=Standin(299, 16, dtype=BF)), dict(dweight=Standin(300, 16, dtype=BF, on=1)), dict(accumulate=True),
    dict(workspace=Standin(64, dtype=torch.uint8, on=1)), dict(workspace=Standin(64, dtype=torch.uint8, stride=(2,))),
])
def test_linear_loss_helpers_refuse(library, grad, bad):  # noqa: F811
    with pytest.raises(ValueError):
        lin(library, grad, **bad)
    assert library.calls == 0


def test_linear_loss_grad_wants_lse(library):  # noqa: F811
    for bad in (None, Standin(3), Standin(4, dtype=BF), Standin(4, on=1)):
        with pytest.raises(ValueError):
            lin(library, True, lse=bad)
    assert library.calls == 0


def dis(grad=False, **kw):
    a = dict(logits=Standin(4, 300, dtype=BF), teacher_ids=Standin(4, 5, dtype=I32), teacher_logits=Standin(4, 5))
    if grad:
        a["lse"] = Standin(4)
    return (tt.distill_loss_grad if grad else tt.distill_loss)(**{**a, **kw})


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("bad", [
    dict(logits=Standin(4, 300, dtype=torch.float64)), dict(logits=Standin(4, 300, dtype=BF, on=-1)),
    dict(logits=Standin(4, 300, dtype=BF, stride=(1, 4))), dict(teacher_ids=None), dict(teacher_ids=Standin(4, 5, dtype=torch.int64)),
    dict(teacher_ids=Standin(4, 6, dtype=I32)), dict(teacher_ids=Standin(20, dtype=I32)), dict(teacher_ids=Standin(4, 5, dtype=I32, on=1)),
    dict(teacher_ids=Standin(4, 5, dtype=I32, stride=(1, 4))), dict(teacher_logits=Standin(3, 5)),
    dict(teacher_logits=Standin(4, 5, dtype=torch.float64)), dict(teacher_logits=Standin(4, 5, on=1)),
    dict(row_grads=Standin(5)), dict(status=Standin(2, dtype=I32)), dict(dlogits=Standin(4, 300)), dict(dlogits=Standin(4, 299, dtype=BF)),
    dict(dlogits=Standin(4, 300, dtype=BF, on=1)),
])
def test_distill_loss_helpers_refuse(library, grad, bad):  # noqa: F811
    with pytest.raises(ValueError):
        dis(grad, **bad)
    assert library.calls == 0


def test_distill_loss_grad_wants_lse(library):  # noqa: F811
    for bad in (None, Standin(3), Standin(4, dtype=BF), Standin(4, on=1)):
        with pytest.raises(ValueError):
            dis(True, lse=bad)
    assert library.calls == 0
