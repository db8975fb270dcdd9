"""The losses of a model's head on the GPU where their kernels' ways part: short last
chunks with divided contractions, small losses of large logits, gradients of one kind
alone, weights with infinities and NaN, the size of the gradients' errors.  Against the
64-bit forms of head_plain.py."""
import math

import pytest

import head_plain as plain
from test_gpu_head import DTYPES, KINDS, gen, rows_of, status_word, targets_of, tt, within  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("last", [1, 65])
def test_linear_loss_short_last_chunk_of_a_divided_contraction(tt, last):  # noqa: F811
    """Floats, chunks of 2304 rows, whose contraction for dweight is cut into two parts, and a
    last chunk of one block of it, or two.  A product of large values goes ahead, so that no
    tensor memory is zero by chance."""
    g = gen(1)
    vocab, dim, n = 151936, 64, 8 * 2304 + last
    h, w = rows_of(n, dim, torch.float32, g), rows_of(vocab, dim, torch.float32, g, scale=0.1)
    t = torch.randint(-1, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    rg = torch.rand(n, generator=g, device="cuda") / n
    tt.linear_loss(h[:3000], w, t[:3000], torch.full((3000,), 1e6, device="cuda"), want_grad=True)
    st = status_word()
    loss, lse, dh, dw = tt.linear_loss(h, w, t, rg, want_grad=True, status=st)
    exact = torch.empty_like(lse)
    want, bound = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda"), 0
    for a in range(0, n, 2304):
        rows = slice(a, a + 2304)
        r = plain.linear(h[rows], w, t[rows], rg[rows])
        b = plain.linear_bounds(r)
        for got, x, e in zip((loss, lse, dh), (r["loss"], r["lse"], r["dh"]), b):
            within(got[rows], x, plain.rounded(e, x, torch.float32))
        exact[rows] = r["lse"]
        want += r["dw"]
        bound = bound + b[3] + plain.EPS * want.abs() * 2  # (each chunk's sums are added in 32 bits)
        del r, b
    within(dw, want, plain.rounded(bound, want, torch.float32), "dweight")
    later = tt.linear_loss_grad(h, w, t, exact, rg, dweight=torch.empty_like(dw), status=st)[1]
    within(later, want, plain.rounded(bound, want, torch.float32), "dweight from lse")
    assert st.item() == 0


def test_linear_loss_dhidden_alone_needs_no_more_scratch_than_asked(tt):  # noqa: F811
    """A width above the vocabulary's size, and so many rows that they are worked on in chunks."""
    n, vocab, dim = 143337, 7471, 7504
    g = gen(2)
    h = torch.empty(n, dim, dtype=torch.bfloat16, device="cuda")
    for a in range(0, n, 20000):
        h[a:a + 20000] = torch.randn(len(h[a:a + 20000]), dim, generator=g, device="cuda")
    w, t = rows_of(vocab, dim, torch.bfloat16, g, scale=0.01), targets_of(n, vocab, 3)
    need = tt.tt_linear_loss_workspace(n, vocab, dim, tt.TT_BF16, 1, tt.TT_F32, 1)
    space = torch.empty(need, dtype=torch.uint8, device="cuda")
    loss, lse, dh, _ = tt.linear_loss(h, w, t, dhidden=torch.empty_like(h), workspace=space)
    later = tt.linear_loss_grad(h, w, t, lse, dhidden=torch.empty_like(h), workspace=space)[0]
    at = torch.tensor([0, 1, 71679, 71680, 71936, n - 2, n - 1], device="cuda")
    r = plain.linear(h[at], w, t[at], torch.ones(len(at), device="cuda"))
    b = plain.linear_bounds(r)
    for got, want, e, kind in ((loss, r["loss"], b[0], torch.float32), (lse, r["lse"], b[1], torch.float32),
                               (dh, r["dh"], b[2], torch.bfloat16), (later, r["dh"], b[2], torch.bfloat16)):
        within(got[at], want, plain.rounded(e, want, kind))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [600, 300, 40, 4])
@pytest.mark.parametrize("lift", [18.0, 300.0])
def test_linear_loss_of_confident_rows(tt, kind, n, lift):  # noqa: F811
    """Rows that give their target nearly all: losses of some 1e-4, small differences of
    logits of 18 and 300, whose products are sums of terms of one sign.  What such sums lose
    is in every logit of a row alike, so that a loss is off by a share of itself and by what
    the sum of powers loses; and no loss is below zero."""
    kind, g = KINDS[kind], gen(3)
    vocab, dim = 3000, 2048
    u = torch.rand(dim, generator=g, device="cuda") + 0.5
    h = (u * (1 + 0.01 * torch.randn(n, dim, generator=g, device="cuda"))).to(kind)
    w = torch.randn(vocab, dim, generator=g, device="cuda") * 1e-3 + (lift - 17) / float(u.sum())
    w[5] += 17 / float(u.sum())
    w = w.to(kind)
    w[vocab - 1] = 0                                       # (a token far below)
    t = torch.full((n,), 5, dtype=torch.int32, device="cuda")
    r = plain.linear(h, w, t, torch.ones(n, device="cuda"))
    worst = plain.product_bound(h.double().abs() @ w.double().abs().T, dim, kind).amax(1)
    bound = r["loss"] * torch.expm1(2 * worst + plain.EPS * (4 * lift + 64)) + plain.EPS * (24 + vocab / 64)
    assert 1e-5 < float(r["loss"].min()) and float(r["loss"].max()) < 1e-2
    for want_grad in (False, True):
        loss = tt.linear_loss(h, w, t, want_grad=want_grad)[0]
        within(loss, r["loss"], plain.rounded(bound, r["loss"], torch.float32), "loss, gradients %s" % want_grad)
        assert not bool((loss < 0).any())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("n,vocab,dim", [(600, 300, 32), (600, 300, 33), (300, 5000, 33), (60, 300, 32), (4, 300, 32)])
def test_linear_loss_padding_rows_are_zero_whatever_the_weight_holds(tt, kind, value, n, vocab, dim):  # noqa: F811
    """NaN and infinities of the weight reach the rows that have a target, none that have not."""
    kind, g = KINDS[kind], gen(4)
    h, w, t = rows_of(n, dim, kind, g), rows_of(vocab, dim, kind, g, scale=0.3), targets_of(n, vocab, 4)
    t[0], t[n - 1] = -1, 7
    w[7, 3] = value
    rg = torch.full((n,), 1 / n, device="cuda")
    none = t < 0
    loss, lse, dh, _ = tt.linear_loss(h, w, t, rg, dhidden=torch.full_like(h, 5))
    assert not bool(loss[none].any()) and not bool(dh[none].any())
    assert not bool(torch.isfinite(dh[~none][:, 3]).any()) and not bool(torch.isfinite(loss[n - 1]))
    dh = tt.linear_loss_grad(h, w, t, torch.zeros_like(lse), rg, dhidden=torch.full_like(h, 5))[0]
    assert not bool(dh[none].any()) and not bool(torch.isfinite(dh[~none][:, 3]).any())


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,vocab,dim", [(64, 5000, 136), (300, 5000, 136), (1030, 3000, 72), (2100, 4352, 256)])
def test_linear_loss_size_of_the_gradients_errors(tt, kind, n, vocab, dim):  # noqa: F811
    """The error of a gradient as a whole, which bounds on each element (worst cases, summed)
    leave room for.  A rounding to nearest is off by as much as u / sqrt(3) of the value's size
    in the mean (u half a spacing, relative, errors even within it; less for values inside a
    binade), and the roundings are independent of each other and of the random hidden states
    and weight that they meet, so that their shares add up as squares.  5% for chance: a norm of
    10^4 elements and more.
      The result's own rounding: 1.  G's: 1, or with bfloat16's powers the share of G that is not
    the target's, twice (its rounding, and the row's factor that takes back the target's), and
    for dweight hidden's copy: 1.  Up to 64 rows G and the copy have a second part: neither.
    From an lse G is rounded as it is, and hidden's copy not."""
    g = gen(5)
    h, w = rows_of(n, dim, kind, g), rows_of(vocab, dim, kind, g, scale=2 / math.sqrt(dim))
    t, rg = targets_of(n, vocab, 5), torch.full((n,), 1 / n, device="cuda")
    r = plain.linear(h, w, t, rg)
    there = (t >= 0).nonzero()[:, 0]
    of_target = (r["G"][there, t[there].long()] ** 2).sum()
    rest = float(1 - of_target / (r["G"] ** 2).sum())
    one = plain.UNIT[kind] / math.sqrt(3) * 1.05

    def size(got, want):
        return float((got.double() - want).norm() / want.norm())
    _, _, dh, dw = tt.linear_loss(h, w, t, rg, want_grad=True)
    powers = kind == torch.bfloat16
    of_g, of_copy = (0, 0) if n <= 64 else (2 * rest, 1) if powers else (1, 0)
    assert size(dh, r["dh"]) <= one * math.sqrt(1 + of_g)
    assert size(dw, r["dw"]) <= one * math.sqrt(1 + of_g + of_copy)
    dh, dw = tt.linear_loss_grad(h, w, t, r["lse"].float(), rg)
    of_g = 0 if n <= 64 else 1
    assert size(dh, r["dh"]) <= one * math.sqrt(1 + of_g)
    assert size(dw, r["dw"]) <= one * math.sqrt(1 + of_g)
