"""The losses of a model's head on the GPU against plain 64-bit forms (head_plain.py):
types, sizes around the kernels' tiles, strides and alignments, padding and invalid
targets, rows far from zero, infinities and NaN, chunks, accumulation, other streams,
graph capture, 32-bit overflow, differences, and a run of the operators together.
Tolerances are the error bounds of head_plain.py."""
import math

import numpy as np
import pytest

import head_plain as plain

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
KINDS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def tt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from exact_bpe_tokenization_gb300 import binding
    return binding


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows_of(n, d, kind, g, stride=None, shift=0, scale=1.0):
    """An [n, d] tensor, its rows `stride` apart, its first element `shift` elements past
    a 16-byte boundary; what lies between is NaN."""
    stride = stride or d
    buf = torch.full((n * stride + shift + 8,), math.nan, dtype=kind, device="cuda")
    x = buf[shift:shift + n * stride].view(n, stride)[:, :d]
    x.copy_(torch.randn(n, d, generator=g, device="cuda") * scale)
    return x


def gaps_untouched(x):
    n, d = x.shape
    s = x.stride(0)
    if n < 2 or s == d:
        return True
    return bool(torch.isnan(torch.as_strided(x, (n - 1, s - d), (s, 1), x.storage_offset() + d)).all())


def targets_of(n, vocab, seed):
    rng = np.random.default_rng(seed)
    t = rng.integers(0, vocab, n).astype(np.int32)
    if n > 3:
        t[rng.random(n) < 0.1] = -1
        t[1], t[2] = vocab - 1, 0
    return torch.from_numpy(t).cuda()


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def within(got, want, bound, what=""):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), "%s: %d of %d off, the worst %.3g where %.3g is allowed" % (
        what, int(bad.sum()), bad.numel(), float((got.double() - want).abs()[bad].max()),
        float(bound.expand_as(want)[bad].min()))


def check_linear(out, r, dwkind=None):
    """(loss, lse, dhidden, dweight) against linear()'s, None left out."""
    loss, lse, dh, dw = plain.linear_bounds(r)
    kind = r["kind"]
    for got, want, b, t, what in zip(out, (r["loss"], r["lse"], r["dh"], r["dw"]), (loss, lse, dh, dw),
                                     (torch.float32, torch.float32, kind, dwkind or kind), ("loss", "lse", "dhidden", "dweight")):
        if got is not None:
            assert got.dtype == t and got.shape == want.shape
            within(got, want, plain.rounded(b, want, t), what)


# ------------------------------------------------------------ linear: sizes and types

# around a tile's 256, a part's 128, a stage's 64, and 16 bytes
SHAPES = [(1, 1, 1), (1, 300, 8), (2, 7, 3), (5, 129, 24), (33, 300, 64), (64, 4352, 64), (127, 128, 63), (128, 255, 65),
          (129, 256, 128), (255, 257, 40), (256, 512, 256), (257, 513, 257), (300, 1000, 641), (700, 2000, 72), (1030, 700, 16),
          (4100, 260, 24), (40, 9000, 520), (7, 4352, 1024), (3, 4352, 1024), (4, 9000, 130), (5, 600, 24), (8, 20000, 130), (9, 511, 1030), (17, 5000, 33), (65, 5000, 130)]


@pytest.mark.parametrize("n,vocab,dim", SHAPES)
@pytest.mark.parametrize("kind", KINDS)
def test_linear_loss(tt, n, vocab, dim, kind):
    kind = KINDS[kind]
    g = gen(n + dim)
    h, w = rows_of(n, dim, kind, g), rows_of(vocab, dim, kind, g, scale=2 / math.sqrt(dim))
    t = targets_of(n, vocab, n)
    rg = torch.rand(n, generator=g, device="cuda") / n
    r = plain.linear(h, w, t, rg)
    st = status_word()
    out = tt.linear_loss(h, w, t, rg, want_grad=True, status=st)
    check_linear(out, r)
    alone = tt.linear_loss(h, w, t, rg, status=st)
    assert len(alone) == 2
    check_linear(alone, r)
    check_linear((None, None) + tt.linear_loss_grad(h, w, t, r["lse"].float(), rg, status=st), r)
    assert not out[0][t < 0].any() and not out[2][t < 0].any()
    assert st.item() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hs,hshift,ws,wshift", [(48, 0, 48, 0), (41, 0, 40, 0), (40, 1, 40, 0), (40, 0, 43, 3), (47, 5, 49, 7), (56, 8, 64, 8)])
@pytest.mark.parametrize("n,dim", [(70, 40), (50, 40), (11, 39), (6, 40), (4, 40), (3, 39)])
def test_linear_loss_strides_and_alignments(tt, kind, hs, hshift, ws, wshift, n, dim):
    kind, g = KINDS[kind], gen(hs + ws)
    vocab = 300
    h, w = rows_of(n, dim, kind, g, hs, hshift), rows_of(vocab, dim, kind, g, ws, wshift, 0.3)
    dh, dw = rows_of(n, dim, kind, g, hs, hshift), rows_of(vocab, dim, kind, g, ws, wshift)
    wide = rows_of(vocab, dim, torch.float32, g, ws, wshift)
    t, rg = targets_of(n, vocab, 3), torch.rand(n, generator=g, device="cuda")
    r = plain.linear(h, w, t, rg)
    out = tt.linear_loss(h, w, t, rg, dhidden=dh, dweight=dw)
    assert out[2] is dh and out[3] is dw
    check_linear(out, r)
    assert gaps_untouched(dh) and gaps_untouched(dw)
    out = tt.linear_loss(h, w, t, rg, dweight=wide)
    assert out[2] is None and out[3] is wide
    check_linear(out, r, torch.float32)
    assert gaps_untouched(wide)
    dh.zero_()
    assert tt.linear_loss_grad(h, w, t, out[1], rg, dhidden=dh) == (dh, None)
    check_linear((None, None, dh), r)


def test_linear_loss_without_row_grads(tt):
    g = gen(5)
    h, w, t = rows_of(33, 64, torch.bfloat16, g), rows_of(300, 64, torch.bfloat16, g, scale=0.2), targets_of(33, 300, 1)
    a = tt.linear_loss(h, w, t, want_grad=True)
    check_linear(a, plain.linear(h, w, t, torch.ones(33, device="cuda")))


@pytest.mark.parametrize("kind", KINDS)
def test_linear_loss_padding_and_invalid_targets(tt, kind):
    kind, g = KINDS[kind], gen(6)
    n, vocab, dim = 40, 260, 32
    h, w = rows_of(n, dim, kind, g), rows_of(vocab, dim, kind, g, scale=0.3)
    rg = torch.ones(n, device="cuda")
    st = status_word()
    for fill, want in ((-1, 0), (-(1 << 31), 0), (vocab, tt.TT_ERR_INVALID_ARG), ((1 << 31) - 1, tt.TT_ERR_INVALID_ARG)):
        t = torch.full((n,), fill, dtype=torch.int32, device="cuda")
        st.zero_()
        loss, lse, dh, dw = tt.linear_loss(h, w, t, rg, want_grad=True, status=st)
        assert st.item() == want
        assert not loss.any() and not dh.any() and not dw.any()
        check_linear((None, lse), plain.linear(h, w, t, rg))
        st.zero_()
        dh, dw = tt.linear_loss_grad(h, w, t, lse, rg, status=st)
        assert st.item() == want and not dh.any() and not dw.any()
    t = targets_of(n, vocab, 8)
    t[5], t[6] = vocab, vocab + 77
    st.zero_()
    check_linear(tt.linear_loss(h, w, t, rg, want_grad=True, status=st), plain.linear(h, w, t, rg))
    assert st.item() == tt.TT_ERR_INVALID_ARG


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("n,vocab", [(300, 300), (300, 5000), (30, 5000), (4, 5000)])
def test_linear_loss_accumulates(tt, kind, wide, n, vocab):
    kind, g = KINDS[kind], gen(7)
    dim = 72
    h, w, t = rows_of(n, dim, kind, g), rows_of(vocab, dim, kind, g, scale=0.2), targets_of(n, vocab, 4)
    dkind = torch.float32 if wide else kind
    before = (torch.randn(vocab, dim, generator=g, device="cuda") * 0.1).to(dkind)
    rg = torch.full((n,), 1 / 64, device="cuda")
    r = plain.linear(h, w, t, rg)
    r["dw"] = r["dw"] + before.double()
    b = plain.linear_bounds(r)[3] + 2 * plain.EPS * r["dw"].abs()
    for call in (lambda d: tt.linear_loss(h, w, t, rg, dweight=d, accumulate=True)[3],
                 lambda d: tt.linear_loss_grad(h, w, t, r["lse"].float(), rg, dweight=d, accumulate=True)[1]):
        within(call(before.clone()), r["dw"], plain.rounded(b, r["dw"], dkind))


def test_linear_loss_without_rows(tt):
    w = torch.randn(300, 24, device="cuda").bfloat16()
    h, t = w[:0], torch.empty(0, dtype=torch.int32, device="cuda")
    loss, lse, dh, dw = tt.linear_loss(h, w, t, want_grad=True)
    assert loss.shape == lse.shape == (0,) and dh.shape == (0, 24) and not dw.any()
    kept = torch.full((300, 24), 3.0, device="cuda")
    tt.linear_loss(h, w, t, dweight=kept, accumulate=True)
    assert bool((kept == 3).all())
    tt.linear_loss_grad(h, w, t, lse, dweight=kept)
    assert not kept.any()
    assert tt.linear_loss_grad(h, w, t, lse, dhidden=dh) == (dh, None)


@pytest.mark.parametrize("kind,dwkind,accumulate", [("bf16", "bf16", False), ("bf16", "bf16", True), ("bf16", "f32", True),
                                                    ("f16", "f16", False), ("f32", "f32", False)])
def test_linear_loss_in_chunks(tt, kind, dwkind, accumulate):
    """More rows than are worked on at a time: the weight's gradient is summed over chunks."""
    kind, dwkind, g = KINDS[kind], KINDS[dwkind], gen(9)
    n, vocab, dim = (1100 if kind != torch.float32 else 400), 1 << 20, 24
    h, w, t = rows_of(n, dim, kind, g), rows_of(vocab, dim, kind, g, scale=0.3), targets_of(n, vocab, 5)
    rg = torch.full((n,), 1 / 256, device="cuda")
    rg[:200] *= 16                                         # (chunks of different scales)
    r = plain.linear(h, w, t, rg)
    dw = (torch.randn(vocab, dim, generator=g, device="cuda") * 2**-8).to(dwkind)
    bounds = plain.linear_bounds(r)
    if accumulate:
        r["dw"] = r["dw"] + dw.double()
    dh = torch.empty_like(h)
    loss, lse, _, _ = tt.linear_loss(h, w, t, rg, dhidden=dh, dweight=dw, accumulate=accumulate)
    for got, want, b, k in zip((loss, lse, dh, dw), (r["loss"], r["lse"], r["dh"], r["dw"]), bounds,
                               (torch.float32, torch.float32, kind, dwkind)):
        within(got, want, plain.rounded(b + 4 * plain.EPS * want.abs(), want, k))


# ------------------------------------------------------------ linear: values

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lift", [-300.0, -60.0, 60.0, 300.0])
@pytest.mark.parametrize("n", [300, 47, 8, 4])
def test_linear_loss_far_from_zero(tt, kind, lift, n):
    """Rows whose logits lie far from zero, all of them or all but the target's, and rows
    of a spread beyond what 32-bit powers hold."""
    kind, g = KINDS[kind], gen(11)
    vocab, dim = 600, 32
    h, w = rows_of(n, dim, kind, g), rows_of(vocab, dim, kind, g, scale=0.3)
    h[:, 0] = 0
    w[:, 0] = 1
    t = targets_of(n, vocab, 6)
    h[::3, 0] = lift                                       # every logit of the row
    h[:, 1] = 0
    w[:, 1] = 0
    w[17, 1] = 1
    h[1::3, 1] = lift                                      # one logit of the row, its target's in some
    t[4::6] = 17
    rg = torch.rand(n, generator=g, device="cuda") + 0.5
    r = plain.linear(h, w, t, rg)
    check_linear(tt.linear_loss(h, w, t, rg, want_grad=True), r)
    check_linear(tt.linear_loss(h, w, t, rg), r)


@pytest.mark.parametrize("kind", KINDS)
def test_linear_loss_of_equal_logits(tt, kind):
    """Hidden states of zeros: log(vocab) for each row, and equal probabilities."""
    kind = KINDS[kind]
    h, w = torch.zeros(5, 16, dtype=kind, device="cuda"), rows_of(777, 16, kind, gen(12))
    t = torch.tensor([0, 5, 776, -1, 3], dtype=torch.int32, device="cuda")
    check_linear(tt.linear_loss(h, w, t, want_grad=True), plain.linear(h, w, t, torch.ones(5, device="cuda")))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n", [300, 60, 8])
def test_linear_loss_nan_and_infinities_stay_in_their_rows(tt, kind, value, n):
    kind, g = KINDS[kind], gen(13)
    vocab, dim = 400, 24
    h, w, t = rows_of(n, dim, kind, g), rows_of(vocab, dim, kind, g, scale=0.3), targets_of(n, vocab, 9)
    rg = torch.full((n,), 1 / n, device="cuda")
    t[7] = 5
    clean = h.clone()
    h[7, 3] = value
    got = tt.linear_loss(h, w, t, rg, want_grad=True)
    assert not bool(torch.isfinite(got[0][7])) and not bool(torch.isfinite(got[1][7])) and bool(torch.isnan(got[2][7]).all())
    others = torch.arange(n, device="cuda") != 7
    r = plain.linear(clean[others], w, t[others], rg[others])
    check_linear([x[others] for x in got[:3]], r)
    # a padding row adds nothing, whatever it holds
    t[7] = -1
    loss, lse, dh, dw = tt.linear_loss(h, w, t, rg, want_grad=True)
    assert loss[7] == 0 and not bool(dh[7].any()) and not bool(torch.isfinite(lse[7]))
    check_linear([x[others] for x in (loss, lse, dh)] + [dw], r)
    rg[7] = math.nan
    dh, dw = tt.linear_loss_grad(h, w, t, torch.where(others, lse, math.nan), rg)
    assert not bool(dh[7].any())
    check_linear((None, None, dh[others], dw), r)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [2.0**-30, 1.0, 2.0**20])
def test_linear_loss_small_and_large_row_grads(tt, kind, size):
    kind, g = KINDS[kind], gen(14)
    n, vocab, dim = 100, 500, 32
    h, w, t = rows_of(n, dim, kind, g), rows_of(vocab, dim, kind, g, scale=0.3), targets_of(n, vocab, 9)
    rg = (torch.rand(n, generator=g, device="cuda") + 0.01) * size
    rg[3] = 0
    dw = torch.empty(vocab, dim, device="cuda")            # (32 bits: 16-bit floats end sooner)
    out = tt.linear_loss(h, w, t, rg, dweight=dw)
    r = plain.linear(h, w, t, rg)
    check_linear((None, None, None, out[3]), r, torch.float32)


def test_linear_loss_gradients_against_differences(tt):
    """The losses' change along a direction, by 32-bit losses at either side."""
    g = gen(15)
    n, vocab, dim = 64, 500, 48
    h, w, t = rows_of(n, dim, torch.float32, g), rows_of(vocab, dim, torch.float32, g, scale=0.3), targets_of(n, vocab, 2)
    rg = torch.rand(n, generator=g, device="cuda")
    _, _, dh, dw = tt.linear_loss(h, w, t, rg, want_grad=True)
    uh, uw = rows_of(n, dim, torch.float32, g), rows_of(vocab, dim, torch.float32, g, scale=0.3)
    total = lambda s: (tt.linear_loss(h + s * uh, w + s * uw, t)[0].double() * rg.double()).sum()  # noqa: E731
    step = 2.0**-8
    slope = (total(step) - total(-step)) / (2 * step)
    want = (dh.double() * uh).sum() + (dw.double() * uw).sum()
    # the next term is a sixth of the third derivative; it is taken from the slope at twice
    # the step, with as much again to spare; and the losses' own errors
    wide = (total(2 * step) - total(-2 * step)) / (4 * step)
    r = plain.linear(h, w, t, rg)
    noise = (2 * plain.linear_bounds(r)[0] * rg.double()).sum() / (2 * step)
    assert abs(slope - want) <= 2 * abs(wide - slope) / 3 + noise


# ------------------------------------------------------------ linear: how it is called

@pytest.mark.parametrize("kind", KINDS)
def test_linear_loss_gives_the_same_bits(tt, kind):
    kind, g = KINDS[kind], gen(16)
    h, w, t = rows_of(513, 264, kind, g), rows_of(5000, 264, kind, g, scale=0.1), targets_of(513, 5000, 2)
    a = tt.linear_loss(h, w, t, want_grad=True)
    for _ in range(3):
        b = tt.linear_loss(h, w, t, want_grad=True)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_linear_loss_workspace_of_the_caller(tt):
    g = gen(17)
    h, w, t = rows_of(70, 40, torch.bfloat16, g), rows_of(900, 40, torch.bfloat16, g, scale=0.3), targets_of(70, 900, 2)
    need = tt.tt_linear_loss_workspace(70, 900, 40, tt.TT_BF16, 1, tt.TT_BF16, 1)
    want = tt.linear_loss(h, w, t, want_grad=True)
    buf = torch.full((need + 1024,), 255, dtype=torch.uint8, device="cuda")
    got = tt.linear_loss(h, w, t, want_grad=True, workspace=buf[512:512 + need])
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert bool((buf[:512] == 255).all()) and bool((buf[512 + need:] == 255).all())
    with pytest.raises(tt.TokTierError):
        tt.linear_loss(h, w, t, want_grad=True, workspace=buf[512:512 + need - 1])


def test_linear_loss_on_other_streams(tt):
    """Two calls at once, each on its own stream with its own workspace."""
    g = gen(18)
    h = [rows_of(600, 136, torch.bfloat16, g) for _ in range(2)]
    w, t = rows_of(3000, 136, torch.bfloat16, g, scale=0.1), targets_of(600, 3000, 3)
    want = [tt.linear_loss(x, w, t, want_grad=True) for x in h]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for x, s in zip(h, streams):
            got.append(tt.linear_loss(x, w, t, want_grad=True, stream=s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [300, 30, 4])
def test_linear_loss_in_a_graph(tt, kind, n):
    kind, g = KINDS[kind], gen(19)
    vocab, dim = 1000, 40
    h, w, t = rows_of(n, dim, kind, g), rows_of(vocab, dim, kind, g, scale=0.3), targets_of(n, vocab, 4)
    tt.linear_loss(h, w, t, want_grad=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tt.linear_loss(h, w, t, want_grad=True)
        later = tt.linear_loss_grad(h, w, t, out[1])
    for seed in (1, 2):
        h.copy_(torch.randn(n, dim, generator=gen(seed), device="cuda"))
        t.copy_(targets_of(n, vocab, seed))
        graph.replay()
        torch.cuda.synchronize()
        want = tt.linear_loss(h, w, t, want_grad=True)
        assert all(torch.equal(x, y) for x, y in zip(out, want))
        assert all(torch.equal(x, y) for x, y in zip(later, tt.linear_loss_grad(h, w, t, want[1])))


def test_linear_loss_offsets_past_32_bits(tt):
    """A weight and its gradient of 2.4e9 elements each, and hidden states of as many."""
    vocab, dim = 1 << 20, 2304
    w = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    g = gen(20)
    at = torch.tensor([vocab - 1, 0, 932068, vocab - 2], device="cuda")
    w[at] = (torch.randn(4, dim, generator=g, device="cuda") * 0.05).bfloat16()
    h, t = rows_of(4, dim, torch.bfloat16, g), at.int()
    rg = torch.ones(4, device="cuda")
    loss, lse, dh, dw = tt.linear_loss(h, w, t, rg, want_grad=True)
    r = plain.linear(h, w, t, rg)
    check_linear((loss, lse, dh), r)
    b = plain.linear_bounds(r)[3]
    for i in list(at.tolist()) + [932067, vocab // 2]:
        within(dw[i], r["dw"][i], plain.rounded(b[i], r["dw"][i], torch.bfloat16))
    del r, b, w, dw
    n = 1000000
    w = rows_of(300, dim, torch.bfloat16, g, scale=0.02)
    h = torch.empty(n, dim, dtype=torch.bfloat16, device="cuda")
    for a in range(0, n, 50000):
        h[a:a + 50000] = torch.randn(50000, dim, generator=g, device="cuda").bfloat16()
    t = torch.randint(-1, 300, (n,), generator=g, device="cuda", dtype=torch.int32)
    loss, lse, dh, _ = tt.linear_loss(h, w, t, dhidden=torch.empty_like(h))
    at = torch.tensor([0, 1, 932066, 932067, 932068, 932069, n - 1, n // 2], device="cuda")
    check_linear((loss[at], lse[at], dh[at]), plain.linear(h[at], w, t[at], torch.ones(8, device="cuda")))


# ------------------------------------------------------------ distill

def entries(n, vocab, k, kind, seed, repeat=0):
    """(ids, values): different IDs in a row where there are enough, padding among them;
    `repeat` of a row's entries once more."""
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(vocab)[:k] if k <= vocab else rng.integers(0, vocab, k) for _ in range(n)]).astype(np.int32)
    if k > 3:
        ids[rng.random((n, k)) < 0.1] = -1
    for i in range(min(repeat, k - 1)):
        ids[:, rng.integers(0, k)] = ids[:, rng.integers(0, k)]
    if n > 2:
        ids[n // 2] = -1
    v = torch.from_numpy(rng.standard_normal((n, k)) * 3).cuda().to(kind)
    return torch.from_numpy(ids).cuda(), v


def check_distill(out, x, ids, values, temperature, rg):
    want, bounds = plain.distill(x, ids, values, temperature, rg)
    for got, w, b, kind, what in zip(out, want, bounds, (torch.float32, torch.float32, x.dtype), ("loss", "lse", "dlogits")):
        if got is not None:
            assert got.dtype == kind and got.shape == w.shape
            within(got, w, plain.rounded(b, w, kind), what)


ROWS = [(60, 75000, 20), (40, 125000, 33), (30, 150000, 9), (1, 1, 1), (3, 2, 2), (4, 7, 5), (9, 300, 1), (33, 300, 31), (5, 1000, 1024), (20, 2048, 64), (7, 2051, 33), (64, 4352, 8),
        (6, 16384, 100), (5, 20001, 256), (40, 50257, 64), (3, 100256, 1000), (400, 100256, 20), (2, 200255, 37), (1, 430000, 64),
        (3, 1 << 20, 50)]


@pytest.mark.parametrize("n,vocab,k", ROWS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("temperature", [1.0, 2.5])
def test_distill_loss(tt, n, vocab, k, kind, temperature):
    kind, g = KINDS[kind], gen(n + k)
    x = rows_of(n, vocab, kind, g, scale=3.0)
    ids, values = entries(n, vocab, k, DTYPES[(n + k) % 3], n, repeat=k // 3 if k > 8 else 0)
    rg = torch.rand(n, generator=g, device="cuda")
    st = status_word()
    out = tt.distill_loss(x, ids, values, temperature, rg, want_grad=True, status=st)
    check_distill(out, x, ids, values, temperature, rg)
    alone = tt.distill_loss(x, ids, values, temperature, rg, status=st)
    assert len(alone) == 2 and torch.equal(alone[0], out[0]) and torch.equal(alone[1], out[1])
    y = x.clone()
    again = tt.distill_loss(y, ids, values, temperature, rg, dlogits=y)
    assert again[2] is y and all(torch.equal(a, b) for a, b in zip(again, out))
    assert st.item() == 0


@pytest.mark.parametrize("n,vocab,k", [(4, 7, 5), (33, 300, 31), (7, 2051, 33), (40, 50257, 64), (2, 200255, 37)])
@pytest.mark.parametrize("kind", KINDS)
def test_distill_loss_grad(tt, n, vocab, k, kind):
    kind, g = KINDS[kind], gen(n + k)
    x = rows_of(n, vocab, kind, g, scale=3.0)
    ids, values = entries(n, vocab, k, torch.float32, n, repeat=2)
    rg = torch.rand(n, generator=g, device="cuda")
    (_, lse, want), (_, _, b) = plain.distill(x, ids, values, 1.5, rg)
    far = (lse.abs() + (x.double() / 1.5).abs().amax(1))[:, None]
    b = b + 4 * plain.EPS * far * (want.abs() + rg[:, None] / 1.5 * torch.exp(x.double() / 1.5 - lse[:, None]))
    got = tt.distill_loss_grad(x, ids, values, lse.float(), 1.5, rg)
    within(got, want, plain.rounded(b, want, kind))
    y = x.clone()
    assert torch.equal(tt.distill_loss_grad(y, ids, values, lse.float(), 1.5, rg, dlogits=y), got)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("stride,shift,out_stride,out_shift", [(304, 0, 304, 0), (301, 0, 301, 0), (300, 3, 300, 5), (320, 8, 307, 1)])
def test_distill_loss_strides_and_alignments(tt, kind, stride, shift, out_stride, out_shift):
    kind, g = KINDS[kind], gen(stride)
    x, d = rows_of(9, 300, kind, g, stride, shift, 2.0), rows_of(9, 300, kind, g, out_stride, out_shift)
    ids, values = entries(9, 300, 11, torch.float16, 2)
    wide = torch.full((9, 13), 299, dtype=torch.int32, device="cuda")
    wide[:, :11] = ids
    far = torch.full((9, 17), math.nan, dtype=torch.float16, device="cuda")
    far[:, :11] = values
    rg = torch.rand(9, generator=g, device="cuda")
    out = tt.distill_loss(x, wide[:, :11], far[:, :11], 2.0, rg, dlogits=d)
    check_distill(out, x, ids, values, 2.0, rg)
    assert gaps_untouched(d)


@pytest.mark.parametrize("vocab", [300, 5000, 60000, 200255])
def test_distill_loss_same_id_many_times(tt, vocab):
    """All of a row's entries at one ID, and at two: their shares add up."""
    g = gen(4)
    x = rows_of(4, vocab, torch.float32, g, scale=2.0)
    ids = torch.full((4, 700), vocab - 1, dtype=torch.int32, device="cuda")
    ids[1, ::2] = vocab // 3
    ids[2, 5:] = 0
    ids[3, 1:] = -1
    values = torch.randn(4, 700, generator=g, device="cuda")
    rg = torch.ones(4, device="cuda")
    check_distill(tt.distill_loss(x, ids, values, 1.0, rg, want_grad=True), x, ids, values, 1.0, rg)


def test_distill_loss_rows_without_entries_and_invalid_ids(tt):
    g = gen(5)
    for kind in DTYPES:
        for vocab in (300, 70000):
            x = rows_of(5, vocab, kind, g, scale=2.0)
            ids, values = entries(5, vocab, 6, torch.float32, 3)
            ids[0] = -1
            ids[1] = torch.tensor([-5, vocab, vocab + 9, (1 << 31) - 1, -(1 << 31), -1])
            values[3] = -math.inf
            values[4, 2:] = -math.inf
            ids[4, :3] = torch.tensor([0, vocab - 1, 5])
            rg = torch.ones(5, device="cuda")
            st = status_word()
            loss, lse, d = tt.distill_loss(x, ids, values, 2.0, rg, want_grad=True, status=st)
            assert st.item() == tt.TT_ERR_INVALID_ARG
            check_distill((loss, lse, d), x, ids, values, 2.0, rg)
            for i in (0, 1, 2, 3):
                assert loss[i] == 0 and not bool(d[i].any())
            st.zero_()
            later = tt.distill_loss_grad(x, ids, values, lse, 2.0, rg, status=st)
            assert st.item() == tt.TT_ERR_INVALID_ARG and not bool(later[:4].any())


@pytest.mark.parametrize("vocab", [300, 70000])
@pytest.mark.parametrize("kind", KINDS)
def test_distill_loss_masks(tt, kind, vocab):
    """-inf and the type's lowest value among the logits and among the teacher's."""
    kind, g = KINDS[kind], gen(6)
    low = torch.finfo(kind).min
    x = rows_of(7, vocab, kind, g, scale=2.0)
    x[0, vocab // 2:] = -math.inf
    x[1, : vocab // 2] = low
    x[2] = low
    x[3] = -math.inf
    x[4, 1:] = -math.inf
    ids = torch.arange(1, 13, dtype=torch.int32, device="cuda").repeat(7, 1)
    ids[1] += vocab // 2
    ids[4] = 0
    ids[4, 1:] = -1
    values = torch.randn(7, 12, generator=g, device="cuda")
    values[5, 3:] = torch.finfo(torch.float32).min
    values[6] = torch.finfo(torch.float32).min
    rg = torch.ones(7, device="cuda")
    loss, lse, d = tt.distill_loss(x, ids, values, 1.0, rg, want_grad=True)
    rows = torch.tensor([0, 1, 4, 5, 6], device="cuda")
    check_distill((loss[rows], lse[rows], d[rows]), x[rows], ids[rows], values[rows], 1.0, rg[rows])
    assert loss[3] == math.inf and lse[3] == -math.inf and not bool(d[3].any())
    # one value throughout: equal probabilities
    q = torch.softmax(values[2].double(), 0)
    want = torch.full((vocab,), 1 / vocab, dtype=torch.float64, device="cuda")
    want[1:13] -= q
    within(d[2], want, plain.rounded(want.abs() * plain.EPS * (64 + vocab / 64), want, kind))
    assert abs(loss[2].item() - float((q * torch.log(q)).sum() + math.log(vocab))) < 1e-5
    # an entry of some weight where the logit is -inf
    ids[0, 0] = vocab - 1
    assert tt.distill_loss(x, ids, values)[0][0].item() == math.inf
    # and one of none
    values[0, 0] = -math.inf
    assert math.isfinite(tt.distill_loss(x, ids, values)[0][0].item())


@pytest.mark.parametrize("vocab", [300, 70000])
def test_distill_loss_nan_stays_in_its_row(tt, vocab):
    g = gen(7)
    x = rows_of(6, vocab, torch.bfloat16, g, scale=2.0)
    ids, values = entries(6, vocab, 9, torch.float32, 3)
    ids[:] = ids.clamp(min=0)
    rg = torch.ones(6, device="cuda")
    want = tt.distill_loss(x, ids, values, 1.0, rg, want_grad=True)
    y, v = x.clone(), values.clone()
    y[1, vocab // 2] = math.nan
    y[2, vocab - 1] = math.inf
    v[3, 4] = math.nan
    v[4, 2] = math.inf
    loss, lse, d = tt.distill_loss(y, ids, v, 1.0, rg, want_grad=True)
    for i in (0, 5):
        assert torch.equal(loss[i], want[0][i]) and torch.equal(lse[i], want[1][i]) and torch.equal(d[i], want[2][i])
    assert bool(torch.isnan(lse[1])) and lse[2] == math.inf and torch.equal(lse[3:5], want[1][3:5])
    assert bool(torch.isnan(loss[[1, 3, 4]]).all()) and not bool(torch.isfinite(loss[2]))
    assert bool(torch.isnan(d[1]).all()) and bool(torch.isnan(d[2, vocab - 1]))


@pytest.mark.parametrize("temperature", [2.0**-20, 0.05, 1e3, 2.0**64])
def test_distill_loss_temperatures(tt, temperature):
    g = gen(8)
    x = rows_of(8, 3001, torch.float32, g, scale=2.0 * min(temperature, 1e4))
    ids, values = entries(8, 3001, 20, torch.float32, 5)
    values = values * min(temperature, 1e4)
    rg = torch.ones(8, device="cuda") * min(temperature, 1e4)
    check_distill(tt.distill_loss(x, ids, values, temperature, rg, want_grad=True), x, ids, values, temperature, rg)


def test_distill_loss_gradient_against_differences(tt):
    g = gen(9)
    x = rows_of(40, 777, torch.float32, g, scale=2.0)
    ids, values = entries(40, 777, 20, torch.float32, 6, repeat=3)
    rg = torch.rand(40, generator=g, device="cuda")
    d = tt.distill_loss(x, ids, values, 1.7, rg, want_grad=True)[2]
    u = rows_of(40, 777, torch.float32, g)
    total = lambda s: (tt.distill_loss(x + s * u, ids, values, 1.7)[0].double() * rg.double()).sum()  # noqa: E731
    step = 2.0**-6
    slope = (total(step) - total(-step)) / (2 * step)
    wide = (total(2 * step) - total(-2 * step)) / (4 * step)
    noise = (2 * (plain.distill(x, ids, values, 1.7, rg)[1][0]) * rg.double()).sum() / (2 * step)
    # and x + s u rounded to 32 bits
    moved = (d.double().abs() * x.double().abs() * 2 * plain.EPS).sum() / step
    assert abs(slope - (d.double() * u).sum()) <= 2 * abs(wide - slope) / 3 + noise + moved


def test_distill_loss_streams_and_graphs(tt):
    g = gen(10)
    x = rows_of(50, 60001, torch.bfloat16, g, scale=2.0)
    ids, values = entries(50, 60001, 30, torch.bfloat16, 6)
    want = tt.distill_loss(x, ids, values, 2.0, want_grad=True)
    s = torch.cuda.Stream()
    got = tt.distill_loss(x, ids, values, 2.0, want_grad=True, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tt.distill_loss(x, ids, values, 2.0, want_grad=True)
        later = tt.distill_loss_grad(x, ids, values, out[1], 2.0)
    for seed in (1, 2):
        x.copy_(torch.randn(50, 60001, generator=gen(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = tt.distill_loss(x, ids, values, 2.0, want_grad=True)
        assert all(torch.equal(a, b) for a, b in zip(want, out))
        assert torch.equal(later, tt.distill_loss_grad(x, ids, values, want[1], 2.0))


def test_distill_loss_offsets_past_32_bits(tt):
    n, vocab = 22000, 100256                               # 2.2e9 logits
    g = gen(11)
    x = torch.zeros(n, vocab, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 21419, 21420, 21421, n - 1], device="cuda")
    x[at] = torch.randn(5, vocab, generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, vocab, (n, 4), generator=g, device="cuda", dtype=torch.int32)
    values = torch.randn(n, 4, generator=g, device="cuda")
    rg = torch.ones(n, device="cuda")
    want, b = plain.distill(x[at], ids[at], values[at], 1.0, rg[at])
    loss, lse, d = tt.distill_loss(x, ids, values, 1.0, rg, dlogits=x)
    for got, w, e, kind in zip((loss[at], lse[at], d[at]), want, b, (torch.float32, torch.float32, torch.bfloat16)):
        within(got, w, plain.rounded(e, w, kind))


# ------------------------------------------------------------ together

def test_a_teacher_trains_a_student(tt):
    """Text to IDs, a teacher's hidden states scored without its logits, its top logits
    distilled into a student, whose table and head get their gradients: against the
    same model in torch doubles with torch's own differentiation."""
    from exact_bpe_tokenization_gb300 import synth
    merges, vb, vo = synth.make_vocab(synth.PROFILE_ASCII, 1 << 18, 300)
    vocab = len(vo) - 1
    tok = tt.Tokenizer(merges, vb, vo, tt.TT_FAMILY_CL100K_STYLE)
    data, offs = synth.batch([synth.transcript(3, 900, synth.PROFILE_ASCII), b"", synth.transcript(4, 500, synth.PROFILE_ASCII)])
    ids, io = tok.encode(torch.from_numpy(data).cuda(), torch.from_numpy(offs).cuda())
    n = int(io[-1].item())
    tok.close()
    ids = ids[:n].contiguous()
    targets = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    targets[:-1] = ids[1:]
    g = gen(21)
    dim, k, temperature = 32, 12, 2.0
    table = (torch.randn(vocab, dim, generator=g, device="cuda") * 0.5)
    head = (torch.randn(vocab, dim, generator=g, device="cuda") * 0.5)
    teacher = torch.randn(n, dim, generator=g, device="cuda")
    rg = torch.full((n,), 1 / n, device="cuda")
    # the teacher: scored without its logits; its top logits row by row
    scored, lse = tt.linear_loss(teacher, head, targets)
    top, at = torch.topk(teacher @ head.T, k, 1)
    # the student: both losses
    st = status_word()
    x = tt.embed(ids, table, status=st)
    loss, _, dx, dhead = tt.linear_loss(x, head, targets, rg, want_grad=True, status=st)
    logits = x @ head.T
    dloss, _, dl = tt.distill_loss(logits, at.int(), top, temperature, rg, dlogits=logits, status=st)
    dx = dx + dl @ head
    dhead = dhead + dl.T @ x
    dtable = tt.embed_grad(ids, dx, vocab, status=st)
    assert st.item() == 0
    # the same in doubles
    T, H = table.double().requires_grad_(), head.double().requires_grad_()
    X = T[ids.long()]
    y = X @ H.T
    there = targets >= 0
    one = torch.where(there, torch.logsumexp(y, 1) - y.gather(1, targets.clamp(min=0).long()[:, None])[:, 0], 0.0)
    q = torch.softmax(top.double() / temperature, 1)
    two = (q * (torch.log(q) - torch.log_softmax(y / temperature, 1).gather(1, at))).sum(1)
    ((one + two) / n).sum().backward()
    t_logits = teacher.double() @ head.double().T
    assert torch.allclose(lse.double(), torch.logsumexp(t_logits, 1), rtol=1e-5)
    assert torch.allclose(scored.double()[there], (torch.logsumexp(t_logits, 1) - t_logits.gather(1, targets.clamp(min=0).long()[:, None])[:, 0])[there],
                          rtol=1e-5, atol=1e-5)
    assert torch.allclose(loss.double(), one.detach(), rtol=1e-5, atol=1e-5)
    assert torch.allclose(dloss.double(), two.detach(), rtol=1e-5, atol=1e-5)
    # sums of n terms of up to 2 / n, in 32 bits
    assert torch.allclose(dtable.double(), T.grad, rtol=1e-4, atol=1e-6)
    assert torch.allclose(dhead.double(), H.grad, rtol=1e-4, atol=1e-6)
