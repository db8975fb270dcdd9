"""The operators around token IDs on the GPU against plain 64-bit forms
(ops_plain.py): types, odd sizes, strides and alignments, padding and invalid
IDs, masks that leave a row empty, infinities and NaN, ties, other streams,
graph capture, and sizes past 32-bit offsets.  Tolerances are error bounds of
32-bit arithmetic and of one rounding to the output's type."""
import math

import numpy as np
import pytest

import ops_plain as plain

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DTYPES = ["float32", "float16", "bfloat16"]


@pytest.fixture(scope="module")
def tt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from exact_bpe_tokenization_gb300 import binding
    return binding


def dtype(name):
    return getattr(torch, name)


def host(x):
    return x.detach().double().cpu().numpy()


def rows_of(n, d, name, gen, stride=None, shift=0, scale=1.0):
    """An [n, d] tensor of a type, its rows `stride` apart, its first element
    `shift` elements past a 16-byte boundary; what lies between is NaN."""
    stride = stride or d
    buf = torch.full((n * stride + shift + 8,), math.nan, dtype=dtype(name), device="cuda")
    x = buf[shift:shift + n * stride].view(n, stride)[:, :d] if n else buf[:0].view(0, d)
    if n:
        x.copy_(torch.randn(n, d, generator=gen, device="cuda") * scale)
    return x


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ embed

SHAPES = [(1, 1, 1), (1, 300, 8), (5, 7, 24), (33, 300, 64), (100, 4352, 257), (64, 300, 1024), (257, 1000, 641),
          (9, 50, 4104), (1000, 300, 40)]


@pytest.mark.parametrize("n,vocab,dim", SHAPES)
@pytest.mark.parametrize("ti", DTYPES)
@pytest.mark.parametrize("to", DTYPES)
def test_embed(tt, n, vocab, dim, ti, to):
    rng = np.random.default_rng(n + dim)
    ids = rng.integers(0, vocab, n).astype(np.int32)
    ids[rng.random(n) < 0.1] = -1
    scale = float(np.float32(math.sqrt(dim)))
    table = rows_of(vocab, dim, ti, gen(dim))
    got = host(tt.embed(torch.from_numpy(ids).cuda(), table, scale=scale, dtype=dtype(to)))
    want = plain.embed(ids, host(table), scale)
    # the product's rounding and the output's
    assert np.all(np.abs(got - want) <= (plain.UNIT[to] * 1.01 + plain.EPS) * np.abs(want) + plain.TINY[to])
    assert not got[ids < 0].any()


@pytest.mark.parametrize("stride,shift", [(24, 0), (31, 0), (24, 3), (32, 8), (29, 1)])
@pytest.mark.parametrize("name", DTYPES)
def test_embed_strides_and_alignments(tt, stride, shift, name):
    ids = torch.tensor([3, 0, 9, -5, 9, 2], dtype=torch.int32, device="cuda")
    table = rows_of(10, 24, name, gen(1), stride, shift)
    out = rows_of(6, 24, name, gen(2), stride, shift)
    tt.embed(ids, table, out=out)
    assert torch.equal(out, torch.where(ids[:, None] < 0, 0, table[ids.long().clamp(min=0)]))
    if stride > 24:                                       # nothing between the rows is written
        gaps = torch.as_strided(out, (5, stride - 24), (stride, 1), out.storage_offset() + 24)
        assert bool(torch.isnan(gaps).all())


def test_embed_count_on_the_device_and_invalid_ids(tt):
    ids = torch.tensor([1, 2, 300, 299, 0, -1, 5], dtype=torch.int32, device="cuda")
    for dim in (16, 17):
        table = rows_of(300, dim, "float32", gen(3))
        for count, stop in ((0, 0), (2, 2), (4, 4), (7, 7), (99, 7), (-3, 0)):
            out = torch.full((7, dim), 7.0, device="cuda")
            st = status_word()
            tt.embed(ids, table, scale=2.0, n_ids=torch.tensor([count], device="cuda"), out=out, status=st)
            want = torch.full((7, dim), 7.0, device="cuda")
            ok = (ids >= 0) & (ids < 300)
            want[:stop] = torch.where(ok[:, None], table[ids.long().clamp(0, 299)] * 2, 0)[:stop]
            assert torch.equal(out, want)
            assert st.item() == (tt.TT_ERR_INVALID_ARG if stop > 2 else 0)


@pytest.mark.parametrize("dim", [2304, 2305])
def test_embed_offsets_past_32_bits(tt, dim):
    vocab = 1 << 20                                        # 2^20 rows of 2304: 2.4e9 elements
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([vocab - 1, 0, vocab - 2, 932068], dtype=torch.int32, device="cuda")
    table[ids.long()] = torch.randn(4, dim, generator=gen(4), device="cuda").bfloat16()
    assert torch.equal(tt.embed(ids, table), table[ids.long()])
    del table
    n = 1000000                                            # and as many of the output
    small = torch.randn(300, dim, generator=gen(5), device="cuda").bfloat16()
    ids = torch.randint(0, 300, (n,), generator=gen(6), device="cuda", dtype=torch.int32)
    out = tt.embed(ids, small)
    at = torch.tensor([0, 1, 932066, 932067, 932068, n - 1], device="cuda")
    assert torch.equal(out[at], small[ids[at].long()])


# ------------------------------------------------------------ embed_grad

def grad_close(got, ids, dout, vocab, scale, to, base=None):
    want, size, count = plain.embed_grad(ids, host(dout), vocab, scale)
    if base is not None:
        want, size = want + base, size + np.abs(base)
    # each of count additions, the scale, the addition to what was there, and the output's rounding
    tol = plain.EPS * 1.01 * (count[:, None] + 3) * size + plain.UNIT[to] * 1.01 * np.abs(want) + plain.TINY[to]
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("n,vocab,dim", SHAPES)
@pytest.mark.parametrize("ti", DTYPES)
@pytest.mark.parametrize("to", DTYPES)
def test_embed_grad(tt, n, vocab, dim, ti, to):
    rng = np.random.default_rng(n + dim)
    ids = np.minimum(rng.zipf(1.3, n) - 1, vocab - 1).astype(np.int32)
    ids[rng.random(n) < 0.1] = -7
    dout = rows_of(n, dim, ti, gen(dim))
    got = tt.embed_grad(torch.from_numpy(ids).cuda(), dout, vocab, scale=0.75, dtype=dtype(to))
    grad_close(host(got), ids, dout, vocab, 0.75, to)


@pytest.mark.parametrize("n", [4095, 4096, 4097, 16384, 16385, 40000, 70001])
@pytest.mark.parametrize("kind", ["zipf", "one", "two", "distinct", "padding", "last"])
def test_embed_grad_token_counts(tt, n, kind):
    """Rows of one token and of all of them, around the sizes where blocks end."""
    rng = np.random.default_rng(n)
    vocab, dim = 5000, 16
    ids = {"zipf": np.minimum(rng.zipf(1.2, n) - 1, vocab - 1), "one": np.full(n, 3), "two": np.where(np.arange(n) < n // 3, 4999, 0),
           "distinct": np.arange(n) % vocab, "padding": np.full(n, -1), "last": np.full(n, vocab - 1)}[kind].astype(np.int32)
    dout = rows_of(n, dim, "float32", gen(n))
    got = tt.embed_grad(torch.from_numpy(ids).cuda(), dout, vocab)
    grad_close(host(got), ids, dout, vocab, 1.0, "float32")
    assert torch.equal(got, tt.embed_grad(torch.from_numpy(ids).cuda(), dout, vocab))    # the same bits again


@pytest.mark.parametrize("vocab", [1, 2, 3, 255, 256, 257, 65535, 65536, (1 << 20) - 1, 1 << 20])
def test_embed_grad_vocabularies(tt, vocab):
    """Every width of the sort's digits; the first and last rows."""
    rng = np.random.default_rng(vocab)
    n, dim = 3000, 8
    ids = rng.integers(0, vocab, n).astype(np.int32)
    ids[:3] = vocab - 1
    ids[3:5] = 0
    dout = rows_of(n, dim, "float32", gen(8))
    got = host(tt.embed_grad(torch.from_numpy(ids).cuda(), dout, vocab))
    want = np.zeros((vocab, dim))
    size = np.zeros((vocab, dim))
    np.add.at(want, ids, host(dout))
    np.add.at(size, ids, np.abs(host(dout)))
    count = np.bincount(ids, minlength=vocab)[:, None]
    assert np.all(np.abs(got - want) <= plain.EPS * 1.01 * (count + 3) * size)


@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("dim,stride,shift", [(16, 16, 0), (24, 31, 0), (17, 17, 1), (24, 32, 8), (24, 24, 5)])
def test_embed_grad_accumulates_strides_and_alignments(tt, name, dim, stride, shift):
    rng = np.random.default_rng(dim)
    n, vocab = 500, 300
    ids = rng.integers(0, vocab // 2, n).astype(np.int32)
    dout = rows_of(n, dim, name, gen(1), stride, shift)
    out = rows_of(vocab, dim, name, gen(2), stride, shift)
    base = host(out)
    tt.embed_grad(torch.from_numpy(ids).cuda(), dout, vocab, scale=-1.5, out=out, accumulate=True)
    grad_close(host(out), ids, dout, vocab, -1.5, name, base)
    assert np.array_equal(host(out)[vocab // 2:], base[vocab // 2:])
    tt.embed_grad(torch.from_numpy(ids).cuda(), dout, vocab, scale=-1.5, out=out)
    grad_close(host(out), ids, dout, vocab, -1.5, name)
    if stride > dim:
        gaps = torch.as_strided(out, (vocab - 1, stride - dim), (stride, 1), out.storage_offset() + dim)
        assert bool(torch.isnan(gaps).all())


def test_embed_grad_count_on_the_device_and_invalid_ids(tt):
    ids = np.array([1, 2, 300, 299, 0, -1, 2], dtype=np.int32)
    dout = rows_of(7, 16, "float32", gen(3))
    for count, stop in ((0, 0), (2, 2), (4, 4), (7, 7), (99, 7), (-3, 0)):
        st = status_word()
        got = tt.embed_grad(torch.from_numpy(ids).cuda(), dout, 300, n_ids=torch.tensor([count], device="cuda"), status=st)
        grad_close(host(got), ids[:stop], dout[:stop], 300, 1.0, "float32")
        assert st.item() == (tt.TT_ERR_INVALID_ARG if stop > 2 else 0)
    got = tt.embed_grad(torch.empty(0, dtype=torch.int32, device="cuda"), dout[:0], 300)
    assert got.shape == (300, 16) and not got.any()


def test_embed_grad_offsets_past_32_bits(tt):
    dim, vocab = 2304, 1 << 20
    ids = torch.tensor([vocab - 1, 0, vocab - 1, 932068], dtype=torch.int32, device="cuda")
    dout = torch.randn(4, dim, generator=gen(4), device="cuda").bfloat16()
    out = torch.full((vocab, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    tt.embed_grad(ids, dout, vocab, out=out)
    assert torch.equal(out[932068], dout[3]) and torch.equal(out[0], dout[1])
    assert torch.equal(out[vocab - 1], (dout[0].float() + dout[2].float()).bfloat16())
    assert sum(int(out[a:a + 65536].count_nonzero()) for a in range(0, vocab, 65536)) <= 3 * dim


def test_embed_grad_is_the_derivative_of_embed(tt):
    """embed is linear in its table, so a difference of any size is exact but
    for rounding: <dout, embed(t + s) - embed(t - s)> = 2 <grad, s>."""
    rng = np.random.default_rng(5)
    ids = torch.from_numpy(rng.integers(-1, 40, 300).astype(np.int32)).cuda()
    t, s, d = rows_of(40, 24, "float32", gen(1)), rows_of(40, 24, "float32", gen(2)), rows_of(300, 24, "float32", gen(3))
    a, b = host(tt.embed(ids, t + s, scale=3.0)), host(tt.embed(ids, t - s, scale=3.0))
    g = host(tt.embed_grad(ids, d, 40, scale=3.0))
    left, right = np.sum(host(d) * (a - b)), 2 * np.sum(g * host(s))
    size = np.sum(np.abs(host(d)) * (np.abs(a) + np.abs(b))) + 2 * np.sum(np.abs(g) * np.abs(host(s)))
    assert abs(left - right) <= plain.EPS * 32 * size


# ------------------------------------------------------------ token_loss

def check_loss(tt, x, targets, g, name, **kw):
    out = tt.token_loss(x, torch.from_numpy(targets).cuda(), None if g is None else torch.from_numpy(g).cuda(),
                        want_grad=True, **kw)
    xs = host(x)
    gs = np.ones(len(xs)) if g is None else g.astype(np.float64)
    loss, lse, d = plain.token_loss(xs, targets, gs)
    fine = np.isfinite(lse)
    tol = np.where(fine, plain.lse_bound(np.where(np.isfinite(xs), xs, -1e4), np.where(fine, lse, 0)), 0)
    got_loss, got_lse, got = (host(o) for o in out)
    assert np.array_equal(got_lse[~fine], lse[~fine])
    assert np.all(np.abs(got_lse[fine] - lse[fine]) <= tol[fine])
    lf = np.isfinite(loss)
    assert np.array_equal(got_loss[~lf], loss[~lf])
    assert np.all(np.abs(got_loss[lf] - loss[lf]) <= tol[lf] + plain.EPS * np.abs(loss[lf]))
    p = np.exp(np.where(fine[:, None], xs - np.where(fine, lse, 0)[:, None], -np.inf))
    far = np.where(np.isfinite(xs), np.abs(xs - np.where(fine, lse, 0)[:, None]), 0)
    # the exponent's error, exp's and the products', and the output's rounding
    dtol = np.abs(gs)[:, None] * (p * (tol[:, None] + plain.EPS * (far + 8)) + 3 * plain.EPS * (p > 0)) + \
        1.01 * plain.UNIT[name] * np.abs(d) + plain.TINY[name]
    assert np.all(np.abs(got - d) <= dtol)
    return out


LOSS_SHAPES = [(1, 1), (1, 2), (3, 7), (5, 257), (64, 4352), (7, 8191), (2, 65537), (3, 200255), (300, 1000), (1, 1 << 20)]


@pytest.mark.parametrize("n,vocab", LOSS_SHAPES)
@pytest.mark.parametrize("name", DTYPES)
def test_token_loss(tt, n, vocab, name):
    rng = np.random.default_rng(vocab)
    x = rows_of(n, vocab, name, gen(vocab), scale=3.0)
    targets = rng.integers(0, vocab, n).astype(np.int32)
    targets[rng.random(n) < 0.2] = -1
    check_loss(tt, x, targets, None, name)
    g = rng.standard_normal(n).astype(np.float32)
    out = check_loss(tt, x, targets, g, name)
    again = tt.token_loss(x, torch.from_numpy(targets).cuda(), torch.from_numpy(g).cuda(), want_grad=True)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    # the gradient alone, from lse, and the loss alone
    later = tt.token_loss_grad(x, torch.from_numpy(targets).cuda(), out[1], torch.from_numpy(g).cuda())
    assert torch.equal(later, out[2])
    alone = tt.token_loss(x, torch.from_numpy(targets).cuda())
    assert torch.equal(alone[0], out[0]) and torch.equal(alone[1], out[1])
    # in place
    y = x.clone()
    tt.token_loss(y, torch.from_numpy(targets).cuda(), torch.from_numpy(g).cuda(), dlogits=y)
    assert torch.equal(y, out[2])


@pytest.mark.parametrize("vocab,stride,shift", [(1000, 1000, 0), (1000, 1003, 0), (1000, 1000, 1), (1001, 1008, 8),
                                                (999, 1001, 5), (70001, 70003, 3)])
@pytest.mark.parametrize("name", DTYPES)
def test_token_loss_strides_and_alignments(tt, vocab, stride, shift, name):
    rng = np.random.default_rng(stride)
    x = rows_of(6, vocab, name, gen(stride), stride, shift)
    targets = rng.integers(0, vocab, 6).astype(np.int32)
    out = check_loss(tt, x, targets, None, name)
    for st, sh in ((vocab, 0), (vocab + 5, 2)):
        d = rows_of(6, vocab, name, gen(1), st, sh)
        tt.token_loss(x, torch.from_numpy(targets).cuda(), dlogits=d)
        assert torch.equal(d, out[2])
        if st > vocab:
            assert bool(torch.isnan(torch.as_strided(d, (5, st - vocab), (st, 1), d.storage_offset() + vocab)).all())
    tt.token_loss(x, torch.from_numpy(targets).cuda(), dlogits=x)
    assert torch.equal(x, out[2])


@pytest.mark.parametrize("vocab", [50, 5000, 120001])
@pytest.mark.parametrize("name", DTYPES)
def test_token_loss_masks(tt, vocab, name):
    """-inf logits; a target under the mask; one token left; none left; the type's lowest value as a mask."""
    x = rows_of(8, vocab, name, gen(7))
    targets = np.array([0, 1, 2, 3, 4, 5, vocab - 1, 7], dtype=np.int32)
    x[0, 1:] = -math.inf                                   # only the target left
    x[1, 1] = -math.inf                                    # the target masked
    x[2] = -math.inf                                       # nothing left
    x[3, : vocab // 2] = -math.inf
    x[3, 3] = 0.5
    x[4] = torch.finfo(dtype(name)).min                    # a row of the lowest value: uniform
    x[5, 6:] = torch.finfo(dtype(name)).min
    x[6, : vocab - 1] = -math.inf
    x[7] = torch.finfo(dtype(name)).max                    # large and equal
    xs = host(x)
    loss, lse, d = (host(o) for o in tt.token_loss(x, torch.from_numpy(targets).cuda(), want_grad=True))
    assert loss[0] == 0 and not d[0].any() and loss[6] == 0 and not d[6].any()
    assert loss[1] == math.inf and abs(d[1].sum()) <= 2.0**-7 and d[1, 1] == -1
    assert loss[2] == math.inf and lse[2] == -math.inf and not d[2].any()
    for r in (4, 7):
        # lse is the common value to within a rounding of it: the loss is that rounding's size, and the gradient follows lse
        assert abs(lse[r] - xs[r, 0]) <= 2 * plain.EPS * abs(xs[r, 0]) + math.log(vocab) * 2
        assert np.isfinite(loss[r]) and np.isfinite(d[r]).all()
    check_loss(tt, x[[0, 1, 2, 3, 5, 6]], targets[[0, 1, 2, 3, 5, 6]], None, name)


@pytest.mark.parametrize("vocab", [10, 3000, 120001])
def test_token_loss_nan_and_infinity(tt, vocab):
    x = rows_of(5, vocab, "float32", gen(9))
    x[0, 3], x[1, 2], x[2, 2], x[3, 0], x[3, 1] = math.nan, math.inf, math.inf, math.inf, math.nan
    targets = torch.tensor([1, 1, 2, 4, 4], dtype=torch.int32, device="cuda")
    loss, lse, d = (host(o) for o in tt.token_loss(x, targets, want_grad=True))
    assert math.isnan(lse[0]) and math.isnan(loss[0]) and np.isnan(d[0]).all()
    assert lse[1] == math.inf and loss[1] == math.inf and math.isnan(d[1, 2]) and d[1, 1] == -1 and d[1, 0] == 0
    assert lse[2] == math.inf and math.isnan(loss[2]) and math.isnan(d[2, 2])
    assert math.isnan(lse[3]) and np.isnan(d[3]).all()
    assert np.isfinite(loss[4]) and np.isfinite(d[4]).all()      # its neighbours say nothing about a row


def test_token_loss_targets_beyond_the_vocabulary(tt):
    x = rows_of(3, 100, "float32", gen(1))
    for bad in (100, 1 << 20, 2**31 - 1):
        st = status_word()
        t = torch.tensor([5, bad, -4], dtype=torch.int32, device="cuda")
        loss, lse, d = tt.token_loss(x, t, want_grad=True, status=st)
        assert st.item() == tt.TT_ERR_INVALID_ARG
        assert loss[1:].tolist() == [0, 0] and not d[1:].any() and torch.isfinite(lse).all()
    st = status_word()
    tt.token_loss(x, torch.tensor([5, -1, -4], dtype=torch.int32, device="cuda"), status=st)
    assert st.item() == 0


def test_token_loss_grad_is_the_derivative(tt):
    """Central differences along a direction of entries in [-1, 1]: the third
    derivative of log-sum-exp along it is a third central moment of values in
    that range, at most 2, so the truncation is below h^2 / 3 a row."""
    rng = np.random.default_rng(3)
    n, vocab, h = 20, 500, 2.0**-6
    x = rows_of(n, vocab, "float32", gen(3))
    v = (torch.rand(n, vocab, generator=gen(4), device="cuda") * 2 - 1).float()
    targets = torch.from_numpy(rng.integers(0, vocab, n).astype(np.int32)).cuda()
    up, down = x + h * v, x - h * v
    a, b = tt.token_loss(up, targets), tt.token_loss(down, targets)
    d = tt.token_loss(x, targets, want_grad=True)[2]
    along = (host(d) * host(v)).sum(1)
    bound = plain.lse_bound(host(x), host(a[1])) + plain.EPS * 16
    assert np.all(np.abs((host(a[0]) - host(b[0])) / (2 * h) - along) <= h * h / 3 + 2 * bound / h)


def test_token_loss_offsets_past_32_bits(tt):
    vocab, n = 1 << 20, 2100                               # 2.2e9 logits
    x = torch.zeros(n, vocab, dtype=torch.bfloat16, device="cuda")
    x[n - 1, 5] = 20.0
    x[n - 1, vocab - 1] = 21.0
    targets = torch.full((n,), 5, dtype=torch.int32, device="cuda")
    tt_loss, lse, d = tt.token_loss(x, targets, dlogits=x)
    z = math.log(math.exp(20) + math.exp(21) + vocab - 2)
    assert abs(lse[n - 1].item() - z) <= 1e-4 and abs(lse[0].item() - math.log(vocab)) <= 1e-4
    assert abs(d[n - 1, vocab - 1].item() - math.exp(21 - z)) <= 2.0**-8 and abs(d[n - 1, 5].item() - math.exp(20 - z) + 1) <= 2.0**-8
    assert d[2050, 5].item() == -1.0 and abs(d[2050, 6].item() * vocab - 1) <= 2.0**-7


# ------------------------------------------------------------ sample

def exp2_gpu(y):
    """The 32-bit power of the header, from the same device."""
    return torch.exp2(torch.from_numpy(np.ascontiguousarray(y)).cuda()).cpu().numpy()


def params(n, rng):
    return dict(temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.0, 1.5, 10.0, 1e-30, 1e30], n).astype(np.float32),
                top_k=rng.choice([0, -1, 1, 2, 7, 50, 1000, 1 << 30], n).astype(np.int32),
                top_p=rng.choice([1.0, 1.0, 0.0, 0.1, 0.5, 0.9, 0.95, 0.999], n).astype(np.float32),
                min_p=rng.choice([0.0, 0.0, 0.0, 1e-12, 0.01, 0.3, 1.0], n).astype(np.float32))


def check_sample(tt, x, uniform, p, pick=None):
    """Every row of x, or those of `pick`, against the plain form."""
    dev = {k: torch.from_numpy(v).cuda() for k, v in p.items()}
    st = status_word()
    ids, lp = tt.sample(x, torch.from_numpy(uniform).cuda(), status=st, **dev)
    assert st.item() == 0
    ids, lp = ids.cpu().numpy(), lp.cpu().numpy()
    one = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    for r in range(len(uniform)) if pick is None else pick:
        q = {k: p[k][r] if k in p else one[k] for k in one}
        w = plain.sample_weights(x[r].float().cpu().numpy(), q["temperature"], exp2_gpu)
        want, want_lp = plain.sample(w, uniform[r], q["temperature"], int(q["top_k"]), q["top_p"], q["min_p"])
        assert ids[r] == want, (r, q, uniform[r])
        if want < 0:
            assert lp[r] == -math.inf
        else:   # the quotient's roundings (in the argument, so absolute in the logarithm) and the logarithm's
            assert abs(lp[r] - want_lp) <= 4 * plain.EPS * (1 + abs(want_lp))
    return ids


SAMPLE_SHAPES = [(4, 1), (8, 2), (40, 33), (64, 1000), (48, 4352), (24, 8193), (16, 50001), (12, 100256), (6, 200255), (2, 1 << 20)]


@pytest.mark.parametrize("n,vocab", SAMPLE_SHAPES)
@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("spread", [0.5, 4.0])
def test_sample(tt, n, vocab, name, spread):
    rng = np.random.default_rng(vocab + int(spread))
    x = rows_of(n, vocab, name, gen(vocab), scale=spread)
    u = rng.random(n).astype(np.float32)
    u[0] = 0
    u[-1] = np.float32(1) - np.float32(2.0**-24)
    u = np.minimum(u, np.float32(1) - np.float32(2.0**-24))
    check_sample(tt, x, u, params(n, rng))
    check_sample(tt, x, u, {}, range(0, n, 4))


@pytest.mark.parametrize("vocab", [5, 1000, 30000, 131072])
@pytest.mark.parametrize("top_k", [0, 1, 3, 900, 20000])
@pytest.mark.parametrize("top_p", [1.0, 0.0, 0.3, 0.77])
def test_sample_ties(tt, vocab, top_k, top_p):
    """Rows of one value, of two, and of few: equal weights are ranked by ID."""
    rng = np.random.default_rng(vocab + top_k)
    x = torch.empty(8, vocab, dtype=torch.bfloat16, device="cuda")
    x[0] = 1.5
    x[1] = 1.5
    x[1, vocab // 2:] = 0.5
    x[2] = torch.from_numpy(rng.integers(0, 3, vocab)).cuda()
    x[3] = torch.from_numpy(rng.integers(0, 30, vocab)).cuda()
    x[4] = -40.0
    x[4, vocab // 3:] = -41.0
    x[5] = 0.0
    x[5, 1::2] = -0.0                                       # zeros of both signs are equal
    x[6] = torch.finfo(torch.bfloat16).min                  # a row of the lowest value
    x[7] = torch.finfo(torch.bfloat16).min
    x[7, vocab - 1] = 1.0
    u = rng.random(8).astype(np.float32)
    u = np.minimum(u, np.float32(1) - np.float32(2.0**-24))
    p = dict(top_k=np.full(8, top_k, np.int32), top_p=np.full(8, top_p, np.float32))
    check_sample(tt, x, u, p)
    for k in range(3):
        check_sample(tt, x, np.float32([0, 0.25, 0.5, 0.75, 0.999, 0.1, 0.9, 0.3]), {**p, "temperature": np.full(8, [0.0, 0.1, 5.0][k], np.float32)})


@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("vocab", [6, 3001, 120000])
def test_sample_masks_infinities_and_nan(tt, name, vocab):
    rng = np.random.default_rng(vocab)
    x = rows_of(9, vocab, name, gen(11))
    x[0] = -math.inf                                        # nothing to draw
    x[1] = math.nan
    x[2] = -math.inf
    x[2, vocab - 1] = -3.0                                  # one token left
    x[3, ::2] = -math.inf
    x[4, 1::3] = math.nan
    x[5, 2] = x[5, vocab - 2] = math.inf                    # +inf takes all the weight
    x[6, : vocab - 2] = math.nan
    x[6, vocab - 2] = -math.inf
    x[7] = -math.inf
    x[7, 0] = math.inf
    p = params(9, rng)
    for k in range(4):
        u = np.minimum(rng.random(9).astype(np.float32), np.float32(1) - np.float32(2.0**-24))
        ids = check_sample(tt, x, u, p if k else {})
        assert ids[0] == ids[1] == -1 and ids[2] == vocab - 1 and ids[5] in (2, vocab - 2) and ids[6] == vocab - 1 and ids[7] == 0


@pytest.mark.parametrize("vocab,stride,shift", [(1000, 1003, 0), (1000, 1000, 1), (1001, 1008, 8), (999, 1001, 5), (70001, 70003, 3)])
@pytest.mark.parametrize("name", DTYPES)
def test_sample_strides_and_alignments(tt, vocab, stride, shift, name):
    rng = np.random.default_rng(stride)
    x = rows_of(16, vocab, name, gen(stride), stride, shift, scale=2.0)
    check_sample(tt, x, rng.random(16).astype(np.float32) * np.float32(0.999), params(16, rng))


def test_sample_refuses_parameters_row_by_row(tt):
    x = rows_of(8, 500, "float32", gen(1))
    good = dict(uniform=0.5, temperature=1.0, top_p=0.9, min_p=0.1)
    for key, values in dict(uniform=[-0.1, 1.0, math.nan], temperature=[-1.0, math.inf, math.nan],
                            top_p=[-0.1, 1.5, math.nan], min_p=[-0.5, 1.01, math.nan]).items():
        for bad in values:
            a = {k: torch.full((8,), v, device="cuda") for k, v in good.items()}
            want = tt.sample(x, **a)[0]
            a[key][3] = bad
            st = status_word()
            ids, lp = tt.sample(x, status=st, **a)
            assert st.item() == tt.TT_ERR_INVALID_ARG and ids[3] == -1 and lp[3] == -math.inf
            want[3] = -1
            assert torch.equal(ids, want)


def test_sample_draws_what_the_softmax_says(tt):
    """Against 64-bit weights: the drawn ID's interval of the distribution
    function holds u, to within the 32-bit exponent's error (its argument up to
    42 with two roundings, the power's two units) and 2^-41 a token."""
    rng = np.random.default_rng(2)
    for vocab in (300, 20000, 150001):
        x = rows_of(64, vocab, "float32", gen(vocab), scale=1.5)
        u = (rng.random(64) * 0.9999).astype(np.float32)
        ids = tt.sample(x, torch.from_numpy(u).cuda())[0].cpu().numpy()
        xs = host(x)
        p = np.exp(xs - xs.max(1, keepdims=True))
        c = np.cumsum(p, 1)
        tol = 2 * plain.EPS * (2 * 42 + 4) + vocab * 2.0**-41 / c[:, -1] + 2.0**-50
        lo = (c - p)[np.arange(64), ids] / c[:, -1]
        hi = c[np.arange(64), ids] / c[:, -1]
        assert np.all(lo - tol <= u) and np.all(u <= hi + tol)


def test_sample_does_not_depend_on_the_batch(tt):
    rng = np.random.default_rng(4)
    n, vocab = 300, 30001
    x = rows_of(n, vocab, "bfloat16", gen(4), scale=2.0)
    p = {k: torch.from_numpy(v).cuda() for k, v in params(n, rng).items()}
    u = torch.from_numpy(rng.random(n).astype(np.float32) * np.float32(0.9999)).cuda()
    ids, lp = tt.sample(x, u, **p)
    for r in (0, 17, 299):
        one = tt.sample(x[r:r + 1], u[r:r + 1], **{k: v[r:r + 1] for k, v in p.items()})
        assert one[0][0] == ids[r] and one[1][0] == lp[r]


def test_sample_offsets_past_32_bits(tt):
    vocab, n = 1 << 20, 2100
    x = torch.full((n, vocab), -math.inf, dtype=torch.bfloat16, device="cuda")
    want = torch.randint(0, vocab, (n,), generator=gen(5), device="cuda")
    x.scatter_(1, want[:, None], 1.0)
    ids, lp = tt.sample(x, torch.rand(n, generator=gen(6), device="cuda"))
    assert torch.equal(ids.long(), want) and not lp.any()


# ------------------------------------------------------------ all of them

def test_other_streams(tt):
    """Work goes to the given stream, ordered after what is there."""
    s = torch.cuda.Stream()
    ids = torch.randint(-1, 500, (3000,), generator=gen(1), device="cuda", dtype=torch.int32)
    table = torch.randn(500, 64, generator=gen(2), device="cuda")
    u = torch.rand(64, generator=gen(3), device="cuda")
    torch.cuda.synchronize()
    want = tt.embed(ids, table)
    grad = tt.embed_grad(ids, want, 500)
    loss = tt.token_loss(table, ids[:500].clamp(max=63), want_grad=True)
    drawn = tt.sample(table[:64], u)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        late = torch.full_like(table, math.nan)
        torch.cuda._sleep(20_000_000)
        late.copy_(table)
    for raw in (s, s.cuda_stream):
        out = tt.embed(ids, late, stream=raw)
        g = tt.embed_grad(ids, out, 500, stream=raw)
        ls = tt.token_loss(late, ids[:500].clamp(max=63), want_grad=True, stream=raw)
        dr = tt.sample(late[:64], u, stream=raw)
        s.synchronize()
        assert torch.equal(out, want) and torch.equal(g, grad)
        assert all(torch.equal(a, b) for a, b in zip(ls, loss)) and all(torch.equal(a, b) for a, b in zip(dr, drawn))


def test_graph_capture(tt):
    ids = torch.randint(0, 300, (5000,), generator=gen(1), device="cuda", dtype=torch.int32)
    table = torch.randn(300, 40, generator=gen(2), device="cuda")
    u = torch.rand(300, generator=gen(3), device="cuda")

    def step():
        out = tt.embed(ids, table, scale=2.0)
        g = tt.embed_grad(ids, out, 300)
        return (out, g) + tuple(tt.token_loss(g, ids[:300].clamp(max=39), want_grad=True)) + tuple(tt.sample(g, u))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    ids.copy_(torch.randint(0, 300, (5000,), generator=gen(5), device="cuda", dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_from_the_tokenizer(tt):
    """IDs and their count as an encode leaves them on the device."""
    from exact_bpe_tokenization_gb300 import synth
    merges, vb, vo = synth.make_vocab(synth.PROFILE_MIXED, 1 << 20, 2000)
    tok = tt.Tokenizer(merges, vb, vo, 1)
    data, offs = synth.batch([synth.transcript(3 + i, 2000 + 500 * i, synth.PROFILE_MIXED) for i in range(5)])
    ids, io = tok.encode(torch.from_numpy(data).cuda(), torch.from_numpy(offs).cuda())
    vocab = len(vo) - 1
    table = torch.randn(vocab, 32, generator=gen(1), device="cuda")
    out = torch.full((len(ids), 32), 9.0, device="cuda")
    st = status_word()
    tt.embed(ids, table, n_ids=io[-1:], out=out, status=st)
    g = tt.embed_grad(ids, out, vocab, n_ids=io[-1:], status=st)
    n = int(io[-1])
    assert 0 < n < len(ids) and st.item() == 0
    assert torch.equal(out[:n], table[ids[:n].long()]) and bool((out[n:] == 9).all())
    count = torch.bincount(ids[:n].long(), minlength=vocab)
    # equal terms: the sum of c copies, each addition rounded
    assert bool(((g - count[:, None] * table).abs() <= plain.EPS * count[:, None]**2 * table.abs()).all())
    tok.close()


def test_example(tt, capsys):
    """The example trains (its loss falls well below the uniform one) and what it
    draws are IDs of its vocabulary."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "bigram.py")
    spec = importlib.util.spec_from_file_location("bigram", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, drawn = m.main(["--steps", "30", "--tokens", "8"])
    assert losses[-1] < losses[0] - 0.5
    assert drawn.shape == (2, 8) and drawn.min() >= 0 and drawn.max() < 1256


# ------------------------------------------------------------ where the kernels' ways part

@pytest.mark.parametrize("n,vocab", [(17, 20011), (73, 20011), (100, 40001), (153, 20011), (300, 17001), (400, 1003), (33, 200255)])
@pytest.mark.parametrize("name", ["float32", "bfloat16"])
def test_sample_batches(tt, n, vocab, name):
    """Batches of every cluster size, their rows a mix of listed ones and ones
    that need histograms."""
    rng = np.random.default_rng(n)
    x = rows_of(n, vocab, name, gen(n), scale=2.0)
    u = np.minimum(rng.random(n).astype(np.float32), np.float32(1) - np.float32(2.0**-24))
    check_sample(tt, x, u, params(n, rng), range(0, n, max(1, n // 40)))


@pytest.mark.parametrize("vocab", [3000, 50000, 200001])
@pytest.mark.parametrize("rows", [3, 40])
def test_sample_flat_rows(tt, vocab, rows):
    """Prefixes that end among thousands of nearly equal weights, at shares
    from a single token to all but one."""
    rng = np.random.default_rng(vocab)
    x = rows_of(rows, vocab, "float32", gen(vocab), scale=0.01)
    x[1] *= 100
    x[2] = torch.round(x[2] * 200)
    p = dict(top_p=np.float32([0.5, 0.999999, 0.9, 1e-6] * 10)[:rows],
             top_k=np.int32([0, 0, 0, vocab - 1, 2000, vocab // 2, 97, 512, 1793, 0] * 4)[:rows],
             min_p=np.float32([0.0, 0.0, 1e-3, 0.0, 0.98] * 8)[:rows],
             temperature=np.float32([1.0, 0.5, 1.0, 2.0] * 10)[:rows])
    for k in range(3):
        u = np.minimum(rng.random(rows).astype(np.float32), np.float32(1) - np.float32(2.0**-24))
        check_sample(tt, x, u, p)


@pytest.mark.parametrize("n,vocab,dim", [(100, 5000, 641), (3000, 20000, 72), (2000, 8000, 9), (40000, 200000, 16)])
@pytest.mark.parametrize("to", ["float32", "bfloat16"])
@pytest.mark.parametrize("stride", [0, 5, 8])
def test_embed_grad_few_tokens(tt, n, vocab, dim, to, stride):
    """Tables of mostly absent rows: cleared, not added to; gaps left alone."""
    rng = np.random.default_rng(n)
    ids = np.minimum(rng.zipf(1.3, n) * 7 % vocab, vocab - 1).astype(np.int32)
    ids[rng.random(n) < 0.1] = -1
    dout = rows_of(n, dim, "float32", gen(n))
    out = rows_of(vocab, dim, to, gen(2), dim + stride)
    tt.embed_grad(torch.from_numpy(ids).cuda(), dout, vocab, out=out)
    want = np.zeros((vocab, dim))
    size = np.zeros((vocab, dim))
    there = ids >= 0
    np.add.at(want, ids[there], host(dout)[there])
    np.add.at(size, ids[there], np.abs(host(dout)[there]))
    count = np.bincount(ids[there], minlength=vocab)[:, None]
    tol = plain.EPS * 1.01 * (count + 3) * size + plain.UNIT[to] * 1.01 * np.abs(want)
    assert np.all(np.abs(host(out) - want) <= tol)
    if stride:
        gaps = torch.as_strided(out, (vocab - 1, stride), (dim + stride, 1), out.storage_offset() + dim)
        assert bool(torch.isnan(gaps).all())


def test_loss_and_lookup_of_many_rows(tt):
    """More rows than run at once, of sizes that leave blocks partly filled."""
    x = rows_of(5000, 777, "bfloat16", gen(1))
    targets = torch.randint(-1, 777, (5000,), generator=gen(2), device="cuda", dtype=torch.int32)
    loss, lse, d = tt.token_loss(x, targets, want_grad=True)
    want, want_lse, want_d = plain.token_loss(host(x), targets.cpu().numpy(), np.ones(5000))
    tol = plain.lse_bound(host(x), want_lse)
    assert np.all(np.abs(host(loss) - want) <= tol + plain.EPS * np.abs(want)) and np.all(np.abs(host(lse) - want_lse) <= tol)
    assert np.all(np.abs(host(d) - want_d) <= plain.UNIT["bfloat16"] * 1.01 * np.abs(want_d) + tol[:, None] + 20 * plain.EPS)
    ids = torch.randint(0, 300, (100001,), generator=gen(3), device="cuda", dtype=torch.int32)
    table = rows_of(300, 264, "float16", gen(4))
    assert torch.equal(tt.embed(ids, table), table[ids.long()])


@pytest.mark.parametrize("name,vocab", [(name, edge // size + more) for name, size in (("float32", 4), ("bfloat16", 2))
                                        for edge in (4096, 32768) for more in (-1, 0, 1)] + [("float16", 16385), ("float32", 33)])
@pytest.mark.parametrize("shift", [0, 3])
def test_token_loss_at_the_sizes_that_choose_the_threads(tt, name, vocab, shift):
    rng = np.random.default_rng(vocab)
    x = rows_of(9, vocab, name, gen(vocab), vocab + 2, shift)
    targets = rng.integers(0, vocab, 9).astype(np.int32)
    targets[:3] = 0, vocab - 1, -1
    out = check_loss(tt, x, targets, None, name)
    t = torch.from_numpy(targets).cuda()
    alone = tt.token_loss(x, t)
    assert torch.equal(alone[0], out[0]) and torch.equal(alone[1], out[1])
    assert torch.equal(tt.token_loss_grad(x, t, out[1]), out[2])
    tt.token_loss(x, t, dlogits=x)
    assert torch.equal(x, out[2])


@pytest.mark.parametrize("dim", [9, 31, 33, 129, 1025])
@pytest.mark.parametrize("name", DTYPES)
def test_embed_grad_of_odd_widths(tt, dim, name):
    ids = torch.randint(-1, 40, (900,), generator=gen(dim), device="cuda", dtype=torch.int32)
    dout = rows_of(900, dim, name, gen(dim), dim + 1, 1)
    got = tt.embed_grad(ids, dout, 40)
    k = ids.cpu().numpy()
    rows, want, size = host(dout), np.zeros((40, dim)), np.zeros((40, dim))
    np.add.at(want, k[k >= 0], rows[k >= 0])
    np.add.at(size, k[k >= 0], np.abs(rows[k >= 0]))
    count = np.bincount(k[k >= 0], minlength=40)[:, None]
    assert np.all(np.abs(host(got) - want) <= plain.EPS * 1.01 * (count + 3) * size)


@pytest.mark.parametrize("n,vocab,name", [(152, 9001, "bfloat16"), (153, 9001, "float16"), (200, 3001, "float32"),
                                          (37, 131072, "float32"), (64, 200255, "float32"), (15, 100256, "float32"),
                                          (36, 100256, "bfloat16"), (76, 60001, "bfloat16")])
def test_sample_on_both_sides_of_the_rules(tt, n, vocab, name):
    """Peaked, flat, tied and masked rows, cut in every way, in the sizes that
    decide how a row is divided and by which kernel it is drawn."""
    rng = np.random.default_rng(n + vocab)
    x = rows_of(n, vocab, name, gen(n), scale=3.0)
    x[1::7] *= 0.1                                            # flat
    x[2::7] = (x[2::7] * 0.5).round()                         # ties
    x[3::7, vocab // 3:] = -math.inf
    x[4::7, ::2] = math.nan
    x[min(5, n - 1)] = -math.inf
    x[min(6, n - 1), vocab // 2] = math.inf
    p = dict(temperature=rng.choice([0.0, 0.7, 1.0, 1.5], n).astype(np.float32),
             top_k=rng.choice([0, 0, 1, 40, 97, 700, vocab // 2], n).astype(np.int32),
             top_p=rng.choice([1.0, 0.9, 0.4], n).astype(np.float32),
             min_p=rng.choice([0.0, 0.0, 0.02], n).astype(np.float32))
    pick = range(n) if n * vocab <= 2_000_000 else sorted(rng.choice(n, 24, replace=False).tolist() + [1, 2, 3, 4, 5, 6])
    check_sample(tt, x, rng.random(n).astype(np.float32), p, pick)


@pytest.mark.parametrize("vocab", [7, 5000, 100256])
@pytest.mark.parametrize("name", DTYPES)
def test_sample_at_the_ends_of_the_parameters(tt, vocab, name):
    """The least and the largest values the header allows, denormal ones among
    them: temperatures whose reciprocal overflows or is denormal, shares and
    random numbers below the least weight."""
    tiny, least = np.float32(1e-45), np.float32(2.0**-126)
    under_one = np.float32(1) - np.float32(2.0**-24)
    rng = np.random.default_rng(vocab)
    n = 24
    x = rows_of(n, vocab, name, gen(vocab + 5), scale=2.0)
    pick = lambda *v: rng.choice(np.array(v, np.float32), n)  # noqa: E731
    for _ in range(3):
        check_sample(tt, x, pick(0, tiny, least, 2.0**-41, under_one),
                     dict(temperature=pick(0, tiny, least, 3e38, np.finfo(np.float32).max, 1),
                          top_k=rng.choice([0, -(1 << 31), 1, vocab - 1, vocab, (1 << 31) - 1], n).astype(np.int32),
                          top_p=pick(0, tiny, least, 2.0**-41, under_one, 1),
                          min_p=pick(0, tiny, 2.0**-41, 2.0**-40, 1.5 * 2.0**-40, under_one, 1)))


@pytest.mark.parametrize("dim", [7, 24, 1024])
@pytest.mark.parametrize("scale", [-2.0, math.inf, math.nan])
@pytest.mark.parametrize("name", DTYPES)
def test_padding_is_zero_whatever_the_scale(tt, dim, scale, name):
    """Rows of padding, and table rows of IDs that do not occur, are +0: their
    zeros are not multiplied."""
    table = rows_of(50, dim, name, gen(dim))
    ids = torch.tensor([3, -1, 49, -7, 0, 50, 3], dtype=torch.int32, device="cuda")
    out = tt.embed(ids, table, scale)
    zero = torch.tensor([1, 3, 5], device="cuda")
    assert not out[zero].any() and not torch.signbit(out[zero]).any()
    want = (table[[3, 49, 0, 3]].double() * scale).to(out.dtype)
    assert torch.equal(out[[0, 2, 4, 6]].isnan(), want.isnan()) and torch.equal(out[[0, 2, 4, 6]].nan_to_num(1), want.nan_to_num(1))
    for n in (7, 2000):                                     # rows mostly absent, and mostly there
        some = (torch.arange(n, device="cuda") % 40).int()
        d = tt.embed_grad(some, rows_of(n, dim, name, gen(n)), 50, scale)
        absent = d[min(n, 40):]
        assert not absent.any() and not torch.signbit(absent).any()
