"""The operators around token IDs where a result is easily lost unnoticed:
gradients of whole numbers, whose sums are exact whatever their order, on every
way through the sort and the sums; losses of rows far from zero; zeros of either
sign among the sampling parameters."""
import math

import numpy as np
import pytest

import ops_plain as plain
from test_gpu_ops import DTYPES, check_sample, dtype, gen, host, rows_of, status_word, tt  # noqa: F401 (tt: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ------------------------------------------------------------ embed_grad, exactly

def whole_rows(n, d, name, seed, stride=None, shift=0):
    """[n, d] whole numbers of -8 .. 8, all different sums."""
    x = rows_of(n, d, name, gen(seed), stride, shift)
    for a in range(0, n, 65536):
        m = min(65536, n - a)
        x[a:a + m] = torch.randint(-8, 9, (m, d), generator=gen(seed + a), device="cuda").to(dtype(name))
    return x


def ids_of(kind, n, vocab, rng):
    if kind == "zipf":
        ids = np.minimum(rng.zipf(1.2, n) - 1, vocab - 1)
    elif kind == "one":
        ids = np.full(n, min(3, vocab - 1))
    elif kind == "last":
        ids = np.full(n, vocab - 1)
    elif kind == "two":
        ids = np.where(np.arange(n) < n // 3, vocab - 1, 0)
    elif kind == "runs":         # rows of 62 .. 65 tokens, whose places drift against every cut
        ids = np.repeat(np.arange(vocab), np.resize([62, 63, 64, 65, 63, 64, 62], vocab))
        ids = np.concatenate([ids[:n], rng.integers(0, vocab, max(0, n - len(ids)))])
        rng.shuffle(ids)
    else:                        # "mixed": a row of a third, rows of one, padding and invalid IDs
        ids = rng.integers(-1, vocab + 1, n)
        ids[rng.random(n) < 0.3] = vocab // 2
    return torch.from_numpy(ids.astype(np.int32)).cuda()


def whole_sums(ids, dout, vocab):
    """The sums by ID, in 64 bits, and that 32 hold every partial one."""
    there = (ids >= 0) & (ids < vocab)
    at = ids[there].long()
    want = torch.zeros(vocab, dout.shape[1], dtype=torch.float64, device="cuda")
    for a in range(0, dout.shape[1], 64):
        want[:, a:a + 64] = want[:, a:a + 64].index_add(0, at, dout[there, a:a + 64].double())
    assert 8 * int(torch.bincount(at, minlength=1).max()) < 1 << 24
    return want


def check_whole(tt, ids, dout, vocab, to="float32", **kw):
    want = whole_sums(ids, dout, vocab)
    got = tt.embed_grad(ids, dout, vocab, scale=0.5, dtype=dtype(to), **kw)
    assert torch.equal(got, (want * 0.5).float().to(dtype(to)))
    return want


KINDS = ["zipf", "one", "last", "two", "runs", "mixed"]


@pytest.mark.parametrize("n", [1, 31, 4097, 16384, 70001, 131072, 131073, 300000, 1048576, 1048577, 1500000])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [8, 7])
def test_embed_grad_of_whole_numbers(tt, n, kind, dim):
    """Two, four and eight tokens a thread of the sort, with the counts before a
    tile added up and scanned; rows cut over up to all of the workers."""
    rng = np.random.default_rng(n)
    vocab = 5000
    ids, dout = ids_of(kind, n, vocab, rng), whole_rows(n, dim, "float32", n)
    want = check_whole(tt, ids, dout, vocab)
    base = torch.arange(vocab * dim, device="cuda").view(vocab, dim) % 1000
    out = base.float()
    tt.embed_grad(ids, dout, vocab, scale=0.5, out=out, accumulate=True)
    assert torch.equal(out, (base + want * 0.5).float())


@pytest.mark.parametrize("n", [200000, 600000, 1100000])
@pytest.mark.parametrize("count", [0, 1, 130000, 199999])
def test_embed_grad_of_fewer_tokens_than_the_bound(tt, n, count):
    rng = np.random.default_rng(n + count)
    ids, dout = ids_of("mixed", n, 3000, rng), whole_rows(n, 8, "bfloat16", n)
    got = tt.embed_grad(ids, dout, 3000, n_ids=torch.tensor([count], device="cuda"), status=(st := status_word()))
    assert torch.equal(got, whole_sums(ids[:count], dout[:count], 3000).float())
    assert st.item() == (tt.TT_ERR_INVALID_ARG if bool((ids[:count] >= 3000).any()) else 0)


@pytest.mark.parametrize("n,dim,name", [(200000, 2048, "bfloat16"), (110000, 2048, "float32"), (250000, 1024, "float16"),
                                        (150000, 1025, "bfloat16"), (90000, 1537, "float32"), (400000, 520, "bfloat16")])
@pytest.mark.parametrize("kind,vocab", [("runs", 300), ("runs", 2500), ("zipf", 4000), ("mixed", 700), ("one", 5)])
def test_embed_grad_of_long_parts(tt, n, dim, name, kind, vocab):
    """Widths where a worker's part of the list is long, with rows around the 63
    tokens up to which a row is not cut."""
    rng = np.random.default_rng(n + vocab)
    ids, dout = ids_of(kind, n, vocab, rng), whole_rows(n, dim, name, n)
    want = check_whole(tt, ids, dout, vocab)
    out = torch.ones(vocab, dim, device="cuda")
    tt.embed_grad(ids, dout, vocab, scale=0.5, out=out, accumulate=True)
    assert torch.equal(out, (1 + want * 0.5).float())


@pytest.mark.parametrize("n,vocab,dim", [(200000, 1 << 20, 8), (200000, 1 << 20, 9), (50000, 200256, 641), (250000, 1000003, 96)])
@pytest.mark.parametrize("kind", ["zipf", "runs", "mixed", "two"])
@pytest.mark.parametrize("to", ["float32", "bfloat16"])
def test_embed_grad_of_whole_numbers_into_mostly_absent_rows(tt, n, vocab, dim, kind, to):
    rng = np.random.default_rng(n + dim)
    check_whole(tt, ids_of(kind, n, vocab, rng), whole_rows(n, dim, "bfloat16", n), vocab, to)


@pytest.mark.parametrize("ti", DTYPES)
@pytest.mark.parametrize("to", DTYPES)
@pytest.mark.parametrize("dim,stride,shift", [(264, 264, 0), (264, 267, 0), (257, 300, 3)])
def test_embed_grad_of_whole_numbers_by_type(tt, ti, to, dim, stride, shift):
    rng = np.random.default_rng(dim)
    check_whole(tt, ids_of("mixed", 20000, 1000, rng), whole_rows(20000, dim, ti, dim, stride, shift), 1000, to)


# ------------------------------------------------------------ losses far from zero

def far_rows(n, vocab, name, offset, shift):
    """Rows around `offset`, as their type holds them, the third with a few of
    the lowest values, the fourth with -inf."""
    x = rows_of(n, vocab, name, gen(vocab), vocab + 3, shift, scale=3.0)
    x += offset
    x[2, : vocab // 2] = torch.finfo(dtype(name)).min
    x[3, vocab // 2:] = -math.inf
    return x


def check_far_loss(tt, x, targets, g, name):
    """Losses and gradients from the maximum M and the sum S of exp(l - M).
    A term's exponent has three roundings (the difference, the product, log2 e)
    and exp an error of 4 units; the running sums and their joins have some 60
    and the additions that follow one another: S is that far off.  M - l_t, log S
    (2 units) and their sum are rounded; a probability has S's error, its
    exponent's, and a few roundings more, p - 1 another one."""
    loss, lse, d = (host(o) for o in tt.token_loss(x, torch.from_numpy(targets).cuda(), torch.from_numpy(g).cuda(), want_grad=True))
    xs = host(x)
    m = xs.max(1, keepdims=True)
    e = np.exp(xs - m)
    s = e.sum(1, keepdims=True)
    p, rows = e / s, np.arange(len(xs))
    far = np.where(p > 0, np.minimum(np.abs(xs - m), 1e4), 0)
    of_sum = plain.EPS * (64 + xs.shape[1] / 128 + 3 * (p * far).sum(1))
    log_s, m = np.log(s)[:, 0], m[:, 0]
    want = m - xs[rows, targets] + log_s
    with np.errstate(over="ignore"):
        want[np.isinf(want.astype(np.float32))] = math.inf    # what rounds to no float
    fine = np.isfinite(want)
    assert np.array_equal(loss[~fine], want[~fine])
    assert np.all(np.abs(loss[fine] - want[fine]) <= of_sum[fine] + 5 * plain.EPS * np.abs(want[fine]))
    assert np.all(np.abs(lse - (m + log_s)) <= of_sum + plain.EPS * (4 * log_s + 2 * np.abs(m)))
    want_d = p.copy()
    want_d[rows, targets] -= 1
    want_d *= g[:, None].astype(np.float64)
    tol = np.abs(g)[:, None] * (p * (of_sum[:, None] + plain.EPS * (3 * far + 16)) + 3 * plain.EPS * (p > 0)) + \
        1.01 * plain.UNIT[name] * np.abs(want_d) + plain.TINY[name]
    assert np.all(np.abs(d - want_d) <= tol)


@pytest.mark.parametrize("name,offset", [("float32", 300.0), ("float32", -1e4), ("float32", 3e6), ("float32", 1e30), ("float16", 1000.0),
                                         ("float16", -60000.0), ("bfloat16", 500.0), ("bfloat16", -1e5), ("bfloat16", 1e38)])
@pytest.mark.parametrize("vocab,shift", [(7, 0), (1000, 0), (4099, 3), (30001, 1), (120001, 0), (300000, 3)])
def test_token_loss_far_from_zero(tt, name, offset, vocab, shift):
    rng = np.random.default_rng(vocab)
    x = far_rows(6, vocab, name, offset, shift)
    targets = rng.integers(0, vocab, 6).astype(np.int32)
    targets[:2] = 0, vocab - 1
    g = rng.standard_normal(6).astype(np.float32)
    check_far_loss(tt, x, targets, g, name)
    # in place, and the loss alone
    out = tt.token_loss(x, torch.from_numpy(targets).cuda(), torch.from_numpy(g).cuda(), want_grad=True)
    alone = tt.token_loss(x, torch.from_numpy(targets).cuda())
    assert torch.equal(alone[0], out[0]) and torch.equal(alone[1], out[1])
    tt.token_loss(x, torch.from_numpy(targets).cuda(), torch.from_numpy(g).cuda(), dlogits=x)
    assert torch.equal(x, out[2])


@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("vocab", [3, 1000, 33333, 200255])
def test_token_loss_of_rows_of_one_value(tt, name, vocab):
    """Whatever the value, the lowest as a mask that leaves nothing among them:
    the loss is log V and the probabilities are equal."""
    info = torch.finfo(dtype(name))
    values = [0.0, 5.0, info.min, info.max, -300.0, 2.0**14]
    x = torch.tensor(values, device="cuda").to(dtype(name))[:, None].repeat(1, vocab)
    targets = np.array([0, 1, 2, vocab - 1, vocab // 2, 1], dtype=np.int32)
    check_far_loss(tt, x, targets, np.ones(6, np.float32), name)


# ------------------------------------------------------------ zeros of either sign

@pytest.mark.parametrize("vocab", [9, 5000, 100256])
@pytest.mark.parametrize("n", [6, 200])
@pytest.mark.parametrize("key", ["temperature", "top_p", "min_p", "uniform"])
def test_sample_takes_a_negative_zero_as_zero(tt, vocab, n, key):
    x = rows_of(n, vocab, "float32", gen(vocab), scale=2.0)
    x[n // 2:] *= 0.01                                        # flat rows, for the histograms
    rng = np.random.default_rng(n)
    a = dict(temperature=torch.ones(n, device="cuda"), top_p=torch.full((n,), 0.9, device="cuda"),
             min_p=torch.zeros(n, device="cuda"), uniform=torch.rand(n, generator=gen(n), device="cuda"),
             top_k=torch.from_numpy(rng.choice([0, 5, 3000], n).astype(np.int32)).cuda())
    a[key] = torch.zeros(n, device="cuda")
    want = tt.sample(x, **a)
    a[key] = torch.full((n,), -0.0, device="cuda")
    st = status_word()
    got = tt.sample(x, status=st, **a)
    assert st.item() == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if key == "temperature":
        assert torch.equal(got[0], x.argmax(1).int())
    check_sample(tt, x, np.zeros(n, np.float32), {"top_p": np.zeros(n, np.float32)}, range(0, n, 20))
