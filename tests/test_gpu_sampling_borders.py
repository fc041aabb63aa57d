"""Rows whose cut falls where the sampling kernels change their way of finding it.

Kept sets are checked in every row: a cut may lie on either side of a token only where that token's
cumulative share is within 2^-26 of top_p (the kernel's border sums are good to about 2^-28), and
nowhere among equal weights, whose whole-number sums are exact.  Probabilities: as in
test_gpu_sampling.py, p (3 a 2^-24 + 2^-21 + n 2^-24), n = 100 roundings in sequence in the sum, or V
/ 1024 (a thread of a whole row adds every 512th vector to one of two sums) and 16 to join them.
Weights below the smallest normal number may flush to zero.
"""
import math
from fractions import Fraction

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from tests.target_reference import make_session  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
INF = math.inf
TOL = 2.0 ** -21 + 100 * 2.0 ** -24


@pytest.fixture(scope="module")
def sess():
    s = make_session()
    yield s
    s.close()


def order64(x):
    """Finite logits in the kernel's order: values in float64, ids.  -0 and +0 are equal."""
    big = torch.finfo(x.dtype).max
    x = x.double() + 0.0
    x = torch.where(x.isnan(), -INF, x).clamp(max=big)
    v, at = x.sort(descending=True, stable=True)
    n = int((v > -INF).sum())
    return v[:n], at[:n]


def cut_range(w, k, p):
    """Fewest and most tokens that top-k and top-p may keep of weights in descending order."""
    n = min(k, w.numel()) if k > 0 else w.numel()
    if p >= 1:
        return n, n
    w = w[:n]
    if bool((w == w[0]).all()):
        exact = max(1, math.ceil(Fraction(p) * n)) if p > 0 else 1
        return exact, exact
    share = (w.cumsum(0) - w) / w.sum()
    return (max(1, int((share < p - 2.0 ** -26).sum())), max(1, int((share < p + 2.0 ** -26).sum())))


def check_row(x, T, k, p, probs, noise, token, prob):
    T, p = (float(torch.tensor(t, dtype=F32)) for t in (T, p))
    v, at = order64(x)
    if v.numel() == 0:
        assert bool((probs == 0).all()) and token == -1 and prob == 0
        return
    if T < 2.0 ** -126:
        a, k, p = torch.zeros_like(v), 1, 1.0
    else:
        a = (v[0] - v) / T
    w = torch.exp(-a)
    lo, hi = cut_range(w, k, p)
    got = probs.double()
    n = int((got > 0).sum())
    part = w / w[:hi].sum()
    assert min(lo, int((part >= 2.0 ** -125).sum())) <= n <= min(hi, int((part >= 2.0 ** -150).sum())), \
        (T, k, p, lo, hi, n)
    kept = torch.zeros(x.numel(), dtype=torch.bool, device=x.device)
    kept[at[:n]] = True
    assert torch.equal(kept, got > 0), (T, k, p)
    want = w[:n] / w[:n].sum()
    tol = want * (3 * a[:n] * 2.0 ** -24 + 2.0 ** -21 + max(100, x.numel() / 1024 + 16) * 2.0 ** -24) + 2.0 ** -126
    assert bool(((got[at[:n]] - want).abs() <= tol).all()), (T, k, p)
    score = w[:n] / noise[at[:n]].double()
    best = int((at[:n] == token).nonzero())
    assert float(score[best]) >= float(score.max()) * (1 - 2.0 ** -14)
    assert abs(prob - float(want[best])) <= float(tol[best])


def check(sess, x, entries, seed=0, many=False, word=0, lead=0, trail=0):
    """Rows of x with (T, top-k, top-p) each; many: the rows repeated until they are a large batch,
    which takes a CTA a row.  lead, trail: elements between the rows.  word: the error word."""
    R, V = x.shape
    times = -(-320 // R) if many else 1
    g = torch.Generator(device="cuda").manual_seed(seed)
    noise = torch.empty((R, V), device="cuda").exponential_(generator=g).clamp_(min=1e-30)
    xs = torch.zeros((R * times, lead + V + trail), dtype=x.dtype, device="cuda")[:, lead:lead + V]
    xs.copy_(x.repeat(times, 1))
    ns = noise.repeat(times, 1)
    T, k, p = zip(*(entries * times))
    ps = dict(temperature=torch.tensor(T, device="cuda"), top_p=torch.tensor(p, device="cuda"),
              top_k=torch.tensor(k, dtype=torch.int32, device="cuda"))
    probs = torch.full(xs.shape, -1.0, device="cuda")
    ids = torch.full((R * times,), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((R * times,), -1.0, device="cuda")
    sess.target_probs(xs, probs, **ps)
    assert sess.error() == word
    sess.sample_tokens(xs, ns, ids, prob=prob, **ps)
    assert sess.error() == word
    # The same row gives the same bits where it lies the same way.  Rows that start at another element
    # of a 16-byte vector are added up in another order: each is within n 2^-24 of the exact sum, n as
    # above, and the weights are the same.
    same = xs.stride(0) * xs.element_size() % 16 == 0
    apart = 0.0 if same else 2.0 * max(100, V / 1024 + 16) * 2.0 ** -24
    for t in (probs, ids, prob):
        first = t[:R].repeat(times, *[1] * (t.dim() - 1))
        assert torch.equal(t > 0, first > 0)
        assert bool(((t.double() - first.double()).abs() <= apart * first.double().abs()).all())
    assert torch.equal(ids, ids[:R].repeat(times))
    for r in range(R):
        check_row(x[r], *entries[r], probs[r], noise[r], int(ids[r]), float(prob[r]))


def levels(V, dtype, seed, *groups):
    """A row of (count, value) groups at random places, -infinity elsewhere."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    at = torch.randperm(V, generator=g, device="cuda").split([n for n, _ in groups] +
                                                             [V - sum(n for n, _ in groups)])
    x = torch.full((V,), -INF, device="cuda")
    for i, (_, value) in zip(at, groups):
        x[i] = value
    return x.to(dtype)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_cuts_at_the_first_tokens_of_the_tail(sess, dtype, many):
    """32 (m - x) log2(e) / T between 1022.40 and 1022.49: the last bin of the histogram holds these
    tokens though their number rounds to the bin before."""
    low = -22.125                                # in both types
    T = 22.125 * math.log2(math.e) / 31.9514     # a = 31.9514
    rows, entries = [], []
    for groups, ks in [([(500, 0.0), (500, low)], (600, 999)),                       # all of the tail
                       ([(500, 0.0), (300, low), (300, -25.0)], (700, 800, 900)),
                       ([(100, 0.0), (2000, low)], (400, 700)),
                       ([(600, 0.0), (1, low), (1500, -30.0)], (601, 602)),
                       ([(1, 0.0), (3000, low)], (2, 513, 3000))]:
        for k in ks:
            rows.append(levels(4099, dtype, k, *groups))
            entries.append((T, k, 1.0))
    check(sess, torch.stack(rows), entries, many=many)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_zeros_of_either_sign_are_equal(sess, dtype, many):
    """-0 and +0 are one logit: the lower id comes first, greedy, in the list and in the histogram."""
    V = 4099
    x = torch.full((10, V), -3.0, device="cuda")
    x[0, 7], x[0, 8] = -0.0, 0.0
    x[1, 0], x[1, V - 1] = -0.0, 0.0
    x[2, :40:2], x[2, 1:40:2] = -0.0, 0.0            # a short list, cut among them
    x[3] = x[2]
    x[4, :2000:2], x[4, 1:2000:2] = -0.0, 0.0        # more than a list holds
    x[5] = x[4]
    x[6], x[7], x[8], x[9] = x[4], x[4], 0.0, -0.0
    x[6, 5], x[7, 5] = 1e-38, -1e-38                 # the smallest neighbours keep their order
    x[8, ::3] = -0.0
    entries = [(0.0, 0, 1.0), (1.0, 1, 1.0), (1.0, 9, 1.0), (1.0, 30, 0.5), (1.0, 600, 1.0), (1.0, 0, 0.3),
               (1.0, 601, 1.0), (1.0, 1500, 0.4), (1.0, 700, 0.9), (1.0, 1000, 1.0)]
    check(sess, x.to(dtype), entries, many=many)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_top_p_below_zero_keeps_the_first_token(sess, dtype, many):
    V = 4099
    flat = torch.ones((2, V), device="cuda")
    flat[1] = torch.linspace(0, 1e-3, V, device="cuda")
    x = torch.cat([flat, flat, flat]).to(dtype)
    check(sess, x, [(1.0, 0, 0.0)] * 2 + [(1.0, 0, -1.0)] * 2 + [(1.0, 0, -3e38), (2.0, 700, -1e10)], many=many)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_largest_temperature_and_the_largest_differences(sess, dtype):
    """At T = 2^100 logits that differ by more than the largest float weigh nothing beside the
    maximum, and keep their place in the order; a temperature above is refused."""
    V, top = 4099, 2.0 ** 100
    x = torch.stack([levels(V, dtype, i, (2000, 3e38), (2000, -3e38)) for i in range(4)])
    check(sess, x[:3], [(top, 0, 0.5), (top, 1500, 1.0), (top, 1200, 0.25)])
    k = torch.tensor([3000, 0, 2000, 1], dtype=torch.int32, device="cuda")
    T = torch.tensor([top, 2 * top, 3e38, top], device="cuda")
    probs = torch.full((4, V), -1.0, device="cuda")
    ids = torch.full((4,), -5, dtype=torch.int32, device="cuda")
    sess.target_probs(x, probs, temperature=T, top_k=k)
    assert sess.error() == 0x80
    sess.sample_tokens(x, torch.ones((4, V), device="cuda"), ids, temperature=T, top_k=k)
    assert sess.error() == 0x80
    assert bool((probs[1:3] == -1).all()) and ids.tolist()[1:3] == [-5, -5]
    high = x > 0
    assert torch.equal(probs[0] > 0, high[0]) and bool(((probs[0][high[0]] * 2000 - 1).abs() < TOL).all())
    first = int(high[3].nonzero()[0])
    assert int(ids[0]) == int(high[0].nonzero()[0]) and int(ids[3]) == first and float(probs[3, first]) == 1


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_variates_that_are_none(sess, dtype, many):
    """Negative and NaN variates draw nothing; a row with no other among its kept tokens has no id."""
    V, spot = 4099, 77
    x = torch.linspace(3, 0, V, device="cuda").to(dtype).expand(9, V).contiguous()
    noise = torch.full((9, V), math.nan, device="cuda")
    noise[3:6] = -1.0
    noise[6:, spot] = 2.0
    times = 40 if many else 1
    n = 9 * times
    ps = dict(temperature=torch.tensor([1.0, 1.0, 1e-3] * 3 * times, device="cuda"),
              top_k=torch.tensor([0, 100, 1000] * 3 * times, dtype=torch.int32, device="cuda"))
    ids = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((n,), -9.0, device="cuda")
    sess.sample_tokens(x.repeat(times, 1), noise.repeat(times, 1), ids, prob=prob, **ps)
    assert sess.error() == 0x80
    assert ids.tolist() == ([-1] * 6 + [spot] * 3) * times
    prob = prob.view(times, 9)
    assert bool((prob[:, :6] == 0).all()) and bool((prob[:, 6:8] > 0).all())
    noise[:6, 5] = 1.0
    sess.sample_tokens(x.repeat(times, 1), noise.repeat(times, 1), ids, prob=prob.view(-1), **ps)
    assert sess.error() == 0
    assert ids.tolist() == ([5] * 6 + [spot] * 3) * times


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1500, 20001, 151936])
def test_borders_among_alike_and_equal_logits(sess, dtype, V, many):
    if many and V > 100000:
        V = 70003                                # (a large batch of distributions that fits a quick test)
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.zeros((6, V), device="cuda")
    x[1] = 1e-3 * torch.randn(V, generator=g, device="cuda")
    x[2] = torch.randint(0, 3, (V,), generator=g, device="cuda")
    x[3, ::2] = 0.25
    x[4] = -30.0
    x[4, V // 2] = 0
    x[5] = 100 + torch.randn(V, generator=g, device="cuda")
    x = x.to(dtype)
    for entry in [(1.0, 0, 0.7), (1.0, V // 3, 1.0), (1.0, V - 1, 0.31), (0.5, 1200, 0.5), (4.0, 0, 0.9999),
                  (1.0, 7, 1.0), (1.0, 0, 1 - 2.0 ** -24), (1e30, 0, 0.25), (1e-30, 2, 0.6), (2.0, 513, 0.999)]:
        check(sess, x, [entry] * 6, many=many)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lead,trail", [(0, 0), (1, 0), (3, 2), (8, 5)])
def test_large_batches_of_rows_to_be_cleaned(sess, dtype, lead, trail):
    """NaN, infinities and the type's lowest value in rows that a CTA reads again in every pass, at
    any element offset."""
    V, low = 3001, torch.finfo(dtype).min
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (2.5 * torch.randn((12, V), generator=g, device="cuda")).to(dtype)
    x[0] = -INF                                  # nothing left
    x[1] = math.nan                              # nothing left
    x[2] = -INF
    x[2, 77] = -3.0                              # one token left
    x[3, 5:] = low                               # masked by the type's lowest value
    x[4] = low                                   # all of it
    x[5, ::3] = math.nan
    x[6, [3, 900]] = INF                         # two infinities share the row
    x[7, ::2] = -INF
    x[8] = torch.finfo(dtype).max
    x[9, :] = -INF
    x[9, -1] = low
    x[10, 0] = x[10, -1] = math.nan              # at the ends
    for entry in [(1.0, 0, 1.0), (0.8, 40, 0.9), (1.0, 0, 0.5), (1.0, 2900, 1.0), (0.0, 0, 1.0), (1.5, 600, 0.97)]:
        check(sess, x, [entry] * 12, many=True, word=0x100, lead=lead, trail=trail)


def test_large_batches_of_odd_vocabularies(sess):
    for dtype in (BF, F32):
        for V in (1, 3, 17, 1023, 8191, 50257):
            g = torch.Generator(device="cuda").manual_seed(V)
            x = (3 * torch.randn((8, V), generator=g, device="cuda")).to(dtype)
            check(sess, x, [(1.0, 0, 1.0), (0.7, 20, 0.95), (1.3, 0, 0.9), (0.0, 0, 1.0), (1.0, 1, 0.5),
                            (2.0, 0, 0.999), (1.0, 1000, 0.8), (3.0, 3, 0.34)], many=True, trail=V % 2)
