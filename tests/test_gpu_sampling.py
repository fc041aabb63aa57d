"""Sampling distribution and token draws against their plain 64-bit form.

A probability w / sum w in fp32: the exponent (x - max) / T carries three roundings (2^-24 each,
relative: times its size in the weight), the base-2 exponential 2^-22, the sum below 100 roundings
in sequence, the last product one: tol = p (3 a 2^-24 + 2^-21 + 100 * 2^-24).  Kept sets have to be
equal, except in a row where a token's cumulative share is within 2^-26 of top_p (the kernel's
border sums are good to about 2^-28).  Drawn ids have to be equal except where the two best race
scores are within 2^-14 of each other.
"""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_diffusion_speculative_fc_gb300 as pkg  # noqa: E402
from tests.target_reference import make_session, sample64  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module")
def sess():
    s = make_session()
    yield s
    s.close()


def f32(v):
    return torch.tensor(v, dtype=F32, device="cuda")


def params(rows):
    """Device arrays of [(T, k, p, min_p)]."""
    T, k, p, m = zip(*rows)
    return dict(temperature=f32(T), top_k=torch.tensor(k, dtype=torch.int32, device="cuda"),
                top_p=f32(p), min_p=f32(m))


def one(v):
    return float(f32(v))      # the fp32 value that the kernel reads


def verify(logits, rows, probs, noise=None, ids=None, prob=None, per=1):
    n = logits.shape[0]
    for r in range(n):
        T, k, p, mp = rows[r // per]
        w, a, near = sample64(logits[r], one(T), k, one(p), one(mp))
        total = float(w.sum())
        if total == 0:
            assert bool((probs[r] == 0).all())
            if ids is not None:
                assert int(ids[r]) == -1 and float(prob[r]) == 0
            continue
        if near < 2.0 ** -26:
            continue
        want, got = w / total, probs[r].double()
        tol = want * (3 * a * 2.0 ** -24 + 2.0 ** -21 + 100 * 2.0 ** -24) + 2.0 ** -126
        over = (got - want).abs() - tol
        assert float(over.max()) <= 0, (r, rows[r // per], float(over.max()), int(over.argmax()))
        # kept sets: tokens below the smallest normal number flush to zero
        small = want < 2.0 ** -125
        assert bool((((got > 0) == (want > 0)) | small).all()), (r, rows[r // per])
        if ids is not None:
            score = w / noise[r].double()
            top = score.topk(min(2, score.numel())).values
            i = int(ids[r])
            if top.numel() == 1 or float(top[1]) < float(top[0]) * (1 - 2.0 ** -14):
                assert i == int(score.argmax()), (r, rows[r // per])
            assert float(w[i]) > 0
            assert abs(float(prob[r]) - float(want[i])) <= float(tol[i])


def both(sess, logits, rows, per=1, seed=0):
    R, V = logits.shape
    probs = torch.full((R, V), NAN, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    noise = torch.empty((R, V), device="cuda").exponential_(generator=g).clamp_(min=1e-30)
    ids = torch.full((R,), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((R,), NAN, device="cuda")
    ps = params(rows)
    sess.target_probs(logits, probs, **ps)
    sess.sample_tokens(logits, noise, ids, prob=prob, **ps)
    verify(logits, rows, probs, noise, ids, prob, per)
    return probs, ids


MIX = [(1.0, 0, 1.0, 0.0), (0.7, 20, 0.95, 0.0), (1.3, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05),
       (0.0, 0, 1.0, 0.0), (0.6, 50, 1.0, 0.02), (1.0, 1, 0.5, 0.0), (2.0, 0, 0.999, 0.0),
       (0.05, 0, 0.5, 0.5), (1.0, 1000, 0.8, 0.001), (1.0, 0, 0.0, 0.0), (3.0, 3, 0.34, 1.0)]


def model_logits(R, V, dtype, seed, spread=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((R, V), generator=g, device="cuda") * spread
    top = torch.randint(0, V, (R, 8), generator=g, device="cuda")
    return x.scatter_add_(1, top, 12 * torch.rand((R, 8), generator=g, device="cuda")).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 500, 1023, 4097, 17001, 50257, 151936, 163840])
def test_every_filter(sess, dtype, V):
    both(sess, model_logits(len(MIX), V, dtype, V), MIX, seed=V)
    assert sess.error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_largest_vocabulary(sess, dtype):
    V = 524288 if dtype == BF else 262144
    both(sess, model_logits(3, V, dtype, 5), MIX[1:4])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1500, 40001, 151936])
def test_flat_rows_and_ties(sess, dtype, V):
    """Rows whose borders fall among very many alike or equal logits: the gathered bin overflows
    and is split by logit, then by id."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.zeros((6, V), device="cuda")
    x[1] = 1e-3 * torch.randn(V, generator=g, device="cuda")
    x[2] = torch.randint(0, 3, (V,), generator=g, device="cuda")
    x[3, ::2] = 0.25
    x[4] = -30.0
    x[4, V // 2] = 0
    x[5] = 100 + torch.randn(V, generator=g, device="cuda")
    x = x.to(dtype)
    for T, k, p, mp in [(1.0, 0, 0.7, 0.0), (1.0, V // 3, 1.0, 0.0), (1.0, V - 1, 0.31, 0.0),
                        (0.5, 1200, 0.5, 0.0), (4.0, 0, 0.9999, 0.0), (1.0, 7, 1.0, 0.0),
                        (1.0, 0, 1 - 2.0 ** -24, 0.0), (1e30, 0, 0.25, 0.0), (1e-30, 2, 0.6, 0.0)]:
        both(sess, x, [(T, k, p, mp)] * 6)
    assert sess.error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masks_infinities_and_nan(sess, dtype):
    V = 3001
    x = model_logits(10, V, dtype, 3)
    low = torch.finfo(dtype).min
    x[0] = -INF                                  # nothing left
    x[1] = NAN                                   # nothing left
    x[2] = -INF
    x[2, 77] = -3.0                              # one token left
    x[3, 5:] = low                               # masked by the type's lowest value
    x[4] = low                                   # all of it
    x[5, ::3] = NAN
    x[6, [3, 900]] = INF                         # two infinities share the row
    x[7, ::2] = -INF
    x[8] = torch.finfo(dtype).max
    x[9, :] = -INF
    x[9, -1] = low
    for row in [(1.0, 0, 1.0, 0.0), (0.8, 40, 0.9, 0.0), (1.0, 0, 0.5, 0.0), (1.0, 2900, 1.0, 0.0),
                (0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.3)]:
        both(sess, x, [row] * 10)
        assert sess.error() == 0x100


def test_rows_of_a_block_share_an_entry_and_rows_are_strided(sess):
    B, S, V = 5, 8, 2003
    store = model_logits(B * S, V + 13, BF, 9)
    for off in (0, 1, 3, 6):                     # rows start at any element
        x = store[:, off:off + V]
        probs = torch.empty((B * S, V), device="cuda")
        rows = MIX[1:1 + B]
        sess.target_probs(x, probs, **params(rows))
        verify(x, rows, probs, per=S)
    x = store[:, 1:1 + V].unflatten(0, (B, S))   # [B, S, V], as the verification takes it
    probs = torch.empty((B, S, V), device="cuda")
    sess.target_probs(x, probs, **params(rows))
    verify(x.flatten(0, 1), rows, probs.flatten(0, 1), per=S)


def test_no_parameters_is_a_softmax(sess):
    x = model_logits(4, 777, F32, 2)
    probs = torch.empty_like(x)
    sess.target_probs(x, probs)
    verify(x, [(1.0, 0, 1.0, 0.0)] * 4, probs)
    sess.target_probs(x, probs, top_k=torch.tensor([5, 9], dtype=torch.int32, device="cuda"))
    verify(x, [(1.0, 5, 1.0, 0.0), (1.0, 9, 1.0, 0.0)], probs, per=2)


def test_many_rows(sess):
    rows = [MIX[i % len(MIX)] for i in range(384)]
    both(sess, model_logits(384, 30011, BF, 4), rows)


def test_bad_parameters_skip_their_rows(sess):
    x = model_logits(7, 500, BF, 6)
    rows = [(1.0, 5, 0.9, 0.0), (-1.0, 5, 0.9, 0.0), (NAN, 5, 0.9, 0.0), (INF, 0, 1.0, 0.0),
            (1.0, 5, NAN, 0.0), (1.0, 0, 1.0, 1.5), (1.0, 0, 1.0, NAN)]
    probs = torch.full((7, 500), 3.0, device="cuda")
    ids = torch.full((7,), -5, dtype=torch.int32, device="cuda")
    sess.target_probs(x, probs, **params(rows))
    assert sess.error() == 0x80
    sess.sample_tokens(x, torch.ones((7, 500), device="cuda"), ids, **params(rows))
    assert sess.error() == 0x80
    verify(x[:1], rows[:1], probs[:1])
    assert bool((probs[1:] == 3.0).all()) and ids.tolist()[1:] == [-5] * 6 and int(ids[0]) >= 0


def test_same_results_every_run_and_on_any_stream(sess):
    x = model_logits(24, 151936, F32, 8)
    rows = [MIX[i % len(MIX)] for i in range(24)]
    first, ids = both(sess, x, rows, seed=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again, ids2 = both(sess, x, rows, seed=3)
    s.synchronize()
    assert torch.equal(first, again) and torch.equal(ids, ids2)


def test_graph_replay(sess):
    x = model_logits(6, 5003, BF, 1)
    ps = params(MIX[:6])
    probs, ids = torch.empty((6, 5003), device="cuda"), torch.empty(6, dtype=torch.int32, device="cuda")
    noise = torch.ones((6, 5003), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sess.target_probs(x, probs, **ps)
        sess.sample_tokens(x, noise, ids, **ps)
    for seed in (11, 12):
        x.copy_(model_logits(6, 5003, BF, seed))
        noise.exponential_().clamp_(min=1e-30)
        g.replay()
        w = params(MIX[:6])
        eager = torch.empty_like(probs)
        sess.target_probs(x, eager, **w)
        assert torch.equal(eager, probs)
        e_ids = torch.empty_like(ids)
        sess.sample_tokens(x, noise, e_ids, **w)
        assert torch.equal(e_ids, ids)
        verify(x, MIX[:6], probs)


def test_draws_follow_the_distribution(sess):
    """65536 draws of one row of 40 tokens: chi-square below its mean + 6 standard deviations."""
    N, V = 65536, 40
    x = model_logits(1, V, F32, 13, spread=1.0)
    x = (x / 4).expand(N, V).contiguous()
    noise = torch.empty((N, V), device="cuda").exponential_(
        generator=torch.Generator(device="cuda").manual_seed(5)).clamp_(min=1e-30)
    ids = torch.empty(N, dtype=torch.int32, device="cuda")
    ps = {k: v for k, v in params([(1.0, 20, 0.95, 0.0)]).items()}
    sess.sample_tokens(x, noise, ids, **ps)
    w, _, _ = sample64(x[0], 1.0, 20, one(0.95), 0.0)
    want = (w / w.sum() * N).cpu()
    got = torch.bincount(ids.cpu().long(), minlength=V).double()
    kept = want > 0
    assert bool((got[~kept] == 0).all())
    chi = float(((got - want)[kept] ** 2 / want[kept]).sum())
    dof = int(kept.sum()) - 1
    assert chi < dof + 6 * math.sqrt(2 * dof)


def test_python_checks(sess):
    x = model_logits(4, 100, BF, 1)
    probs, ids = torch.empty((4, 100), device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    for bad in [lambda: sess.target_probs(x.half(), probs), lambda: sess.target_probs(x.t(), probs),
                lambda: sess.target_probs(x, probs[:3]), lambda: sess.target_probs(x, probs.double()),
                lambda: sess.target_probs(x, probs, temperature=f32([1, 1, 1])),
                lambda: sess.target_probs(x, probs, top_k=f32([1])),
                lambda: sess.target_probs(x, probs, top_p=f32([1]), min_p=f32([0, 0])),
                lambda: sess.target_probs(x[:, ::2], probs[:, :50].contiguous()),
                lambda: sess.sample_tokens(x, probs, ids.long()),
                lambda: sess.sample_tokens(x, probs.cpu(), ids),
                lambda: sess.target_probs(x.unflatten(0, (2, 2)).transpose(0, 1), probs.view(2, 2, 100))]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(pkg.DFlashError):
        both32 = torch.empty((4, 100), device="cuda")
        sess.target_probs(both32, both32)
