"""Key weights beyond their plain form: the error of a single term that the header states, factors that count for
nothing, requests without rows.

A weight's term is row_weight exp(scale q.K - lse).  Its exponent, taken by parts, is off by (units of 2^-24):
lse times log2 e 1.3 (the constant and the product), log2 of row_weight 2, their difference 1, the division by scale
log2 e 2, the product's addition 2 (with the score), the product with scale log2 e 1; so at most 8 2^-24 = 2^-21 of
|lse| and of |ln row_weight|.  The exponential is good to 2^-22, the last sum adds 2^-24: 2^-21 for both.
Here every score is 0, so that the score's own error has no part in it.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from tests.target_reference import Paged, make_session  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
KINDS = [(BF, 128), (BF, 64), (F32, 128), (F32, 64)]


@pytest.fixture(scope="module")
def sess():
    s = make_session()
    yield s
    s.close()


def f32(*shape, g, lo, hi):
    return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -100, 0.088, 0.3, -0.7, 20.0])
@pytest.mark.parametrize("weighted", [False, True])
def test_error_of_a_single_term(sess, dtype, dim, scale, weighted):
    B = 1000
    pb = Paged([1] * B, [2] * B, kvh=1, dim=dim, dtype=dtype, seed=dim)
    pb.k.zero_()
    q = pb.normal(B, 1, dim)
    lse = f32(B, 1, g=pb.g, lo=-60, hi=60)
    rw = f32(B, g=pb.g, lo=-20, hi=20).exp() if weighted else None
    got = torch.full((B, 1, 3), -7.0, device="cuda")
    sess.key_weights(pb.layer(1), q, pb.row_start, pb.kv_len, lse, got, row_weight=rw, decay=0.0, scale=scale)
    assert sess.error() == 0
    ln = torch.zeros((B, 1), dtype=torch.float64, device="cuda") if rw is None else rw.double().log()[:, None]
    want = torch.exp(ln - lse.double())
    bound = 2.0 ** -21 * (1 + lse.double().abs() + ln.abs())
    for key in range(3):
        assert float(((got[:, :, key].double() / want - 1).abs() / bound).max()) <= 1


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("heads,kvh,rows", [(4, 1, 6), (16, 2, 40), (64, 1, 9)])
def test_factors_that_count_for_nothing(sess, dtype, dim, heads, kvh, rows):
    """Factors below zero, infinite ones and NaN are as zero: the same weights, bit for bit."""
    pb = Paged([rows, 3], [200, 64], kvh=kvh, dim=dim, dtype=dtype, seed=rows)
    q, lse = pb.normal(pb.rows, heads, dim), f32(pb.rows, heads, g=pb.g, lo=3, hi=6)
    rw = f32(pb.rows, g=pb.g, lo=0.1, hi=2)
    inf, none = float("inf"), [0, 2, 3, 5, rows + 1]
    got = []
    for what in ([0.0] * 5, [-0.0, -1e-30, -3.0, inf, float("nan")], [-inf, -inf, inf, -0.5, -float("nan")]):
        rw[none] = torch.tensor(what, device="cuda")
        w = torch.ones((2, kvh, 64 * pb.width), device="cuda")
        sess.key_weights(pb.layer(heads), q, pb.row_start, pb.kv_len, lse, w, row_weight=rw, decay=0.5)
        got.append(w)
    assert sess.error() == 0
    assert bool(got[0].isfinite().all()) and torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_request_without_rows_keeps_its_weights(sess, dtype):
    pb = Paged([2, 0, 1], [30, 64, 7], kvh=1, dim=64, dtype=dtype, seed=3)
    q, lse = pb.normal(3, 2, 64), torch.zeros((3, 2), device="cuda")
    w = torch.rand((3, 1, 80), generator=pb.g, device="cuda")
    old = w.clone()
    sess.key_weights(pb.layer(2), q, pb.row_start, pb.kv_len, lse, w, decay=0.5)
    assert sess.error() == 0
    assert torch.equal(w[1], old[1]) and not bool((w[0, 0, :30] == old[0, 0, :30]).any())
