"""Tree attention without a mask against the paged attention: the same arithmetic, bit for bit."""
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


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("lens,ctx,heads,kvh,prefix", [
    ([30, 200], [77, 300], 8, 2, 64), ([1, 16, 0, 5], [0, 63, 9, 130], 5, 1, 0), ([1], [3000], 8, 8, 0),
    ([64] * 40, [64 + 9 * i for i in range(40)], 8, 2, 512), ([700, 3], [0, 1000], 16, 1, 0)])
@pytest.mark.parametrize("scale", [None, -0.2])
def test_without_a_mask_the_bits_are_the_paged_attentions(sess, dtype, dim, lens, ctx, heads, kvh, prefix, scale):
    """One row a thread, and every sum in the same order, in both calls."""
    pb = Paged(lens, ctx, prefix=prefix, kvh=kvh, dim=dim, dtype=dtype, seed=len(lens))
    q, lay = pb.normal(pb.rows, heads, dim), pb.layer(heads)
    ws = sess.attention_workspace(lay, len(lens), pb.rows)
    a, b = (torch.full(q.shape, -7.0, dtype=dtype, device="cuda") for _ in "ab")
    sess.tree_attention(lay, q, pb.row_start, pb.kv_len, a, ws, scale=scale)
    sess.paged_attention(lay, q, pb.row_start, pb.kv_len, b, ws, scale=scale)
    assert sess.error() == 0
    assert bool(a.isfinite().all()) and torch.equal(a, b)
