"""Row ranges that claim more rows than there are: flagged, and no output is written, in either type."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from tests.target_reference import Paged, i32, make_session  # noqa: E402

FILL = -7.0


@pytest.fixture(scope="module")
def sess():
    s = make_session()
    yield s
    s.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,heads,prefix", [(128, 64, 0), (64, 2, 0), (128, 2, 128)])
@pytest.mark.parametrize("starts,skipped", [
    ([0, 6] * 20 + [0], None),       # all rows again and again, decreasing pairs between
    ([0, 5, 4, 6, 6, 6], None),      # 0..4, then 4..5: one row twice, every other has one owner
    ([0, 4, 2, 6], 0),               # a request without a place in its pages claims its rows all the same
])
def test_nothing_is_written(sess, dtype, dim, heads, prefix, starts, skipped):
    B = len(starts) - 1
    pb = Paged([6] + [0] * (B - 1), [10] * B, prefix=prefix, kvh=1, dim=dim, dtype=dtype, seed=4)
    q, lay = pb.normal(pb.rows, heads, dim), pb.layer(heads)
    pb.row_start = i32(starts)
    word = 0x40
    if skipped is not None:
        pb.kv_len[skipped] = -1
        word = 0x41
    out = torch.full((pb.rows, heads, dim), FILL, dtype=dtype, device="cuda")
    sess.paged_attention(lay, q, pb.row_start, pb.kv_len, out, sess.attention_workspace(lay, B, pb.rows))
    # (the fp32 kernel need not reach the lengths)
    assert sess.error() in (0x40, word)
    assert bool((out == FILL).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ranges_that_claim_every_row_once(sess, dtype):
    """As many rows as there are, a range that is none among them: the others are served."""
    pb = Paged([2, 4], [10, 70], kvh=1, dim=128, dtype=dtype, seed=4)
    q, lay = pb.normal(pb.rows, 2, 128), pb.layer(2)
    out = torch.full((pb.rows, 2, 128), FILL, dtype=dtype, device="cuda")
    ws = sess.attention_workspace(lay, 2, pb.rows)
    sess.paged_attention(lay, q, pb.row_start, pb.kv_len, out, ws)
    assert sess.error() == 0 and bool((out != FILL).all())
    again = torch.full_like(out, FILL)
    sess.paged_attention(lay, q, i32([0, 2, 7]), pb.kv_len, again, ws)     # past the end
    assert sess.error() == 0x40
    assert torch.equal(again[:2], out[:2]) and bool((again[2:] == FILL).all())
