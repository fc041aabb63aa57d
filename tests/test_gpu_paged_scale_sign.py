"""A negative scale is the positive one with negated queries, bit for bit, in both attention calls."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from tests.target_reference import Paged, i32, make_session  # noqa: E402


@pytest.fixture(scope="module")
def sess():
    s = make_session()
    yield s
    s.close()


@pytest.mark.parametrize("dtype,dim", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 128), (torch.float32, 64)])
@pytest.mark.parametrize("lens,ctx,heads,kvh,prefix", [([30, 200], [77, 300], 8, 2, 64), ([1, 16, 0, 5], [0, 63, 9, 130], 5, 1, 0),
                                                       ([1], [3000], 8, 8, 0), ([700, 3], [0, 1000], 16, 1, 0)])
def test_sign_of_the_scale(sess, dtype, dim, lens, ctx, heads, kvh, prefix):
    pb = Paged(lens, ctx, prefix=prefix, kvh=kvh, dim=dim, dtype=dtype, seed=len(lens))
    pb.v[:, ::5, :, 3] = float("inf")          # some rows are done again
    q, lay, T = pb.normal(pb.rows, heads, dim), pb.layer(heads), pb.rows
    ws = sess.attention_workspace(lay, len(lens), T)
    words = (max(lens) + 31) // 32
    par = i32([p for n in lens if n for p in [-1] + [i // 2 for i in range(n - 1)]])
    mask = torch.zeros((T, words), dtype=torch.int32, device="cuda")
    sess.tree_plan(pb.row_start, par, mask, root=pb.kv_len)
    got = []
    for x, scale in ((q, 0.2), (-q, -0.2)):
        a, b, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros((T, heads), device="cuda")
        sess.paged_attention(lay, x, pb.row_start, pb.kv_len, a, ws, scale=scale)
        sess.tree_attention(lay, x, pb.row_start, pb.kv_len, b, ws, mask=mask, scale=scale, lse=lse)
        got.append([a, b, lse])
    assert sess.error() == 0
    for x, y in zip(*got):
        assert torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0))
