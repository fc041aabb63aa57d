"""Ranges of rows that overlap, in the calls for trees and key weights."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_diffusion_speculative_fc_gb300 as pkg  # noqa: E402
from tests.target_reference import Paged, i32, make_session  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sess():
    s = make_session()
    yield s
    s.close()


def test_rows_that_two_requests_claim_are_flagged(sess):
    """Ranges that share rows have a pair between them that falls: its request sets ROW_RANGE."""
    starts, T = [0, 5, 3, 8], 12
    rs = i32(starts)
    par = i32([-1, 0, 0, -1, 0, 0, 0, 0] + [0] * 4)
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    mask, pos = i(T, 1), i(T)
    sess.tree_plan(rs, par, mask, pos, root=i32([0, 0, 0]))
    assert "ROW_RANGE" in pkg.decode_error(sess.error())
    assert bool((mask[8:] == 0).all())
    sess.accept_tree(rs, par, i(T) + 1, i(T) + 2, i(3), i(3), i(3), i(3), i(3, 2), i(3, 2))
    assert "ROW_RANGE" in pkg.decode_error(sess.error())
    for dt in (BF, F32):
        pb = Paged([5, 0, 5], [20, 0, 70], kvh=1, dim=64, dtype=dt, seed=2)
        q, out, lse = pb.normal(T, 2, 64), torch.zeros((T, 2, 64), dtype=dt, device="cuda"), torch.zeros((T, 2), device="cuda")
        lay = pb.layer(2)
        sess.tree_attention(lay, q, rs, pb.kv_len, out, sess.attention_workspace(lay, 3, T), lse=lse)
        assert "ROW_RANGE" in pkg.decode_error(sess.error())
        assert bool((out[8:] == 0).all()) and bool((lse[8:] == 0).all())
        w = torch.zeros((3, 1, 128), device="cuda")
        sess.key_weights(lay, q, rs, pb.kv_len, lse, w)
        assert "ROW_RANGE" in pkg.decode_error(sess.error())
        assert bool((w[1] == 0).all())
