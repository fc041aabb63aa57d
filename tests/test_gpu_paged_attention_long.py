"""Values that are not finite behind a row's last key, in batches of long contexts: rows that do not
see them are as without them (tolerance as in test_gpu_paged_attention.py), and the call ends without
a wait that runs out."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_diffusion_speculative_fc_gb300 as pkg  # noqa: E402
from tests.target_reference import PAGE, i32, make_session  # noqa: E402

BF = torch.bfloat16
FILL = -7.0


@pytest.fixture(scope="module")
def sess():
    s = make_session()
    yield s
    s.close()


@pytest.mark.parametrize("dim,prefix", [(128, 0), (128, 192), (64, 0)])
def test_hidden_values_behind_long_contexts(sess, dim, prefix):
    """160 requests x 4 rows over 200000 keys (one set of pages, a last page of each request's own):
    more requests than SMs, so that each is one item that no other CTA shares."""
    B, n, ctx, heads = 160, 4, 200000, 8
    whole = ctx // PAGE
    g = torch.Generator(device="cuda").manual_seed(1)
    shape = (whole + B + prefix // PAGE, PAGE, 1, dim)
    k, v = (torch.randn(shape, generator=g, device="cuda").to(BF) for _ in "kv")
    q = torch.randn((B * n, heads, dim), generator=g, device="cuda").to(BF)
    table = torch.cat([torch.arange(whole).expand(B, whole), whole + torch.arange(B)[:, None]], 1)
    pre = torch.arange(whole + B, whole + B + prefix // PAGE)
    lay = pkg.LayerKV(heads, k, v, i32(table).contiguous(), i32(pre) if prefix else None)
    out = torch.full((B * n, heads, dim), FILL, dtype=BF, device="cuda")
    spoiled = (0, 3, 159)
    for b in spoiled:                              # the value of each one's third row
        v[whole + b, ctx % PAGE + 2, 0, 5] = float("nan")
    row_start, kv_len = i32([n * b for b in range(B + 1)]), i32([prefix + ctx] * B)
    ws = sess.attention_workspace(lay, B, B * n)
    for _ in range(2):
        out.fill_(FILL)
        sess.paged_attention(lay, q, row_start, kv_len, out, ws)
        assert sess.error() == 0
    half = torch.finfo(BF).eps / 2
    for b in spoiled + (1,):
        pages = torch.cat([pre, table[b]]).cuda()
        kb, vb = (t[pages].flatten(0, 1)[:prefix + ctx + n, 0].double() for t in (k, v))
        for i in range(n):
            m = prefix + ctx + i + 1
            x = q[n * b + i].double()
            s = x @ kb[:m].T * dim ** -0.5
            mag = (x.abs() @ kb[:m].abs().T).amax(1) * dim ** -0.5
            p = torch.softmax(s, -1)
            want, spread = p @ vb[:m], p @ vb[:m].abs()
            tol = half * want.abs() + (half + 2 * ((dim + 8) * 2.0 ** -24 * mag)[:, None] + 2.0 ** -18) * spread * (1 + half)
            got = out[n * b + i].double()
            seen = torch.zeros(dim, dtype=torch.bool, device="cuda")
            seen[5] = b in spoiled and i >= 2
            assert torch.equal(~torch.isfinite(got), seen.expand(heads, dim)), (b, i)
            over = ((got - want).abs() - tol)[:, ~seen]
            assert float(over.max()) <= 0, (b, i, float(over.max()))


@pytest.mark.parametrize("lens,ctx,heads,kvh,dim,prefix", [
    ([1], [20000], 32, 8, 128, 0), ([1], [20000], 128, 1, 128, 1024), ([2], [9000], 5, 1, 64, 0),
    ([1] * 64, [70 * i for i in range(64)], 64, 8, 128, 16384), ([16] * 30, [100 * i for i in range(30)], 32, 8, 128, 0),
    ([700, 257, 64], [0, 1000, 31], 21, 3, 64, 640), ([33, 1, 0, 47], [5000, 6000, 0, 130], 2, 2, 64, 128)])
def test_nothing_is_written_behind_the_workspace(sess, lens, ctx, heads, kvh, dim, prefix):
    from tests.target_reference import Paged
    pb = Paged(lens, ctx, prefix=prefix, kvh=kvh, dim=dim, seed=3)
    lay, q = pb.layer(heads), pb.normal(pb.rows, heads, dim)
    n = sess.attention_workspace(lay, len(lens), pb.rows).numel()
    ws = torch.full((n + (1 << 20),), 0x5a, dtype=torch.uint8, device="cuda")
    out = torch.full((pb.rows, heads, dim), FILL, dtype=BF, device="cuda")
    sess.paged_attention(lay, q, pb.row_start, pb.kv_len, out, ws[:n])
    assert sess.error() == 0
    assert bool((ws[n:] == 0x5a).all())
    assert bool(torch.isfinite(out).all())
