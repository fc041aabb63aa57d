"""Paged attention with a shared prefix against its plain 64-bit form.

Tolerance, element by element: out rounded once to the storage type (finfo.eps / 2 of the value);
in bf16 every weight of the softmax is rounded once for the second product (eps / 2 of it, so eps /
2 of sum_p softmax |V| in all); a score's error, (D + 8) 2^-24 of the largest scale * sum_d |q_d k_d|
(products summed in fp32 in any order, the scale, the base-2 exponential's argument), moves numerator
and denominator by as much: 2 of it times sum_p softmax |V|; sums over the keys in fp32 and the
approximate exponential: 2^-18 of the same.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_diffusion_speculative_fc_gb300 as pkg  # noqa: E402
from tests.target_reference import PAGE, Paged, attend64, i32, make_session  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
FILL = -7.0


@pytest.fixture(scope="module")
def sess():
    s = make_session()
    yield s
    s.close()


def close(pb, q, heads, out, scale, causal):
    dt, D = pb.dtype, pb.dim
    half = torch.finfo(dt).eps / 2
    owned = torch.zeros(pb.rows, dtype=torch.bool, device="cuda")
    for t, (want, spread, mag) in attend64(pb, q, heads, scale, causal).items():
        owned[t] = True
        ds = ((D + 8) * 2.0 ** -24 * mag)[:, None]
        tol = half * want.abs() + (half * (dt == BF) + 2 * ds + 2.0 ** -18) * spread * (1 + half)
        over = (out[t].double() - want).abs() - tol
        assert float(over.max()) <= 0, (t, float(over.max()), float(want.abs().max()))
    assert bool((out[~owned] == FILL).all())


def run(sess, lens, ctx, heads, kvh, dim, dtype=BF, prefix=0, causal=True, scale=None, qscale=1.0,
        seed=0, strided=False, spoil=True, **kw):
    pb = Paged(lens, ctx, prefix=prefix, kvh=kvh, dim=dim, dtype=dtype, seed=seed, **kw)
    if spoil:
        # every cache row that belongs to no request holds NaN, those past a request's last too
        used = torch.zeros((pb.n_pages, PAGE), dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            pages, rows = pb.slots(b, 0, prefix + ctx[b] + n)
            used[pages, rows] = True
        pb.k[~used] = float("nan")
        pb.v[~used] = float("nan")
    if strided:
        q = pb.normal(pb.rows, heads * dim + 64, scale=qscale)[:, :heads * dim].unflatten(1, (heads, dim))
        out = torch.full((pb.rows, heads * dim + 8), FILL, dtype=dtype, device="cuda")
        out = out[:, :heads * dim].unflatten(1, (heads, dim))
    else:
        q = pb.normal(pb.rows, heads, dim, scale=qscale)
        out = torch.full((pb.rows, heads, dim), FILL, dtype=dtype, device="cuda")
    lay = pb.layer(heads)
    ws = sess.attention_workspace(lay, len(lens), pb.rows)
    ws.fill_(255)                              # nothing is expected of the workspace
    sess.paged_attention(lay, q, pb.row_start, pb.kv_len, out, ws, scale=scale, causal=causal)
    assert sess.error() == 0
    close(pb, q, heads, out, dim ** -0.5 if scale is None else scale, causal)
    return pb, q, lay, ws, out


KINDS = [(BF, 128), (BF, 64), (F32, 128), (F32, 64)]


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("heads,kvh", [(1, 1), (8, 2), (5, 1), (16, 2), (128, 1), (21, 3)])
def test_head_layouts(sess, dtype, dim, heads, kvh):
    run(sess, [1, 16, 0, 5], [0, 63, 9, 130], heads, kvh, dim, dtype, seed=heads)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("prefix", [0, 64, 192, 1024])
@pytest.mark.parametrize("causal", [True, False])
def test_shared_prefix(sess, dtype, dim, prefix, causal):
    run(sess, [16, 3, 1, 0, 40], [0, 64, 127, 5, 300], 8, 2, dim, dtype, prefix=prefix, causal=causal,
        seed=prefix, lead=1, trail=2, strided=True)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("lens,ctx", [([1], [0]), ([1], [63]), ([1], [64]), ([2], [127]), ([1], [128]),
                                      ([64], [0]), ([65], [0]), ([129], [1]), ([300], [100]),
                                      ([1, 1], [2000, 0])])
def test_lengths(sess, dtype, dim, lens, ctx):
    run(sess, lens, ctx, 4, 1, dim, dtype, seed=sum(lens) + sum(ctx))


@pytest.mark.parametrize("lens,ctx,heads,kvh,prefix", [
    ([700, 257, 64], [0, 1000, 31], 8, 2, 0),          # prompts: many row tiles, split keys
    ([90, 33], [500, 3], 16, 1, 640),                  # row tiles that cross requests in the prefix
    ([1] * 130, list(range(0, 1300, 10)), 8, 1, 256),  # more requests than a row tile has rows
    ([1], [20000], 8, 8, 0),                           # one long context: keys split over the GPU
    ([2, 1], [9000, 40], 4, 4, 8192),
])
def test_large(sess, lens, ctx, heads, kvh, prefix):
    run(sess, lens, ctx, heads, kvh, 128, BF, prefix=prefix, seed=len(lens))


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("scale,qscale", [(1.0, 3.0), (0.0, 1.0), (-0.3, 2.0), (20.0, 4.0)])
def test_scales_and_peaks(sess, dtype, dim, scale, qscale):
    """Peaked rows move the running maximum far between tiles; scale 0 is a plain mean."""
    run(sess, [17, 4], [400, 200], 4, 2, dim, dtype, prefix=128, scale=scale, qscale=qscale, seed=5)


@pytest.mark.parametrize("dtype,dim", KINDS)
def test_scores_far_below_zero(sess, dtype, dim):
    """Every score of the first keys far below the later ones, and the other way round."""
    for sign in (1.0, -1.0):
        pb = Paged([3], [500], kvh=1, dim=dim, dtype=dtype, seed=2)
        pages, rows = pb.slots(0, 0, 503)
        ramp = torch.linspace(-4, 4, 503, device="cuda") * sign
        pb.k[pages, rows] = (ramp[:, None, None] * torch.ones(1, 1, dim, device="cuda")).to(dtype)
        q = torch.full((3, 2, dim), 2.0, dtype=dtype, device="cuda")
        out = torch.full((3, 2, dim), FILL, dtype=dtype, device="cuda")
        lay = pb.layer(2)
        sess.paged_attention(lay, q, pb.row_start, pb.kv_len, out, sess.attention_workspace(lay, 1, 3))
        close(pb, q, 2, out, dim ** -0.5, True)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("lens,ctx,j", [([16], [20], 5), ([16], [115], 12), ([300], [0], 140), ([9], [3000], 3)])
@pytest.mark.parametrize("prefix", [0, 128])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(sess, dtype, dim, lens, ctx, j, prefix):
    """Row j's value has a NaN and infinities: rows before j are as without it, from j on those
    dims and no others are not finite.  The same with a NaN key: every dim from j on."""
    for what in ("v", "k"):
        pb = Paged(lens, ctx, prefix=prefix, kvh=1, dim=dim, dtype=dtype, seed=8)
        q = pb.normal(pb.rows, 5, dim)
        want = attend64(pb, q, 5, dim ** -0.5, True)
        pages, rows = pb.slots(0, prefix + ctx[0] + j, prefix + ctx[0] + j + 1)
        if what == "v":
            pb.v[pages, rows, 0, 3] = float("nan")
            pb.v[pages, rows, 0, dim - 2] = float("inf")
            pb.v[pages, rows, 0, dim // 2] = float("-inf")
        else:
            pb.k[pages, rows, 0, 9] = float("nan")
        hit = torch.zeros(dim, dtype=torch.bool, device="cuda")
        hit[[3, dim - 2, dim // 2] if what == "v" else slice(None)] = True
        out = torch.full((pb.rows, 5, dim), FILL, dtype=dtype, device="cuda")
        lay = pb.layer(5)
        sess.paged_attention(lay, q, pb.row_start, pb.kv_len, out, sess.attention_workspace(lay, 1, pb.rows))
        assert sess.error() == 0
        for t, (exact, spread, mag) in want.items():
            if t < j:
                half = torch.finfo(dtype).eps / 2
                ds = ((dim + 8) * 2.0 ** -24 * mag)[:, None]
                tol = half * exact.abs() + (half * (dtype == BF) + 2 * ds + 2.0 ** -18) * spread * (1 + half)
                assert float(((out[t].double() - exact).abs() - tol).max()) <= 0, t
            else:
                assert torch.equal(~torch.isfinite(out[t]), hit.expand(5, dim)), t


def test_batch_limits(sess):
    lens = [1 if i % 3 else 0 for i in range(1024)]
    run(sess, lens, [i % 70 for i in range(1024)], 2, 1, 64, BF, seed=1)
    run(sess, lens, [i % 70 for i in range(1024)], 2, 1, 128, BF, prefix=128, seed=1)
    run(sess, [0, 0], [3, 4], 2, 1, 128, BF, prefix=64, seed=1, trail=3)     # nobody has rows


def bad_case(sess, word, survivors, dtype, dim, prefix=0, **change):
    pb = Paged([3, 4, 2], [10, 60, 0], prefix=prefix, kvh=1, dim=dim, dtype=dtype, seed=6, trail=2)
    q = pb.normal(pb.rows, 2, dim)
    want = attend64(pb, q, 2, dim ** -0.5, True)
    for name, f in change.items():
        setattr(pb, name, f(getattr(pb, name)))
    out = torch.full((pb.rows, 2, dim), FILL, dtype=dtype, device="cuda")
    lay = pb.layer(2)
    sess.paged_attention(lay, q, pb.row_start, pb.kv_len, out, sess.attention_workspace(lay, 3, pb.rows))
    assert sess.error() == word
    rows = [t for b in survivors for t in range(pb.starts[b], pb.starts[b] + pb.lens[b])]
    for t in range(pb.rows):
        if t in rows:
            assert float((out[t].double() - want[t][0]).abs().max()) < 0.05
        else:
            assert bool((out[t] == FILL).all()), t


def put(i, v):
    def f(t):
        t = t.clone()
        t.view(-1)[i] = v
        return t
    return f


@pytest.mark.parametrize("dtype,dim", KINDS)
def test_requests_without_a_place_are_flagged_and_skipped(sess, dtype, dim):
    """Bad lengths and ranges: checked on the device before any cache access."""
    bad_case(sess, 0x1, [0, 2], dtype, dim, kv_len=put(1, -1))
    bad_case(sess, 0x1, [0, 2], dtype, dim, kv_len=put(1, 2 * PAGE - 3))
    bad_case(sess, 0x1, [0, 2], dtype, dim, kv_len=put(1, 2 ** 31 - 2))
    bad_case(sess, 0x1, [0, 2], dtype, dim, prefix=128, kv_len=put(1, 127))
    bad_case(sess, 0x40, [1, 2], dtype, dim, row_start=put(0, -1))
    bad_case(sess, 0x40, [0, 1], dtype, dim, row_start=put(3, 12))


@pytest.mark.parametrize("dim,prefix", [(128, 0), (64, 0), (128, 128)])
def test_ranges_that_repeat_every_row_are_flagged_and_nothing_is_written(sess, dim, prefix):
    """40 ranges, 20 of them all rows and 20 decreasing: more rows than the workspace was sized for."""
    pb = Paged([6] + [0] * 39, [10] * 40, prefix=prefix, kvh=1, dim=dim, dtype=BF, seed=4)
    q, lay = pb.normal(pb.rows, 64, dim), pb.layer(64)
    pb.row_start = i32([0, 6] * 20 + [0])
    out = torch.full((pb.rows, 64, dim), FILL, dtype=BF, device="cuda")
    sess.paged_attention(lay, q, pb.row_start, pb.kv_len, out, sess.attention_workspace(lay, 40, pb.rows))
    assert sess.error() == 0x40
    assert bool((out == FILL).all())
    run(sess, [3], [4], 4, 1, dim, BF, prefix=prefix)


@pytest.mark.parametrize("dtype,dim", KINDS)
def test_bad_pages_are_flagged(sess, dtype, dim):
    """An id outside the pool is never followed; the other requests are right."""
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        pb = Paged([3, 4], [10, 60], kvh=1, dim=dim, dtype=dtype, seed=6)
        q = pb.normal(7, 2, dim)
        want = attend64(pb, q, 2, dim ** -0.5, True)
        pb.table = put(0, bad)(pb.table)
        out = torch.full((7, 2, dim), FILL, dtype=dtype, device="cuda")
        lay = pb.layer(2)
        sess.paged_attention(lay, q, pb.row_start, pb.kv_len, out, sess.attention_workspace(lay, 2, 7))
        assert sess.error() == 0x2
        for t in range(3, 7):
            assert float((out[t].double() - want[t][0]).abs().max()) < 0.05


@pytest.mark.parametrize("dtype,dim", KINDS)
def test_two_streams_with_a_workspace_each(sess, dtype, dim):
    jobs = []
    for seed in (1, 2):
        pb = Paged([16] * 6, [900, 3, 64, 700, 128, 1], prefix=256, kvh=2, dim=dim, dtype=dtype, seed=seed)
        lay = pb.layer(8)
        q = pb.normal(pb.rows, 8, dim)
        jobs.append((pb, lay, q, torch.full_like(q, FILL), sess.attention_workspace(lay, 6, pb.rows),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for pb, lay, q, out, ws, s in jobs:
            with torch.cuda.stream(s):
                sess.paged_attention(lay, q, pb.row_start, pb.kv_len, out, ws)
    torch.cuda.synchronize()
    for pb, lay, q, out, ws, s in jobs:
        close(pb, q, 8, out, dim ** -0.5, True)


@pytest.mark.parametrize("dtype,dim", KINDS)
def test_graph_replays_follow_the_lengths(sess, dtype, dim):
    """Captured once; replays read the lengths that the device arrays hold then.  Two graphs share
    the workspace and run one after the other."""
    pb = Paged([16, 16], [300, 40], prefix=64, kvh=2, dim=dim, dtype=dtype, seed=3)
    lay = pb.layer(8)
    q = pb.normal(32, 8, dim)
    outs = [torch.full_like(q, FILL) for _ in range(2)]
    ws = sess.attention_workspace(lay, 2, 32)
    graphs = []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sess.paged_attention(lay, q, pb.row_start, pb.kv_len, out, ws)
        graphs.append(g)
    for ctx in ([300, 40], [5, 17], [64, 0]):
        pb.ctx = ctx
        pb.kv_len.copy_(i32([64 + c for c in ctx]))
        for g in graphs:
            g.replay()
        for out in outs:
            close(pb, q, 8, out, dim ** -0.5, True)


def test_same_bits_every_run(sess):
    pb, q, lay, ws, out = run(sess, [16] * 40, [100 * i for i in range(40)], 32, 8, 128, prefix=1024,
                              seed=8, spoil=False)
    again = torch.full_like(out, FILL)
    for _ in range(3):
        sess.paged_attention(lay, q, pb.row_start, pb.kv_len, again, ws)
        assert torch.equal(out, again)


def test_python_checks(sess):
    pb = Paged([2], [0], kvh=1, dim=64, seed=1)
    lay, q = pb.layer(2), pb.normal(2, 2, 64)
    ws, out = sess.attention_workspace(lay, 1, 2), torch.empty(2, 2, 64, dtype=BF, device="cuda")
    args = dict(layer=lay, q=q, row_start=pb.row_start, kv_len=pb.kv_len, out=out, workspace=ws)
    for bad in [dict(q=q.float()), dict(out=out[:1]), dict(q=q.transpose(0, 1)), dict(workspace=ws.int()),
                dict(row_start=pb.row_start[:1]), dict(kv_len=pb.kv_len.long()), dict(q=q.cpu())]:
        with pytest.raises(ValueError):
            sess.paged_attention(**{**args, **bad})
    for bad in [dict(workspace=ws[:0]), dict(out=q)]:
        with pytest.raises(pkg.DFlashError):
            sess.paged_attention(**{**args, **bad})
    with pytest.raises(ValueError):
        pkg.LayerKV(2, pb.k, pb.v[:1], pb.table)
    with pytest.raises(ValueError):
        pkg.LayerKV(2, pb.k[:, :32], pb.v[:, :32], pb.table)
