"""Eviction from a cache against plain forms: attention weight per cached row, the rows that a budget
keeps, moving rows together.

Tolerance of a weight, from tests.tree_reference.weights64: every term's exponent has a score's error, (D +
8) 2^-24 of scale * sum_d |q_d k_d|, 2^-22 of |lse| and of |log row_weight| (their products with log2 e and
roundings), 2^-20 for the exponential; a sum of n terms n 2^-24 of itself; the old weight is met by three
roundings (of the factor, the product, the last addition), 2^-24 each.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_diffusion_speculative_fc_gb300 as pkg  # noqa: E402
from tests.target_reference import PAGE, Paged, i32, make_session  # noqa: E402
from tests.tree_reference import (causal, choose, closure, pack, random_parents, rng_of, scores64,  # noqa: E402
                                  weights64)

BF, F32 = torch.bfloat16, torch.float32
FILL = -7.0
KINDS = [(BF, 128), (BF, 64), (F32, 128), (F32, 64)]


@pytest.fixture(scope="module")
def sess():
    s = make_session()
    yield s
    s.close()


# ---------------------------------------------------------------- weights
def weigh(sess, lens, ctx, heads, kvh, dim, dtype=BF, prefix=0, seed=0, decay=1.0, kind="causal", rows="all",
          scale=None, spare=0, strided=True, **kw):
    pb = Paged(lens, ctx, prefix=prefix, kvh=kvh, dim=dim, dtype=dtype, seed=seed, **kw)
    sc = dim ** -0.5 if scale is None else scale
    used = torch.zeros((pb.n_pages, PAGE), dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        pages, rw = pb.slots(b, 0, prefix + ctx[b] + n)
        used[pages, rw] = True
    pb.k[~used] = float("nan")
    pb.v[:] = float("nan")                     # values have no part in it
    rng = rng_of(seed)
    seen = [(closure(random_parents(n, rng)) if kind == "tree" else causal(n)) if n else None for n in lens]
    words = (max(lens) + 31) // 32
    mask = pack([m for m in seen if m is not None], pb.rows, [s for s, n in zip(pb.starts, lens) if n], words,
                fill=-1) if kind == "tree" else None
    q = pb.normal(pb.rows, heads * dim + 64)[:, :heads * dim].unflatten(1, (heads, dim)) if strided else \
        pb.normal(pb.rows, heads, dim)
    lse = torch.zeros((pb.rows, heads), device="cuda")
    for b, n in enumerate(lens):
        if n:
            lse[pb.starts[b]:pb.starts[b] + n] = torch.logsumexp(scores64(pb, q, heads, sc, b, seen[b])[0], -1).float()
    row_weight = None
    if rows == "some":
        row_weight = (torch.rand(pb.rows, generator=pb.g, device="cuda") < 0.5).float()
    elif rows == "any":
        row_weight = torch.rand(pb.rows, generator=pb.g, device="cuda") * 3
    width = max(c + n for c, n in zip(ctx, lens)) + spare
    old = torch.rand((len(lens), kvh, width), generator=pb.g, device="cuda")
    for b, n in enumerate(lens):               # nothing is read of the rows of the call, nor with decay 0
        old[b, :, (0 if decay == 0 else ctx[b]):ctx[b] + n] = float("nan") if n else 0.5
    want, tol, live = weights64(pb, q, heads, sc, seen, lse, row_weight, decay, old.nan_to_num(0.0) if decay == 0 else old)
    got = old.clone()
    lay = pb.layer(heads)
    sess.key_weights(lay, q, pb.row_start, pb.kv_len, lse, got, mask=mask, row_weight=row_weight, decay=decay,
                     scale=scale)
    assert sess.error() == 0
    at = live[:, None].expand_as(got)
    over = (got.double() - want).abs()[at] - tol[at]
    assert float(over.max()) <= 0, (float(over.max()), float(want[at].max()))
    assert torch.equal(got[~at].nan_to_num(9.0), old[~at].nan_to_num(9.0))
    again = old.clone()
    sess.key_weights(lay, q, pb.row_start, pb.kv_len, lse, again, mask=mask, row_weight=row_weight, decay=decay,
                     scale=scale)
    assert torch.equal(again[at], got[at])     # the same in every run
    return pb, q, lse, got, old


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("heads,kvh", [(1, 1), (8, 2), (5, 1), (128, 1), (21, 3), (16, 16)])
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_head_layouts(sess, dtype, dim, heads, kvh, kind):
    weigh(sess, [1, 16, 0, 5], [0, 63, 9, 130], heads, kvh, dim, dtype, seed=heads, kind=kind)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("lens,ctx", [([1], [0]), ([1], [63]), ([1], [127]), ([1], [128]), ([2], [64]), ([33], [0]),
                                      ([64], [200]), ([65], [63]), ([129], [1]), ([300], [100]),
                                      ([1, 1], [2000, 0])])
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_lengths(sess, dtype, dim, lens, ctx, kind):
    weigh(sess, lens, ctx, 4, 1, dim, dtype, seed=sum(lens) + sum(ctx), kind=kind, spare=5)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("rows", ["all", "some", "any"])
@pytest.mark.parametrize("prefix", [0, 192])
def test_decay_rows_prefix(sess, dtype, dim, decay, rows, prefix):
    weigh(sess, [16, 3, 1, 0, 40], [0, 64, 127, 5, 300], 8, 2, dim, dtype, prefix=prefix, seed=7, decay=decay,
          rows=rows, kind="tree", lead=1, trail=2)


@pytest.mark.parametrize("lens,ctx,heads,kvh", [
    ([64, 64], [3000, 9000], 16, 2),            # windows: two blocks of query rows, many tiles
    ([700], [0], 8, 1),                         # a prompt: blocks that see none of the late keys
    ([1] * 130, list(range(0, 1300, 10)), 8, 1),
    ([1], [20000], 8, 8),
    ([100, 1, 33], [10, 5000, 300], 128, 1),    # 50 blocks of query rows
    ([1000], [500], 2, 1),
])
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_large(sess, lens, ctx, heads, kvh, kind):
    weigh(sess, lens, ctx, heads, kvh, 128, BF, seed=len(lens), kind=kind, decay=0.9, rows="some")


# 129 to 256 query rows a request and KV head on average, more and fewer in some
@pytest.mark.parametrize("lens,ctx,heads,kvh", [([64] * 5, [700, 0, 64, 1999, 5000], 32, 8),
                                                ([33, 90, 1, 17], [100, 3000, 777, 0], 8, 2),
                                                ([20, 2, 9], [1500, 40, 0], 128, 8)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_middling_rows(sess, lens, ctx, heads, kvh, dim, kind):
    weigh(sess, lens, ctx, heads, kvh, dim, BF, seed=dim, decay=0.5, rows="some", kind=kind)


# whole prompts: most shares of the keys are seen by the later blocks of query rows alone
@pytest.mark.parametrize("lens,ctx,heads,kvh", [([3000], [0], 16, 2), ([1500, 1, 900], [0, 40, 129], 64, 1)])
@pytest.mark.parametrize("dim", [64, 128])
def test_blocks_that_see_nothing_of_a_share(sess, lens, ctx, heads, kvh, dim):
    weigh(sess, lens, ctx, heads, kvh, dim, BF, seed=dim, decay=0.5, rows="any")


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_scales(sess, dtype, dim, scale):
    weigh(sess, [17, 4], [400, 200], 4, 2, dim, dtype, scale=scale, seed=5)


@pytest.mark.parametrize("dtype,dim", KINDS)
def test_rows_that_count_for_nothing(sess, dtype, dim):
    """Queries of rows without weight, or whose lse is not finite, may hold anything; a key that is not
    finite spoils its own weight alone, and only where a row that counts sees it."""
    lens, ctx, heads = [20, 6], [150, 40], 8
    pb = Paged(lens, ctx, kvh=2, dim=dim, dtype=dtype, seed=4)
    rng = rng_of(1)
    seen = [closure(random_parents(n, rng)) for n in lens]
    mask = pack(seen, 26, pb.starts, 1)
    q = pb.normal(26, heads, dim)
    lse = torch.zeros((26, heads), device="cuda")
    for b, n in enumerate(lens):
        lse[pb.starts[b]:pb.starts[b] + n] = torch.logsumexp(
            scores64(pb, q, heads, dim ** -0.5, b, seen[b])[0], -1).float()
    rw = torch.ones(26, device="cuda")
    rw[[2, 9, 21]] = torch.tensor([0.0, -1.0, float("nan")], device="cuda")
    lse[5], lse[6], lse[7] = float("inf"), -float("inf"), float("nan")
    out = [2, 5, 6, 7, 9, 21]
    q[out] = float("nan")
    q[out[0]] = float("inf")
    clean = q.clone()
    clean[out] = 0
    base = torch.zeros((2, 2, 170), device="cuda")
    want, tol, live = weights64(pb, clean, heads, dim ** -0.5, seen, lse, rw, 0.0, base)
    got = base.clone()
    sess.key_weights(pb.layer(heads), q, pb.row_start, pb.kv_len, lse, got, mask=mask, row_weight=rw, decay=0.0)
    assert sess.error() == 0
    assert bool(((got.double() - want).abs() <= tol)[live[:, None].expand_as(got)].all())
    # new row 19 of request 0 (a leaf, seen by itself alone) and cached row 3, which every row sees
    pages, rows = pb.slots(0, 0, 170)
    for row, what in ((169, float("inf")), (169, float("nan")), (3, float("nan"))):
        keep = pb.k[pages[row], rows[row]].clone()
        pb.k[pages[row], rows[row]] = what
        rw[19] = 0.0
        want2, tol2, _ = weights64(pb, clean, heads, dim ** -0.5, [torch.where(torch.arange(20)[:, None] == 19, False, seen[0]),
                                                                  seen[1]], lse, rw, 0.0, base)
        sess.key_weights(pb.layer(heads), q, pb.row_start, pb.kv_len, lse, got, mask=mask, row_weight=rw, decay=0.0)
        pb.k[pages[row], rows[row]] = keep
        others = live.clone()
        others[0, row] = False
        assert bool(((got.double() - want2).abs() <= tol2)[others[:, None].expand_as(got)].all())
        if row == 169:                          # no row that counts sees it
            assert bool((got[0, :, row] == 0).all())
        else:
            assert bool(got[0, :, row].isnan().all())
    assert sess.error() == 0


def test_weights_refuse_lengths_and_pages(sess):
    for dt in (BF, F32):
        pb = Paged([4, 4, 40, 4], [100, 100, 10, 100], kvh=1, dim=64, dtype=dt, seed=1)
        q, lse = pb.normal(52, 2, 64), torch.zeros((52, 2), device="cuda")
        lay = pb.layer(2)
        pb.kv_len[1] = 64 * pb.width - 3
        mask = torch.zeros((52, 1), dtype=torch.int32, device="cuda")
        got = torch.full((4, 1, 104), FILL, device="cuda")
        sess.key_weights(lay, q, pb.row_start, pb.kv_len, lse, got, mask=mask, decay=0.0)
        assert set(pkg.decode_error(sess.error())) == {"KV_CAPACITY", "TREE"}
        assert bool((got[1:3] == FILL).all()) and bool((got[[0, 3]] != FILL).all())
        got = torch.full((4, 1, 103), FILL, device="cuda")       # a row too narrow
        pb.kv_len[1] = 99
        pb.table[1, 1] = -1
        sess.key_weights(lay, q, pb.row_start, pb.kv_len, lse, got, decay=0.0)
        assert set(pkg.decode_error(sess.error())) == {"KV_CAPACITY", "PAGE_RANGE"}
        assert bool((got[[0, 3]] == FILL).all()) and bool((got[1] != FILL).all())


# ---------------------------------------------------------------- which rows
def chosen(sess, w, n, keep, first, last, prefix=0, max_keep=None, kvh=None):
    B, KVH, width = w.shape
    max_keep = max_keep or max(1, max(keep))
    rows = torch.full((B, KVH, max_keep), -9, dtype=torch.int32, device="cuda")
    count = torch.full((B, KVH), -9, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros((1, PAGE, KVH, 64), device="cuda") for _ in "kv")
    pp = torch.zeros(prefix // 64, dtype=torch.int32, device="cuda") if prefix else None
    lay = pkg.LayerKV(KVH, k, v, torch.zeros((B, 1), dtype=torch.int32, device="cuda"), pp)
    sess.choose_rows(lay, w, i32([prefix + x for x in n]), i32(keep), rows, count, first=first, last=last)
    return rows, count


@pytest.mark.parametrize("n", [[1], [2, 0, 7], [31, 32, 33, 64], [1000, 5, 4097], [40000], [70000, 131, 400000]])
@pytest.mark.parametrize("first,last", [(0, 0), (4, 0), (3, 40), (10 ** 9, 5), (0, 10 ** 9)])
@pytest.mark.parametrize("kind", ["spread", "few", "same", "tiny"])
def test_choose(sess, n, first, last, kind):
    B, KVH, width = len(n), 3, max(n) + 2
    g = torch.Generator(device="cuda").manual_seed(sum(n))
    w = torch.rand((B, KVH, width), generator=g, device="cuda")
    if kind == "spread":
        w = torch.exp(20 * (w - 0.5)) * torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.1, -1, 1)
    elif kind == "few":
        w = (w * 5).floor()
    elif kind == "same":
        w = torch.zeros_like(w)
        w[:, 0, ::2] = -0.0                    # equal to 0
        w[:, 1] = float("nan")
    else:
        w = w * 1e-40                          # subnormal ones keep their order
        w[..., ::5] = -w[..., ::5]
    if kind == "spread" and max(n) > 20:
        w[..., 3], w[..., 5], w[..., 7], w[..., 9] = float("inf"), -float("inf"), float("nan"), 3.0e38
    keep = [max(0, (x * 3 + b) // (4 + b)) for b, x in enumerate(n)]
    rows, count = chosen(sess, w, n, keep, first, last)
    assert sess.error() == 0
    wl = w.cpu()
    for b, x in enumerate(n):
        for h in range(KVH):
            want = choose(wl[b, h].tolist(), x, keep[b], first, last)
            assert int(count[b, h]) == len(want)
            got = rows[b, h].cpu()
            assert torch.equal(got[:len(want)], torch.tensor(want, dtype=torch.int32)), (b, h)
            assert bool((got[len(want):] == -9).all())


def test_choose_behind_a_prefix_many_lists_and_edges(sess):
    g = torch.Generator(device="cuda").manual_seed(3)
    n = [5 * i for i in range(300)]
    w = torch.rand((300, 2, 1500), generator=g, device="cuda")
    keep = [(7 * i) % 400 for i in range(300)]
    rows, count = chosen(sess, w, n, keep, 2, 3, prefix=128, max_keep=450)
    assert sess.error() == 0
    wl = w.tolist()
    for b in range(300):
        for h in range(2):
            want = choose(wl[b][h], n[b], keep[b], 2, 3)
            assert rows[b, h, :int(count[b, h])].tolist() == want
    # budgets and lengths out of range
    rows, count = chosen(sess, w[:4], [100, 100, -1, 1501], [-1, 11, 5, 5], 0, 0, max_keep=10)
    assert set(pkg.decode_error(sess.error())) == {"ROW_LIST", "KV_CAPACITY"}
    assert bool((rows == -9).all()) and bool((count == -9).all())


# ---------------------------------------------------------------- moving rows
def moved(pb, first, lists, weights):
    k, v = pb.k.clone(), pb.v.clone()
    w = weights.clone() if weights is not None else None
    for b, per in enumerate(lists):
        for g in range(pb.kvh):
            rows = per[g % len(per)]
            pages, at = pb.slots(b, 0, pb.prefix + 64 * len(pb.lists[b]))
            for i, r in enumerate(rows):
                s, d = first[b] + r, first[b] + i
                k[pages[d], at[d], g], v[pages[d], at[d], g] = pb.k[pages[s], at[s], g], pb.v[pages[s], at[s], g]
            if w is not None:
                own = first[b] - pb.prefix
                w[b, g, own:own + len(rows)] = weights[b, g][[own + r for r in rows]]
    return k, v, w


def lists_of(rng, B, L, rows, most):
    out = []
    for b in range(B):
        out.append([sorted(rng.sample(range(rows[b]), min(rows[b], rng.randrange(most[b] + 1)))) for _ in range(L)])
    return out


def keep_call(sess, pb, first, lists, weights, spare=2):
    B, L = len(lists), len(lists[0])
    width = max(1, max(len(r) for p in lists for r in p)) + spare
    rows = torch.full((B, L, width), -1, dtype=torch.int32)
    for b, per in enumerate(lists):
        for g, r in enumerate(per):
            rows[b, g, :len(r)] = torch.tensor(r, dtype=torch.int32)
    count = i32([[len(r) for r in p] for p in lists])
    sess.keep_rows(pb.layer(pb.kvh), rows.cuda(), count, first=None if first is None else i32(first), weights=weights)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("kvh", [1, 3, 8])
@pytest.mark.parametrize("per_head", [True, False])
@pytest.mark.parametrize("weighted", [True, False])
def test_keep(sess, dtype, dim, kvh, per_head, weighted):
    ctx = [0, 700, 64, 130, 1]
    pb = Paged([30, 3, 1, 70, 0], ctx, prefix=64, kvh=kvh, dim=dim, dtype=dtype, seed=kvh)
    rng = rng_of(kvh)
    rows = [30, 703, 65, 200, 1] if per_head else [30, 3, 1, 70, 0]
    first = [64] * 5 if per_head else [64 + c for c in ctx]
    lists = lists_of(rng, 5, kvh if per_head else 1, rows, rows)
    weights = torch.rand((5, kvh, 703), device="cuda") if weighted else None
    k, v, w = moved(pb, first, lists, weights)
    keep_call(sess, pb, None if per_head else first, lists, weights)
    assert sess.error() == 0
    assert torch.equal(pb.k, k) and torch.equal(pb.v, v)
    assert w is None or torch.equal(weights, w)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("share", [0.02, 0.5, 0.97])
@pytest.mark.parametrize("batch", [1, 40])
def test_keep_long_lists(sess, dtype, share, batch):
    """Many steps of every CTA, with sources near and far from their places."""
    n = 9000 if batch == 1 else 1500
    pb = Paged([1] * batch, [n - 1] * batch, kvh=2, dim=128, dtype=dtype, seed=batch)
    g = torch.Generator().manual_seed(int(100 * share))
    lists = [[(torch.rand(n, generator=g) < share).nonzero()[:, 0].tolist() for _ in range(2)] for _ in range(batch)]
    weights = torch.rand((batch, 2, n), device="cuda")
    k0, v0, w0 = pb.k.clone(), pb.v.clone(), weights.clone()
    keep_call(sess, pb, None, lists, weights)
    assert sess.error() == 0
    for b in range(batch):
        pages, at = (torch.tensor(x, device="cuda") for x in pb.slots(b, 0, n))
        for h in range(2):
            src = torch.tensor(lists[b][h], device="cuda")
            d = torch.arange(len(src), device="cuda")
            k0[pages[d], at[d], h], v0[pages[d], at[d], h] = k0[pages[src], at[src], h], v0[pages[src], at[src], h]
            w0[b, h, d] = w0[b, h, src]
    assert torch.equal(pb.k, k0) and torch.equal(pb.v, v0) and torch.equal(weights, w0)


def test_keep_all_or_none_changes_nothing(sess):
    pb = Paged([5, 5], [200, 64], kvh=2, dim=64)
    k0, v0 = pb.k.clone(), pb.v.clone()
    keep_call(sess, pb, None, [[list(range(205))] * 2, [[], []]], None)
    assert sess.error() == 0 and torch.equal(pb.k, k0) and torch.equal(pb.v, v0)


def test_keep_refuses_a_list_whole(sess):
    pb = Paged([10] * 6, [100] * 6, kvh=2, dim=64, prefix=64, seed=9)
    k0, v0 = pb.k.clone(), pb.v.clone()
    weights = torch.rand((6, 2, 110), device="cuda")
    w0 = weights.clone()
    lay = pb.layer(2)
    rows = i32([[1, 3, 2], [1, 1, 2], [-1, 2, 3], [1, 2, 28], [1, 2, 10], [2, 5, 9]])
    first = i32([164, 164, 164, 164, 63, 164])
    for count, errors in (([3, 3, 3, 3, 3, 3], {"ROW_LIST", "KV_CAPACITY"}), ([-1, 4, 0, 0, 0, 0], {"ROW_LIST"})):
        pb.k.copy_(k0), pb.v.copy_(v0)
        sess.keep_rows(lay, rows, i32(count), first=first, weights=None)
        assert set(pkg.decode_error(sess.error())) == errors
        k, v, _ = moved(Like(pb, k0, v0), [164] * 6, [[[]]] * 5 + [[[2, 5, 9] if count[5] else []]], None)
        assert torch.equal(pb.k, k) and torch.equal(pb.v, v)
    # a weight's row that is not there (own row 110), a page that is not
    pb.k.copy_(k0), pb.v.copy_(v0)
    pb.table[1, 1] = 10 ** 6
    sess.keep_rows(lay, rows[:2].clone().copy_(i32([[1, 2, 10], [1, 2, 9]])), i32([3, 3]), first=i32([164, 164]),
                   weights=weights[:2])
    assert set(pkg.decode_error(sess.error())) == {"KV_CAPACITY", "PAGE_RANGE"}
    assert torch.equal(pb.k, k0) and torch.equal(pb.v, v0) and torch.equal(weights, w0)


class Like:
    """A batch's layout over other pages."""

    def __init__(self, pb, k, v):
        self.k, self.v, self.kvh, self.prefix, self.lists, self.slots = k, v, pb.kvh, pb.prefix, pb.lists, pb.slots
