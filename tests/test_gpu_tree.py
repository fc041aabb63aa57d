"""Trees of drafted tokens against their plain forms: masks and positions, rotation to given positions,
attention under masks with the log of the softmax sum, the walk and its commit.

Tolerance of the attention, element by element, as for the paged attention: out rounded once to the
storage type; in bf16 every weight rounded once (eps / 2 of sum_p softmax |V| in all); a score's error,
(D + 8) 2^-24 of the largest scale * sum_d |q_d k_d|, moves numerator and denominator by as much; 2^-18 for
fp32 sums and the exponential.  lse: a score's error, 2^-18 for the sum, 2^-22 of itself for the
product with ln 2, log2 and the last addition.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_diffusion_speculative_fc_gb300 as pkg  # noqa: E402
from tests.target_reference import PAGE, Paged, i32, make_session, rope64  # noqa: E402
from tests.tree_reference import (attend_tree64, causal, closure, pack, random_parents, rng_of,  # noqa: E402
                                  walk)

BF, F32 = torch.bfloat16, torch.float32
FILL = -7.0
VOCAB = 256
KINDS = [(BF, 128), (BF, 64), (F32, 128), (F32, 64)]


@pytest.fixture(scope="module")
def sess():
    s = make_session(vocab=VOCAB)
    yield s
    s.close()


# ---------------------------------------------------------------- masks and positions
def starts_of(lens, lead=0):
    s = [lead]
    for n in lens:
        s.append(s[-1] + n)
    return s


@pytest.mark.parametrize("lens,words", [([1], 1), ([0, 1, 0, 2], 1), ([32, 31, 33], 2), ([64], 2),
                                        ([5, 1000, 1024, 3], 32), ([256] * 40, 8), ([17, 200], 32)])
def test_plan(sess, lens, words):
    rng = rng_of(sum(lens))
    starts = starts_of(lens, lead=2)
    T = starts[-1] + 3
    trees = [random_parents(n, rng, back=rng.choice([1, 2, 8, 2000])) if n else [] for n in lens]
    par = [0, 0] + [p for t in trees for p in t] + [0] * 3
    root = [rng.randrange(100000) for _ in lens]
    mask = torch.full((T, words), -77, dtype=torch.int32, device="cuda")
    pos = torch.full((T,), -5, dtype=torch.int32, device="cuda")
    sess.tree_plan(i32(starts), i32(par), mask, pos, root=i32(root))
    assert sess.error() == 0
    seen = [closure(t) for t in trees if t]
    want = pack(seen, T, [s for s, t in zip(starts, trees) if t], words)
    own = slice(2, starts[-1])
    assert torch.equal(mask[own], want[own])
    depth = [int(x) - 1 for m in seen for x in m.sum(1)]
    base = [r for r, t in zip(root, trees) for _ in t]
    assert pos[own].tolist() == [a + b for a, b in zip(base, depth)]
    for t in (mask, pos):
        assert bool((t[:2] == (-77 if t is mask else -5)).all()) and bool((t[starts[-1]:] == (-77 if t is mask else -5)).all())


def test_plan_of_a_forest_and_without_positions(sess):
    par = [-1, -1, 0, 1, -1, 4, 2]
    mask = torch.zeros((7, 1), dtype=torch.int32, device="cuda")
    sess.tree_plan(i32([0, 7]), i32(par), mask, root=i32([3]))
    assert mask[:, 0].tolist() == [0b1, 0b10, 0b101, 0b1010, 0b10000, 0b110000, 0b1000101]
    assert sess.error() == 0


@pytest.mark.parametrize("bad", [[-1, 0, 2], [-1, 0, 3], [-1, -2, 0], [0, 0, 0], [-1, 2 ** 30, 0]])
def test_plan_and_walk_refuse_a_parent_out_of_range(sess, bad):
    mask = torch.full((5, 1), 9, dtype=torch.int32, device="cuda")
    par, rs = i32([-1, 0] + bad), i32([0, 2, 5])
    sess.tree_plan(rs, par, mask, root=i32([0, 0]))
    assert pkg.decode_error(sess.error()) == ["TREE"]
    assert mask[:, 0].tolist() == [1, 3, 9, 9, 9]            # the other request is served
    got = accept(sess, [2, 3], [-1, 0] + bad, [1] * 5, [1] * 5, 4)
    assert pkg.decode_error(sess.error()) == ["TREE"]
    assert got["commit_len"].tolist() == [2, FILL_I]
    assert got["path"][1].tolist() == [FILL_I] * 4


def test_more_rows_than_the_mask_has_room_for(sess):
    mask = torch.full((35, 1), 9, dtype=torch.int32, device="cuda")
    sess.tree_plan(i32([0, 33, 35]), i32([-1] + [0] * 32 + [-1, 0]), mask, root=i32([0, 0]))
    assert pkg.decode_error(sess.error()) == ["TREE"]
    assert bool((mask[:33] == 9).all()) and mask[33:, 0].tolist() == [1, 3]
    for dt in (BF, F32):
        pb = Paged([33, 2], [10, 5], kvh=1, dim=64, dtype=dt)
        out, lse = attend(sess, pb, 1, pack([closure([-1, 0])], 35, [33], 1), strided=False, check_error=False)[1:3]
        assert pkg.decode_error(sess.error()) == ["TREE"]
        assert bool((out[:33] == FILL).all()) and bool((lse[:33] == FILL).all())
        assert bool((out[33:] != FILL).all())


# ---------------------------------------------------------------- rotation to given positions
@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("rot,inter", [(64, False), (64, True), (32, False), (10, False)])
def test_append_at_positions(sess, dtype, dim, rot, inter):
    pb = Paged([3, 0, 20], [70, 5, 0], prefix=64, kvh=2, dim=dim, dtype=dtype, seed=rot, lead=1, trail=1,
               fill=FILL)
    T = pb.rows
    q, k, v = pb.normal(T, 4, dim), pb.normal(T, 2, dim), pb.normal(T, 2, dim)
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=pb.g, device="cuda", dtype=torch.int32)
    pos[::2] %= 1000
    plan = pkg.rope_plan(rot, 1e6, interleaved=inter)
    out = torch.full_like(q, FILL)
    lay = pb.layer(4)
    sess.append_kv(lay, q, k, v, pb.row_start, pb.kv_len, plan, q_out=out, positions=pos)
    assert sess.error() == 0
    # angles as the plan holds them: turns of 2^-64, reduced exactly
    turns = torch.tensor([[(int(p) * t) % 2 ** 64 / 2.0 ** 64 for t in plan.turns[:rot // 2]] for p in pos.tolist()],
                         dtype=torch.float64, device="cuda") * 2 * torch.pi
    half = torch.finfo(dtype).eps / 2
    written = torch.zeros((pb.n_pages, PAGE), dtype=torch.bool, device="cuda")
    for b, n in enumerate(pb.lens):
        if not n:
            continue
        rows = slice(pb.starts[b], pb.starts[b] + n)
        at = pb.slots(b, 64 + pb.ctx[b], 64 + pb.ctx[b] + n)
        written[at[0], at[1]] = True
        for src, got in ((q[rows], out[rows]), (k[rows], pb.k[at])):
            for i in range(n):
                y, big = rope64(src[i:i + 1].double(), torch.ones(1, device="cuda"), turns[rows][i], 1.0, inter)
                assert bool(((got[i:i + 1].double() - y).abs() <= half * y.abs() + 2.0 ** -20 * big).all())
        assert torch.equal(pb.v[at], v[rows])
    assert bool((pb.k[~written] == FILL).all()) and bool((pb.v[~written] == FILL).all())
    assert bool((out[0] == FILL).all()) and bool((out[-1] == FILL).all())


def test_append_at_the_cache_rows_is_append(sess):
    pb = Paged([5, 9], [100, 3], kvh=2, dim=128)
    T = pb.rows
    q, k, v = pb.normal(T, 4, 128), pb.normal(T, 2, 128), pb.normal(T, 2, 128)
    plan, lay = pkg.rope_plan(128, 1e6), pb.layer(4)
    res = []
    for pos in (None, i32([100 + i for i in range(5)] + [3 + i for i in range(9)])):
        pb.k.zero_()
        out = torch.zeros_like(q)
        sess.append_kv(lay, q, k, v, pb.row_start, pb.kv_len, plan, q_out=out, positions=pos)
        res.append((out, pb.k.clone()))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    assert sess.error() == 0


# ---------------------------------------------------------------- attention under masks
def attend(sess, pb, heads, mask, scale=None, qscale=1.0, strided=True, want_lse=True, check_error=True):
    dt, D = pb.dtype, pb.dim
    if strided:
        q = pb.normal(pb.rows, heads * D + 64, scale=qscale)[:, :heads * D].unflatten(1, (heads, D))
        out = torch.full((pb.rows, heads * D + 8), FILL, dtype=dt, device="cuda")
        out = out[:, :heads * D].unflatten(1, (heads, D))
    else:
        q = pb.normal(pb.rows, heads, D, scale=qscale)
        out = torch.full((pb.rows, heads, D), FILL, dtype=dt, device="cuda")
    lse = torch.full((pb.rows, heads), FILL, device="cuda") if want_lse else None
    lay = pb.layer(heads)
    ws = sess.attention_workspace(lay, len(pb.lens), pb.rows)
    ws.fill_(255)                              # nothing is expected of the workspace
    sess.tree_attention(lay, q, pb.row_start, pb.kv_len, out, ws, mask=mask, scale=scale, lse=lse)
    if check_error:
        assert sess.error() == 0
    return q, out, lse


def close(pb, q, heads, out, lse, scale, seen):
    dt, D = pb.dtype, pb.dim
    half = torch.finfo(dt).eps / 2
    owned = torch.zeros(pb.rows, dtype=torch.bool, device="cuda")
    for t, (want, spread, mag, want_lse) in attend_tree64(pb, q, heads, scale, seen).items():
        owned[t] = True
        ds = ((D + 8) * 2.0 ** -24 * mag)[:, None]
        tol = half * want.abs() + (half * (dt == BF) + 2 * ds + 2.0 ** -18) * spread * (1 + half)
        over = (out[t].double() - want).abs() - tol
        assert float(over.max()) <= 0, (t, float(over.max()), float(want.abs().max()))
        if lse is not None:
            none = want_lse == -torch.inf
            assert bool((lse[t][none] == -torch.inf).all())
            d = (lse[t].double() - want_lse).abs()[~none]
            assert bool((d <= (ds[:, 0] + 2.0 ** -18 + 2.0 ** -22 * want_lse.abs())[~none]).all()), t
    assert bool((out[~owned] == FILL).all())
    assert lse is None or bool((lse[~owned] == FILL).all())


def spoil(pb):
    """Every cache row that belongs to no request holds NaN, those past a request's last too."""
    used = torch.zeros((pb.n_pages, PAGE), dtype=torch.bool, device="cuda")
    for b, n in enumerate(pb.lens):
        pages, rows = pb.slots(b, 0, pb.prefix + pb.ctx[b] + n)
        used[pages, rows] = True
    pb.k[~used] = float("nan")
    pb.v[~used] = float("nan")


def run(sess, lens, ctx, heads, kvh, dim, dtype=BF, prefix=0, seed=0, scale=None, qscale=1.0, kind="tree",
        extra_words=0, **kw):
    pb = Paged(lens, ctx, prefix=prefix, kvh=kvh, dim=dim, dtype=dtype, seed=seed, **kw)
    spoil(pb)
    rng = rng_of(seed)
    if kind == "tree":
        seen = [closure(random_parents(n, rng)) if n else None for n in lens]
    elif kind == "any":                       # any mask, rows that see no new row among them
        seen = [torch.rand((n, n), generator=torch.Generator().manual_seed(seed + n)) <
                torch.linspace(0, 1, n)[torch.randperm(n, generator=torch.Generator().manual_seed(n))][:, None]
                if n else None for n in lens]
    else:
        seen = [causal(n) if n else None for n in lens]
    words = (max(lens) + 31) // 32 + extra_words
    mask = None if kind == "causal" else pack([m for m in seen if m is not None], pb.rows,
                                              [s for s, n in zip(pb.starts, lens) if n], words, fill=-1 if seed % 2 else 0)
    q, out, lse = attend(sess, pb, heads, mask, scale, qscale, strided=seed % 3 > 0, want_lse=seed % 4 > 0)
    close(pb, q, heads, out, lse, dim ** -0.5 if scale is None else scale, seen)
    return pb, q, out, lse, mask, seen


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("kind", ["tree", "any", "causal"])
@pytest.mark.parametrize("heads,kvh", [(1, 1), (8, 2), (5, 1), (128, 1), (21, 3)])
def test_head_layouts(sess, dtype, dim, kind, heads, kvh):
    run(sess, [1, 16, 0, 5], [0, 63, 9, 130], heads, kvh, dim, dtype, seed=heads, kind=kind)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("prefix", [0, 64, 192, 1024])
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_shared_prefix(sess, dtype, dim, prefix, kind):
    run(sess, [16, 3, 1, 0, 40], [0, 64, 127, 5, 300], 8, 2, dim, dtype, prefix=prefix, seed=prefix + 5, lead=1,
        trail=2, kind=kind)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("lens,ctx", [([1], [0]), ([2], [0]), ([32], [0]), ([33], [63]), ([64], [64]), ([65], [127]),
                                      ([129], [1]), ([300], [100]), ([31, 97], [95, 33]), ([1, 1], [2000, 0])])
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_lengths(sess, dtype, dim, lens, ctx, kind):
    run(sess, lens, ctx, 4, 1, dim, dtype, seed=sum(lens) + sum(ctx), kind=kind, extra_words=sum(lens) % 2)


@pytest.mark.parametrize("lens,ctx,heads,kvh,prefix", [
    ([1000, 257, 64], [0, 1000, 31], 8, 2, 0),         # the largest trees: masks of 32 words, split keys
    ([90, 33], [500, 3], 16, 1, 640),                  # row tiles that cross requests in the prefix
    ([64], [20000], 8, 8, 0),                          # one long context: keys split over the GPU
    ([24] * 50, list(range(0, 1000, 20)), 8, 1, 256),
])
@pytest.mark.parametrize("kind", ["tree", "any", "causal"])
def test_large(sess, lens, ctx, heads, kvh, prefix, kind):
    run(sess, lens, ctx, heads, kvh, 128, BF, prefix=prefix, seed=len(lens), kind=kind)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("scale,qscale", [(1.0, 3.0), (0.0, 1.0), (-0.3, 2.0), (20.0, 4.0)])
def test_scales_and_peaks(sess, dtype, dim, scale, qscale):
    run(sess, [17, 40], [400, 0], 4, 2, dim, dtype, prefix=128, scale=scale, qscale=qscale, seed=5)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ctx,prefix", [(0, 0), (100, 0), (1000, 128)])
def test_rows_that_are_not_finite_reach_only_those_that_see_them(sess, dtype, dim, what, ctx, prefix):
    lens, heads = [40, 12], 8
    for part in ("k", "v", "kv"):
        pb = Paged(lens, [ctx, 30], prefix=prefix, kvh=2, dim=dim, dtype=dtype, seed=3)
        spoil(pb)
        rng = rng_of(11)
        seen = [closure(random_parents(n, rng)) for n in lens]
        hurt = [7, 23, 39]
        pages, rows = pb.slots(0, prefix + ctx, prefix + ctx + 40)
        for r in hurt:
            if "k" in part:
                pb.k[pages[r], rows[r]] = what
            if "v" in part:
                pb.v[pages[r], rows[r], :, ::9] = what
        q, out, lse = attend(sess, pb, heads, pack(seen, pb.rows, pb.starts, 2), strided=False)
        sees = seen[0][:, hurt].any(1)
        ok = (~sees).nonzero()[:, 0].tolist()
        assert len(ok) > 5 and bool(sees.any())
        res = attend_tree64(pb, q, heads, dim ** -0.5, [torch.where(sees[:, None], False, seen[0]), seen[1]])
        half = torch.finfo(dtype).eps / 2
        for t in ok + list(range(40, 52)):
            want, spread, mag, want_lse = res[t]
            ds = ((dim + 8) * 2.0 ** -24 * mag)[:, None]
            tol = half * want.abs() + (half * (dtype == BF) + 2 * ds + 2.0 ** -18) * spread * (1 + half)
            assert bool(((out[t].double() - want).abs() <= tol).all()), t
            assert bool(((lse[t].double() - want_lse).abs() <= ds[:, 0] + 2.0 ** -18 + 2.0 ** -22 * want_lse.abs()).all())
        if part == "v" and what != what:
            for t in sees.nonzero()[:, 0].tolist():
                assert bool(out[t, :, ::9].isnan().all())


@pytest.mark.parametrize("dtype,dim", KINDS)
def test_rows_that_see_nothing(sess, dtype, dim):
    """No cache before them, and a mask without bits: zeros, and a sum whose log is -infinity."""
    pb = Paged([3, 70, 1], [0, 0, 0], kvh=2, dim=dim, dtype=dtype, seed=2)
    spoil(pb)
    seen = [torch.zeros((3, 3), dtype=torch.bool), torch.eye(70, dtype=torch.bool),
            torch.zeros((1, 1), dtype=torch.bool)]
    seen[1][5] = False
    q, out, lse = attend(sess, pb, 4, pack(seen, pb.rows, pb.starts, 3), strided=False)
    close(pb, q, 4, out, lse, dim ** -0.5, seen)
    for t in (0, 1, 2, 8, 73):
        assert bool((out[t] == 0).all()) and bool((lse[t] == -torch.inf).all())


@pytest.mark.parametrize("dtype,dim", KINDS)
def test_without_a_mask_it_is_the_paged_attention(sess, dtype, dim):
    pb, q, out, lse, _, _ = run(sess, [30, 200], [77, 300], 8, 2, dim, dtype, prefix=64, seed=6, kind="causal")
    lay = pb.layer(8)
    ws = sess.attention_workspace(lay, 2, pb.rows)
    ref = torch.full(out.shape, FILL, dtype=dtype, device="cuda")
    sess.paged_attention(lay, q.contiguous(), pb.row_start, pb.kv_len, ref, ws)
    # fp32: the same arithmetic; bf16: a row's sum is of two threads here, of one there, so the results are
    # two roundings of values 2^-22 apart, both held to the 64-bit ones
    if dtype == F32:
        assert torch.equal(ref, out)
    else:
        close(pb, q, 8, ref, None, dim ** -0.5, [causal(30), causal(200)])
        assert bool(((ref.double() - out.double()).abs() <= 2.0 ** -7 * ref.double().abs() + 2.0 ** -18).all())


def test_a_tree_that_is_a_chain_is_causal(sess):
    pb = Paged([50, 20], [200, 64], kvh=2, dim=128, seed=8)
    seen = [causal(50), causal(20)]
    q, out, lse = attend(sess, pb, 8, pack(seen, pb.rows, pb.starts, 2), strided=False)
    lay = pb.layer(8)
    ref, ref_lse = torch.empty_like(out), torch.empty_like(lse)
    sess.tree_attention(lay, q, pb.row_start, pb.kv_len, ref, sess.attention_workspace(lay, 2, pb.rows), lse=ref_lse)
    close(pb, q, 8, ref, ref_lse, 128 ** -0.5, seen)
    close(pb, q, 8, out, lse, 128 ** -0.5, seen)


def test_bad_pages_and_lengths(sess):
    for dt in (BF, F32):
        pb = Paged([4, 4, 4], [100, 100, 100], kvh=1, dim=64, dtype=dt, seed=1)
        pb.table[1, 0] = 10 ** 6               # read as page 0, flagged
        pb.kv_len[2] = 64 * pb.width - 3       # one row too many
        seen = [causal(4)] * 3
        q, out, lse = attend(sess, pb, 2, pack(seen, 12, pb.starts, 1), strided=False, check_error=False)
        assert set(pkg.decode_error(sess.error())) == {"PAGE_RANGE", "KV_CAPACITY"}
        assert bool((out[8:] == FILL).all()) and bool((lse[8:] == FILL).all())
        pb.kv_len[1], pb.lens, pb.ctx = 0, [4, 0, 0], [100, 0, 0]
        res = attend_tree64(pb, q, 2, 64 ** -0.5, seen)
        assert all(float((out[t].double() - res[t][0]).abs().max()) < 0.05 for t in range(4))


# ---------------------------------------------------------------- the walk
FILL_I = -9


def accept(sess, lens, par, tok, post, most, seq=None, ids=None, lead=0, weight=None):
    B = len(lens)
    full = lambda *s: torch.full(s, FILL_I, dtype=torch.int32, device="cuda")  # noqa: E731
    got = {"accept_len": full(B), "commit_len": full(B), "bonus": full(B), "out_tokens": full(B, most),
           "path": full(B, most)}
    got["seq_len"] = i32(seq if seq is not None else [10 * b for b in range(B)])
    sess.accept_tree(i32(starts_of(lens, lead)), i32(par), i32(tok), i32(post), got["seq_len"], got["accept_len"],
                     got["commit_len"], got["bonus"], got["out_tokens"], got["path"], output_ids=ids,
                     row_weight=weight)
    return got


@pytest.mark.parametrize("lens,most", [([1], 1), ([1, 0, 2], 4), ([64], 8), ([33, 200, 1, 7], 64), ([1024, 1000], 1024),
                                       ([16] * 130, 5)])
@pytest.mark.parametrize("few", [2, 5, 200])
def test_walk(sess, lens, most, few):
    rng = rng_of(sum(lens) + few)
    lead, par, tok, post, want, weight = 3, [], [], [], [], []
    for n in lens:
        p = random_parents(n, rng, back=rng.choice([1, 3, 9])) if n else []
        t = [rng.randrange(few) for _ in range(n)]              # few tokens: equal children among them
        y = [rng.randrange(few) for _ in range(n)]
        if few == 200:                                          # mostly right
            for i in range(1, n):
                if rng.random() < 0.9:
                    y[p[i]] = t[i]
        par, tok, post = par + p, tok + t, post + y
        path = walk(p, t, y, most) if n else None
        want.append((path, t, y))
        weight += [1.0 if path and i in set(path) else 0.0 for i in range(n)]
    pad = [5] * lead
    T = lead + sum(lens)
    w = torch.full((T,), FILL, device="cuda")
    ids = torch.full((len(lens), 10 * len(lens) + 1100), FILL_I, dtype=torch.int32, device="cuda")
    got = accept(sess, lens, pad + par, pad + tok, pad + post, most, ids=ids, lead=lead, weight=w)
    assert sess.error() == 0
    for b, (path, t, y) in enumerate(want):
        if path is None:
            assert int(got["commit_len"][b]) == FILL_I and int(got["seq_len"][b]) == 10 * b
            continue
        c = len(path)
        bonus = y[path[-1]]
        assert got["path"][b].tolist() == path + [-1] * (most - c)
        assert got["out_tokens"][b].tolist() == [t[r] for r in path[1:]] + [bonus] + [0] * (most - c)
        assert [int(got[k][b]) for k in ("accept_len", "commit_len", "bonus", "seq_len")] == \
            [c - 1, c, bonus, 10 * b + c]
        row = [FILL_I] * ids.shape[1]
        row[10 * b:10 * b + c + 1] = [t[r] for r in path] + [bonus]
        assert ids[b].tolist() == row
    assert w.tolist() == [FILL] * lead + weight


def test_a_chain_commits_what_the_block_would(sess):
    """A tree without branches against dflash_accept_commit."""
    S, B = 2, 4
    tok = [[5, 7], [5, 7], [3, 3], [0, 255]]
    post = [[7, 9], [8, 9], [3, 3], [255, 0]]
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    ref = {"seq_len": i32([0, 10, 20, 30]), "accept_len": z(B), "commit_len": z(B), "bonus": z(B), "out_tokens": z(B, S)}
    sess.accept(B, i32(tok), i32(post), ref["seq_len"], ref["accept_len"], ref["commit_len"], ref["bonus"],
                ref["out_tokens"])
    flat = lambda x: [v for r in x for v in r]  # noqa: E731
    got = accept(sess, [S] * B, [-1, 0] * B, flat(tok), flat(post), S)
    assert sess.error() == 0
    for k, v in ref.items():
        assert torch.equal(v, got[k]), k


def test_walk_refuses_ids_and_rows_out_of_range(sess):
    ids = torch.full((3, 12), FILL_I, dtype=torch.int32, device="cuda")
    # a bonus outside the vocabulary; a wrong id off the path; a commit past the row's end
    got = accept(sess, [2, 3, 2], [-1, 0, -1, 0, 0, -1, 0], [1, 2, 1, 999, 3, 1, 2], [2, VOCAB, 3, 0, 4, 2, 4], 4,
                 seq=[0, 4, 10], ids=ids)
    assert set(pkg.decode_error(sess.error())) == {"TOKEN_RANGE", "OUTPUT_ROW"}
    assert got["commit_len"].tolist() == [FILL_I, 2, FILL_I]
    assert got["seq_len"].tolist() == [0, 6, 10]
    assert ids[1].tolist() == [FILL_I] * 4 + [1, 3, 4] + [FILL_I] * 5
    assert bool((ids[0] == FILL_I).all()) and bool((ids[2] == FILL_I).all())
    got = accept(sess, [1025], [-1] + [0] * 1024, [1] * 1025, [1] * 1025, 4)
    assert pkg.decode_error(sess.error()) == ["TREE"] and got["commit_len"].tolist() == [FILL_I]
    # rows -1..0, and rows 1..2, whose first has a parent
    got = accept(sess, [2, 2], [-1, 0, -1, 0], [1] * 4, [1] * 4, 4, lead=-1)
    assert pkg.decode_error(sess.error()) == ["ROW_RANGE", "TREE"]
    assert got["commit_len"].tolist() == [FILL_I, FILL_I]
    got = accept(sess, [2, 2], [0, -1, 0, 0], [1] * 4, [1] * 4, 4, lead=-1)
    assert pkg.decode_error(sess.error()) == ["ROW_RANGE"] and got["commit_len"].tolist() == [FILL_I, 2]
