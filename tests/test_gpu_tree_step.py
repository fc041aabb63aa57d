"""Tree verification and eviction as they are used: two layers of append at the rows' depths, attention
under the trees' masks and the weights of the cached rows, tokens for every row, the walk, the accepted rows
moved together; then the caches cut to a budget, and a step on what is left -- eager and as captured graphs,
against the plain 64-bit forms."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_diffusion_speculative_fc_gb300 as pkg  # noqa: E402
from tests.target_reference import Paged, i32, make_session, norm64, rope64  # noqa: E402
from tests.tree_reference import (attend_tree64, choose, closure, pack, random_parents, rng_of, walk,  # noqa: E402
                                  weights64)

N, H, KVH, D, V, PREFIX, LAYERS, WORDS = [20, 33, 1, 12, 40], 8, 2, 128, 32, 128, 2, 2
B, T, MOST = len(N), sum(N), 16
BF = torch.bfloat16
z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731


@pytest.fixture(scope="module")
def sess():
    s = make_session(vocab=V)
    yield s
    s.close()


class Step:
    def __init__(self, sess, ctx):
        self.sess = sess
        # (rooms for 60 more rows behind the trees)
        self.pb = [Paged([n + 60 for n in N], ctx, prefix=PREFIX, kvh=KVH, dim=D, seed=7 + i) for i in range(LAYERS)]
        g = self.pb[0].g
        n = lambda *s, scale=1.0: (torch.randn(s, generator=g, device="cuda") * scale).to(BF)  # noqa: E731
        self.width = max(c + m + 60 for c, m in zip(ctx, N))
        self.starts = [sum(N[:b]) for b in range(B + 1)]
        self.row_start, self.kv_len = i32(self.starts), i32([PREFIX + c for c in ctx])
        self.position = i32([PREFIX + c + 1000 * b for b, c in enumerate(ctx)])     # rows have been evicted before
        self.qkv = [n(T, (H + 2 * KVH) * D) for _ in range(LAYERS)]
        self.head = n(H * D, V, scale=0.3)
        self.gain = [(0.5 + torch.rand(D, generator=g, device="cuda")).to(BF) for _ in range(LAYERS)]
        self.plan = pkg.rope_plan(D, 1e6)
        for pb in self.pb:
            pb.lens, pb.starts, pb.row_start, pb.kv_len = list(N), self.starts, self.row_start, self.kv_len
        self.layers = [p.layer(H) for p in self.pb]
        self.ws = sess.attention_workspace(self.layers[0], B, T)
        self.parent, self.tokens, self.post = z(T), z(T), z(T)
        self.mask, self.pos = z(T, WORDS), z(T)
        self.q = [z(T, H, D, dt=BF) for _ in range(LAYERS)]
        self.out = [z(T, H, D, dt=BF) for _ in range(LAYERS)]
        self.lse = [z(T, H, dt=torch.float32) for _ in range(LAYERS)]
        self.weights = [torch.rand((B, KVH, self.width), generator=g, device="cuda") for _ in range(LAYERS)]
        self.logits, self.noise = z(T, V, dt=BF), torch.ones((T, V), device="cuda")
        self.seq, self.acc, self.com, self.bon = z(B), z(B), z(B), z(B)
        self.tok, self.path, self.rw = z(B, MOST), z(B, MOST), z(T, dt=torch.float32)
        self.new_tree(0)

    def new_tree(self, seed):
        rng = rng_of(seed)
        self.parents = [random_parents(n, rng) for n in N]
        self.parent.copy_(i32([p for t in self.parents for p in t]))
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.tokens.copy_(torch.randint(0, 3, (T,), generator=g, device="cuda", dtype=torch.int32))
        for x in self.qkv:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))

    def calls(self):
        s = self.sess
        s.tree_plan(self.row_start, self.parent, self.mask, self.pos, root=self.position)
        for i in range(LAYERS):
            q, k, v = (t.unflatten(1, (-1, D)) for t in self.qkv[i].split([H * D, KVH * D, KVH * D], dim=1))
            s.append_kv(self.layers[i], q, k, v, self.row_start, self.kv_len, self.plan, q_gain=self.gain[i],
                        k_gain=self.gain[i], q_out=self.q[i], positions=self.pos)
            s.tree_attention(self.layers[i], self.q[i], self.row_start, self.kv_len, self.out[i], self.ws,
                             mask=self.mask, lse=self.lse[i])
        torch.matmul(self.out[-1].view(T, H * D), self.head, out=self.logits)
        self.logits[:, 3:].fill_(-100.0)                     # three tokens: walks of some length
        s.sample_tokens(self.logits, self.noise, self.post)
        s.accept_tree(self.row_start, self.parent, self.tokens, self.post, self.seq, self.acc, self.com, self.bon,
                      self.tok, self.path, row_weight=self.rw)
        for i in range(LAYERS):
            s.key_weights(self.layers[i], self.q[i], self.row_start, self.kv_len, self.lse[i], self.weights[i],
                          mask=self.mask, row_weight=self.rw, decay=0.5)

    def commit(self):
        for i in range(LAYERS):
            self.sess.keep_rows(self.layers[i], self.path, self.com, first=self.kv_len, weights=self.weights[i])
        self.kv_len += self.com
        self.position += self.com

    def verify(self, old):
        """Every call against its plain form on the inputs that it got; returns what the commit leaves."""
        ctx = [int(k) - PREFIX for k in self.kv_len]
        seen = [closure(p) for p in self.parents]
        assert torch.equal(self.mask, pack(seen, T, self.starts, WORDS))
        depth = torch.cat([m.sum(1) - 1 for m in seen]).cuda()
        req = torch.repeat_interleave(torch.arange(B), torch.tensor(N)).cuda()
        assert torch.equal(self.pos.long(), self.position.long()[req] + depth)
        inv = torch.tensor([t / 2.0 ** 64 * 2 * torch.pi for t in self.plan.turns[:D // 2]], dtype=torch.float64,
                           device="cuda")
        eps = 2.0 ** -8
        for i, pb in enumerate(self.pb):
            pb.ctx = ctx
            q, k, v = (t.unflatten(1, (-1, D)) for t in self.qkv[i].split([H * D, KVH * D, KVH * D], dim=1))
            for b in range(B):
                rows, first = slice(self.starts[b], self.starts[b + 1]), PREFIX + ctx[b]
                at = pb.slots(b, first, first + N[b])
                for src, got in ((q[rows], self.q[i][rows]), (k[rows], pb.k[at])):
                    y, big = rope64(norm64(src, self.gain[i], 1e-6), self.pos[rows], inv, 1.0, 0)
                    assert bool(((got.double() - y).abs() <= eps * y.abs() + 2.0 ** -18 * big).all())
                assert torch.equal(pb.v[at], v[rows])
            for t, (want, spread, mag, lse) in attend_tree64(pb, self.q[i], H, D ** -0.5, seen).items():
                ds = 2 * (D + 8) * 2.0 ** -24 * mag[:, None]
                tol = eps * want.abs() + (eps + ds + 2.0 ** -18) * spread * (1 + eps)
                assert bool(((self.out[i][t].double() - want).abs() <= tol).all()), (i, t)
                assert bool(((self.lse[i][t].double() - lse).abs() <= ds[:, 0] + 2.0 ** -18 + 2.0 ** -22 * lse.abs()).all())
            want, tol, live = weights64(pb, self.q[i], H, D ** -0.5, seen, self.lse[i], self.rw, 0.5, old[i])
            at = live[:, None].expand_as(want)
            assert bool(((self.weights[i].double() - want).abs() <= tol)[at].all())
        assert torch.equal(self.post, self.logits.argmax(-1).int())
        tok, post = self.tokens.tolist(), self.post.tolist()
        paths = []
        for b in range(B):
            rows = slice(self.starts[b], self.starts[b + 1])
            paths.append(walk(self.parents[b], tok[rows], post[rows], MOST))
            assert self.path[b, :int(self.com[b])].tolist() == paths[b] and int(self.com[b]) == len(paths[b])
            assert int(self.bon[b]) == post[rows][paths[b][-1]]
            assert self.rw[rows].nonzero()[:, 0].tolist() == paths[b]
        return ctx, paths

    def snapshot(self):
        return [(pb.k.clone(), pb.v.clone(), w.clone()) for pb, w in zip(self.pb, self.weights)]

    def verify_moved(self, before, first, lists):
        """lists[b]: one list, or one a head; first[b]: own row that they count from."""
        for pb, w, (k, v, w0) in zip(self.pb, self.weights, before):
            for b in range(B):
                pages, at = pb.slots(b, 0, PREFIX + 64 * len(pb.lists[b]))
                for h in range(KVH):
                    rows = lists[b][h] if lists[b] and isinstance(lists[b][0], list) else lists[b]
                    for i, r in enumerate(rows):
                        s, d = PREFIX + first[b] + r, PREFIX + first[b] + i
                        assert torch.equal(pb.k[pages[d], at[d], h], k[pages[s], at[s], h])
                        assert torch.equal(pb.v[pages[d], at[d], h], v[pages[s], at[s], h])
                    assert torch.equal(w[b, h, first[b]:first[b] + len(rows)], w0[b, h, [first[b] + r for r in rows]])


def test_steps_then_eviction_then_a_step(sess):
    st = Step(sess, [0, 100, 300, 64, 700])
    old = [w.clone() for w in st.weights]
    st.calls()
    assert sess.error() == 0
    ctx, paths = st.verify(old)
    before = st.snapshot()
    st.commit()
    assert sess.error() == 0
    st.verify_moved(before, ctx, paths)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.calls()
    for seed in (1, 2):
        st.new_tree(seed)
        old = [w.clone() for w in st.weights]
        g.replay()
        torch.cuda.synchronize()
        ctx, paths = st.verify(old)
        before = st.snapshot()
        st.commit()
        st.verify_moved(before, ctx, paths)
    # cut to 90 rows a head: the first two, the last 16, the heaviest between
    keep, rows, count = i32([90] * B), z(B, KVH, 90), z(B, KVH)
    n = [int(k) - PREFIX for k in st.kv_len]
    before = st.snapshot()
    for i in range(LAYERS):
        sess.choose_rows(st.layers[i], st.weights[i], st.kv_len, keep, rows, count, first=2, last=16)
        lists = [[choose(before[i][2][b, h].tolist(), n[b], 90, 2, 16) for h in range(KVH)] for b in range(B)]
        for b in range(B):
            assert [rows[b, h, :int(count[b, h])].tolist() for h in range(KVH)] == lists[b]
        sess.keep_rows(st.layers[i], rows, count, weights=st.weights[i])
        pb, w = st.pb, st.weights
        st.pb, st.weights = pb[i:i + 1], w[i:i + 1]
        st.verify_moved(before[i:i + 1], [0] * B, lists)
        st.pb, st.weights = pb, w
    st.kv_len.copy_(PREFIX + count[:, 0])
    assert sess.error() == 0
    # the same graph on what is left
    st.new_tree(3)
    old = [w.clone() for w in st.weights]
    g.replay()
    torch.cuda.synchronize()
    st.verify(old)
    assert sess.error() == 0


def test_two_streams_with_their_own_workspaces(sess):
    """Steps of two batches side by side give what they give one after the other."""
    a, b = Step(sess, [0, 100, 300, 64, 700]), Step(sess, [10, 0, 64, 200, 90])
    b.new_tree(5)
    want = []
    for st in (a, b):
        st.saved = [w.clone() for w in st.weights]
        st.calls()
        torch.cuda.synchronize()
        want.append([x.clone() for x in st.out + st.lse + st.weights + [st.path, st.com]])
        for w, s in zip(st.weights, st.saved):
            w.copy_(s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st, s in zip((a, b), streams):
        with torch.cuda.stream(s):
            st.calls()
    torch.cuda.synchronize()
    for st, w in zip((a, b), want):
        for x, y in zip(st.out + st.lse + st.weights + [st.path, st.com], w):
            assert torch.equal(x, y)
    assert sess.error() == 0


def test_per_kernel_timing_names_the_calls(sess):
    st = Step(sess, [0, 100, 300, 64, 700])
    pkg.dflash_profile_enable(sess.h, 32)
    st.calls()
    st.commit()
    sess.choose_rows(st.layers[0], st.weights[0], st.kv_len, i32([9] * B), z(B, KVH, 9), z(B, KVH))
    got = pkg.dflash_profile_collect(sess.h)
    pkg.dflash_profile_disable(sess.h)
    for name, n in (("tree_plan", 1), ("append_kv", LAYERS), ("tree_attention", LAYERS), ("key_weights", LAYERS),
                    ("accept_tree", 1), ("keep_rows", LAYERS), ("choose_rows", 1)):
        assert got[name][0] == n and got[name][1] > 0


def test_the_session_refuses_wrong_tensors(sess):
    st = Step(sess, [0, 10, 5, 64, 7])
    lay = st.layers[0]
    att = dict(layer=lay, q=st.q[0], row_start=st.row_start, kv_len=st.kv_len, out=st.out[0], workspace=st.ws,
               mask=st.mask, lse=st.lse[0])
    wei = dict(layer=lay, q=st.q[0], row_start=st.row_start, kv_len=st.kv_len, lse=st.lse[0], weights=st.weights[0],
               mask=st.mask, row_weight=st.rw)
    acc = dict(row_start=st.row_start, parent=st.parent, tokens=st.tokens, posterior=st.post, seq_len=st.seq,
               accept_len=st.acc, commit_len=st.com, bonus=st.bon, out_tokens=st.tok, path=st.path, row_weight=st.rw)
    cho = dict(layer=lay, weights=st.weights[0], kv_len=st.kv_len, keep=i32([9] * B), rows=z(B, KVH, 9),
               count=z(B, KVH))
    kee = dict(layer=lay, rows=st.path, count=st.com, first=st.kv_len, weights=st.weights[0])
    pla = dict(row_start=st.row_start, parent=st.parent, mask=st.mask, positions=st.pos, root=st.position)
    for call, good, bad in [
        (sess.tree_attention, att, [dict(mask=st.mask[1:]), dict(mask=st.mask.float()), dict(lse=st.lse[0].half()),
                                    dict(lse=st.lse[0][:, :1]), dict(mask=st.mask.cpu()), dict(q=st.q[0].float())]),
        (sess.key_weights, wei, [dict(weights=st.weights[0][:1]), dict(weights=st.weights[0][:, :, ::2]),
                                 dict(row_weight=st.rw[1:]), dict(lse=st.lse[0][1:]), dict(mask=st.mask[:, 0])]),
        (sess.accept_tree, acc, [dict(path=st.path[1:]), dict(out_tokens=st.tok[:, 1:]), dict(tokens=st.tokens[1:]),
                                 dict(seq_len=st.seq.long()), dict(row_weight=st.rw.double()),
                                 dict(output_ids=z(B - 1, 9))]),
        (sess.choose_rows, cho, [dict(count=z(B, 1)), dict(rows=z(B, 9)), dict(keep=i32([9])),
                                 dict(weights=st.weights[0].half())]),
        (sess.keep_rows, kee, [dict(rows=st.path[:, None].expand(B, 3, MOST).contiguous()), dict(count=st.com[1:]),
                               dict(first=st.kv_len.long()), dict(weights=st.weights[0][1:]), dict(rows=z(B))]),
        (sess.tree_plan, pla, [dict(root=None), dict(root=z(B + 1)), dict(mask=z(T)), dict(parent=st.parent.long()),
                               dict(positions=z(T + 1))])]:
        call(**good)
        for b in bad:
            with pytest.raises(ValueError):
                call(**{**good, **b})
    sess.error()


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_pages_far_into_a_large_pool(sess, dtype):
    """Pages behind 2^32 elements of the pool give what the same pages at its start give: append, attention,
    weights, chosen and moved rows."""
    rows, heads, far = [20, 1, 33], 4, 2 ** 32 // (64 * KVH * D) + 5
    got = []
    for shift in (0, far):
        pb = Paged(rows, [300, 64, 5], prefix=64, kvh=KVH, dim=D, dtype=dtype, seed=3)
        n_pages, T = pb.n_pages, pb.rows
        if shift:
            small = (pb.k, pb.v)
            pb.k, pb.v = (torch.empty((far + n_pages, 64, KVH, D), dtype=dtype, device="cuda") for _ in "kv")
            pb.k[far:], pb.v[far:] = small
            pb.table += far
            pb.prefix_pages += far
        lay, q, k, v = pb.layer(heads), pb.normal(T, heads, D), pb.normal(T, KVH, D), pb.normal(T, KVH, D)
        parent = i32([p for n in rows for p in random_parents(n, rng_of(n))])
        mask, pos = z(T, WORDS), z(T)
        sess.tree_plan(pb.row_start, parent, mask, pos, root=pb.kv_len)
        sess.append_kv(lay, q, k, v, pb.row_start, pb.kv_len, pkg.rope_plan(D, 1e6), q_out=q, positions=pos)
        out, lse = torch.zeros_like(q), z(T, heads, dt=torch.float32)
        sess.tree_attention(lay, q, pb.row_start, pb.kv_len, out, sess.attention_workspace(lay, 3, T), mask=mask, lse=lse)
        weights = z(3, KVH, 64 * pb.width, dt=torch.float32)
        sess.key_weights(lay, q, pb.row_start, pb.kv_len, lse, weights, mask=mask)
        keep, count = z(3, KVH, 40), z(3, KVH)
        sess.choose_rows(lay, weights, pb.kv_len, i32([40, 30, 5]), keep, count, first=2, last=3)
        sess.keep_rows(lay, keep, count, weights=weights)
        assert sess.error() == 0
        got.append([out, lse, weights, keep, count, pb.k[shift:].clone(), pb.v[shift:].clone()])
        del lay, pb
    for x, y in zip(*got):
        assert torch.equal(x, y)
