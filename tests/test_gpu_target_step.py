"""The target's side of a cycle as it is used: two layers of append and attention over a verify
block that shares a prefix, logits, the sampling distribution, then the sampled verification on it
-- eager and as one captured graph, against the plain 64-bit forms and the oracle's acceptance."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_diffusion_speculative_fc_gb300 as pkg  # noqa: E402
from oracle import dflash_oracle as O  # noqa: E402
from tests.target_reference import Paged, attend64, i32, make_session, norm64, rope64, sample64  # noqa: E402

B, S, H, KVH, D, V, PREFIX, LAYERS = 5, 8, 8, 2, 128, 512, 128, 2
BF = torch.bfloat16


@pytest.fixture(scope="module")
def sess():
    s = make_session(block=S, vocab=V, max_batch=B)
    yield s
    s.close()


class Step:
    """The buffers of one verification step and its calls."""

    def __init__(self, sess):
        self.sess = sess
        self.pb = [Paged([S] * B, [0, 63, 200, 64, 700], prefix=PREFIX, kvh=KVH, dim=D, seed=7 + i)
                   for i in range(LAYERS)]
        g = self.pb[0].g
        W = (H + 2 * KVH) * D
        n = lambda *s, scale=1.0: (torch.randn(s, generator=g, device="cuda") * scale).to(BF)  # noqa: E731
        self.x = n(B * S, 256)
        self.w_in = [n(256 if i == 0 else H * D, W, scale=0.06 if i == 0 else 0.03) for i in range(LAYERS)]
        self.head = n(H * D, V, scale=0.25)
        self.gain = [(0.5 + torch.rand(D, generator=g, device="cuda")).to(BF) for _ in range(LAYERS)]
        self.plan = pkg.rope_plan(D, 1e6, scaling="yarn", factor=4, original_positions=4096)
        self.layers = [p.layer(H) for p in self.pb]
        self.ws = sess.attention_workspace(self.layers[0], B, B * S)
        z = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.q = [z(B * S, H, D) for _ in range(LAYERS)]
        self.out = [z(B * S, H, D) for _ in range(LAYERS)]
        self.qkv = [z(B * S, W) for _ in range(LAYERS)]
        self.logits, self.probs = z(B, S, V), z(B, S, V, dt=torch.float32)
        self.draft = torch.randint(0, V, (B, S), generator=g, device="cuda", dtype=torch.int32)
        self.params = dict(temperature=torch.tensor([1.0, 0.7, 0.0, 2.0, 1.0], device="cuda"),
                           top_k=i32([0, 40, 0, 0, 300]),
                           top_p=torch.tensor([1.0, 0.9, 1.0, 0.98, 0.9], device="cuda"),
                           min_p=torch.tensor([0.0, 0.0, 0.0, 0.01, 0.0], device="cuda"))
        self.u = torch.rand((B, S - 1), generator=g, device="cuda") * 0.02
        self.noise = torch.empty((B, V), device="cuda").exponential_(generator=g).clamp_(min=1e-30)
        zi = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.seq, self.acc, self.com, self.bon, self.tok = zi(B), zi(B), zi(B), zi(B), zi(B, S)
        self.first, self.first_noise = zi(B, S), torch.ones((B, S, V), device="cuda")

    def calls(self):
        x = self.x
        for i in range(LAYERS):
            torch.matmul(x, self.w_in[i], out=self.qkv[i])
            q, k, v = (t.unflatten(1, (-1, D)) for t in
                       self.qkv[i].split([H * D, KVH * D, KVH * D], dim=1))
            pb = self.pb[i]
            self.sess.append_kv(self.layers[i], q, k, v, pb.row_start, pb.kv_len, self.plan,
                                q_gain=self.gain[i], k_gain=self.gain[i], q_out=self.q[i])
            self.sess.paged_attention(self.layers[i], self.q[i], pb.row_start, pb.kv_len, self.out[i],
                                      self.ws)
            x = self.out[i].view(B * S, H * D)
        torch.matmul(x, self.head, out=self.logits.view(B * S, V))
        self.sess.target_probs(self.logits, self.probs, **self.params)
        self.sess.sample_tokens(self.logits, self.first_noise, self.first, **self.params)
        self.seq.zero_()
        self.sess.accept_sampled(B, self.draft, self.probs, self.u, self.noise, self.seq, self.acc,
                                 self.com, self.bon, self.tok)

    def verify(self):
        """Every call against its plain form on the inputs that it got."""
        eps = 2.0 ** -8
        inv = torch.tensor([t / 2.0 ** 64 * 2 * np.pi for t in self.plan.turns[:D // 2]],
                           dtype=torch.float64, device="cuda")
        for i, pb in enumerate(self.pb):
            q, k, v = (t.unflatten(1, (-1, D)) for t in
                       self.qkv[i].split([H * D, KVH * D, KVH * D], dim=1))
            for b in range(B):
                rows, first = slice(b * S, b * S + S), PREFIX + pb.ctx[b]
                pos = torch.arange(first, first + S, device="cuda")
                at = pb.slots(b, first, first + S)
                for src, got in ((q[rows], self.q[i][rows]), (k[rows], pb.k[at])):
                    y, big = rope64(norm64(src, self.gain[i], 1e-6), pos, inv, self.plan.amplitude, 0)
                    assert bool(((got.double() - y).abs() <= eps * y.abs() + 2.0 ** -18 * big).all())
                assert torch.equal(pb.v[at], v[rows])
            for t, (want, spread, mag) in attend64(pb, self.q[i], H, D ** -0.5, True).items():
                tol = eps * want.abs() + (eps + 2 * (D + 8) * 2.0 ** -24 * mag[:, None] + 2.0 ** -18) * spread * (1 + eps)
                assert bool(((self.out[i][t].double() - want).abs() <= tol).all()), (i, t)
        P = {k: v.tolist() for k, v in self.params.items()}
        for b in range(B):
            for s in range(S):
                w, a, near = sample64(self.logits[b, s], P["temperature"][b], P["top_k"][b],
                                      P["top_p"][b], P["min_p"][b])
                if near < 2.0 ** -26:
                    continue
                want = w / w.sum()
                tol = want * (3 * a * 2.0 ** -24 + 2.0 ** -21 + 100 * 2.0 ** -24) + 2.0 ** -126
                assert bool(((self.probs[b, s].double() - want).abs() <= tol).all()), (b, s)
                # all variates 1: the largest weight, lowest id on ties
                assert int(self.first[b, s]) == int(w.argmax())
            acc, bonus, commit, toks = O.accept_block_sampled(
                self.draft[b].cpu().numpy(), self.probs[b].cpu().numpy(), self.u[b].cpu().numpy(),
                self.noise[b].cpu().numpy())
            assert (int(self.acc[b]), int(self.bon[b]), int(self.com[b])) == (acc, bonus, commit)
            assert np.array_equal(self.tok[b].cpu().numpy(), toks)


def test_eager_then_captured(sess):
    st = Step(sess)
    st.calls()
    assert sess.error() == 0
    st.verify()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.calls()
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        st.x.copy_(torch.randn(st.x.shape, generator=gen, device="cuda"))
        # the accepted rows of the step before are context now
        for pb in st.pb:
            pb.ctx = [min(c + int(n), 64 * len(pb.lists[b]) - S) for b, (c, n) in
                      enumerate(zip(pb.ctx, st.com.tolist()))]
            pb.kv_len.copy_(i32([PREFIX + c for c in pb.ctx]))
        g.replay()
        torch.cuda.synchronize()
        st.verify()
    assert sess.error() == 0


def test_per_kernel_timing_names_the_calls(sess):
    st = Step(sess)
    pkg.dflash_profile_enable(sess.h, 32)
    st.calls()
    got = pkg.dflash_profile_collect(sess.h)
    pkg.dflash_profile_disable(sess.h)
    for name, n in (("append_kv", LAYERS), ("paged_attention", LAYERS), ("target_probs", 1),
                    ("sample_tokens", 1)):
        assert got[name][0] == n and got[name][1] > 0
