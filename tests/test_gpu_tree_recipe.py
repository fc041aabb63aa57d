"""The README's lines for a tree of drafted tokens, run as they stand there over buffers that are used again
from step to step, with a request that has no rows in the second step and one that is refused."""
import os
import re

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_diffusion_speculative_fc_gb300 as pkg  # noqa: E402
from tests.target_reference import Paged, i32, make_session  # noqa: E402

V, H, KVH, PREFIX, WORDS, MOST, ROOM, KEPT = 64, 8, 2, 64, 1, 8, 60, 400
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
PARENT = [-1, 0, 0, 2, 2, 4, 4]                 # the target's tokens lead over rows 0, 2, 4, 6
CTX = [70, 33, 200, 5]
z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731


def lines():
    with open(README) as f:
        text = f.read()
    return re.search(r"A tree of drafted tokens, and a cache kept to a budget:\n\n```python\n(.*?)```", text, re.S).group(1)


def path_of(n):
    return [r for r in (0, 2, 4, 6) if r < n]


@pytest.fixture(scope="module")
def sess():
    s = make_session(vocab=V)
    yield s
    s.close()


@pytest.mark.parametrize("dtype,dim", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_requests_that_commit_nothing_keep_their_cache(sess, dtype, dim):
    B = len(CTX)
    pb = Paged([ROOM] * B, CTX, prefix=PREFIX, kvh=KVH, dim=dim, dtype=dtype, seed=5)
    layer = pb.layer(H)
    # what lives from step to step
    env = dict(sess=sess, layer=layer, rope=pkg.rope_plan(dim, 1e6), prefix_len=PREFIX, kv_len=pb.kv_len,
               position=pb.kv_len.clone(), seq_len=z(B), accept_len=z(B), commit_len=z(B), bonus=z(B),
               out_tokens=z(B, MOST), path=z(B, MOST), budget=i32([KEPT] * B), rows=z(B, KVH, KEPT), count=z(B, KVH),
               weights=torch.rand((B, KVH, max(CTX) + ROOM), generator=pb.g, device="cuda"))
    on_path = z(64, dt=torch.float32)
    kv_len, weights = env["kv_len"], env["weights"]

    def step(lens, refused=()):
        T, starts = sum(lens), [sum(lens[:b]) for b in range(B + 1)]
        post = [[30, 30, 30, 30, 30, 30, 30][:n] for n in lens]
        for b, n in enumerate(lens):
            for r, child in ((0, 2), (2, 4), (4, 6)):
                if child < n:
                    post[b][r] = child + 1      # row i's token is i + 1
            if b in refused:
                post[b][0] = V                  # no token of the vocabulary
        env.update(row_start=i32(starts), parent=i32([p for n in lens for p in PARENT[:n]]),
                   tokens=i32([i + 1 for n in lens for i in range(n)]), target_ids=i32([t for p in post for t in p]),
                   mask=z(T, WORDS), positions=z(T), q=pb.normal(T, H, dim), k=pb.normal(T, KVH, dim),
                   v=pb.normal(T, KVH, dim), out=z(T, H, dim, dt=dtype), lse=z(T, H, dt=torch.float32),
                   on_path=on_path[:T], ws=sess.attention_workspace(layer, B, T))
        exec(lines(), env)

    step([7, 5, 6, 1])
    assert sess.error() == 0
    assert env["commit_len"].tolist() == [4, 3, 3, 1]
    assert kv_len.tolist() == [PREFIX + c + n for c, n in zip(CTX, (4, 3, 3, 1))]
    before = kv_len.tolist()
    k0, v0, w0, pos0 = pb.k.clone(), pb.v.clone(), weights.clone(), env["position"].tolist()
    step([6, 0, 7, 1], refused=[2])
    assert pkg.decode_error(sess.error()) == ["TOKEN_RANGE"]
    # the request without rows: every row of its pages, committed or not, and its weights
    pages, rows = pb.slots(1, PREFIX, PREFIX + CTX[1] + ROOM)
    assert torch.equal(pb.k[pages, rows], k0[pages, rows]) and torch.equal(pb.v[pages, rows], v0[pages, rows])
    assert torch.equal(weights[1], w0[1])
    # the refused one: its committed rows; no row of the step counts for their weights, which decay; behind them
    # stand the step's rows where they were appended
    own = before[2] - PREFIX
    pages, rows = pb.slots(2, PREFIX, before[2])
    assert torch.equal(pb.k[pages, rows], k0[pages, rows]) and torch.equal(pb.v[pages, rows], v0[pages, rows])
    assert bool(((weights[2, :, :own] - 0.99 * w0[2, :, :own]).abs() <= 2.0 ** -22 * w0[2, :, :own]).all())
    pages, rows = pb.slots(2, before[2], before[2] + 7)
    assert torch.equal(pb.v[pages, rows], env["v"][6:13])
    grown = [len(path_of(6)), 0, 0, 1]
    assert kv_len.tolist() == [a + n for a, n in zip(before, grown)]
    assert env["position"].tolist() == [a + n for a, n in zip(pos0, grown)]
    # and a step after it serves them as before
    before = kv_len.tolist()
    step([1, 7, 7, 0])
    assert sess.error() == 0
    assert kv_len.tolist() == [a + n for a, n in zip(before, [1, 4, 4, 0])]
