"""Head norms, rotary positions and the cache append against their plain 64-bit form.

Tolerance, element by element: one rounding to the storage type (finfo.eps / 2 of the value), and
the fp32 arithmetic before it.  That is: the mean square, rsqrt and the gain (below 140 roundings of
2^-24 in all, most of them averaged in the sum of up to 128 squares: 2^-20 covers the worst case of
a chunked sum), sin and cos (angle cut to 2^-25 half turns, a few units of 2^-24 in the functions:
below 2^-21 absolute), two products and a sum -- each relative to |a| + |b| of the pair.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_diffusion_speculative_fc_gb300 as pkg  # noqa: E402
from tests.target_reference import PAGE, Paged, i32, make_session, norm64, rope64  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
FILL = -7.0


@pytest.fixture(scope="module")
def sess():
    s = make_session()
    yield s
    s.close()


def frequencies(plan):
    n = plan.rotary_dim // 2
    t = torch.tensor([x / 2.0 ** 64 for x in plan.turns[:n]], dtype=torch.float64, device="cuda")
    return t * (2 * torch.pi)


def close(got, want, big, dtype, name):
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -18 * big
    over = (got.double() - want).abs() - tol
    assert float(over.max()) <= 0, (name, float(over.max()))


def check(pb, heads, plan, q, k, v, qg, kg, eps, q_out, rows_of_requests=None):
    """Every owned row against the plain form; every other row of q_out and cell of the pools as it was."""
    inv, dt = frequencies(plan), pb.dtype
    touched = torch.zeros((pb.n_pages, PAGE), dtype=torch.bool, device="cuda")
    owned = torch.zeros(pb.rows, dtype=torch.bool, device="cuda")
    for b, n in enumerate(pb.lens):
        if n == 0 or (rows_of_requests is not None and b not in rows_of_requests):
            continue
        first = pb.prefix + pb.ctx[b]
        pos = torch.arange(first, first + n, device="cuda")
        rows = slice(pb.starts[b], pb.starts[b] + n)
        owned[rows] = True
        pages, at = pb.slots(b, first, first + n)
        touched[pages, at] = True
        if q is not None:
            y, big = rope64(norm64(q[rows], qg, eps), pos, inv, plan.amplitude, plan.interleaved)
            close(q_out[rows], y, big, dt, "q")
        y, big = rope64(norm64(k[rows], kg, eps), pos, inv, plan.amplitude, plan.interleaved)
        close(pb.k[pages, at], y, big, dt, "k")
        assert torch.equal(pb.v[pages, at], v[rows])
    if q is not None:
        assert bool((q_out[~owned] == FILL).all())
    assert bool((pb.k[~touched] == FILL).all()) and bool((pb.v[~touched] == FILL).all())


def run(sess, pb, heads, plan, norm=True, packed=False, inplace=False, with_q=True, eps=1e-6):
    kvh, D, T, dt = pb.kvh, pb.dim, pb.rows, pb.dtype
    if packed:
        parts = pb.normal(T, (heads + 2 * kvh) * D).split([heads * D, kvh * D, kvh * D], dim=1)
        q, k, v = (t.unflatten(1, (-1, D)) for t in parts)
    else:
        q, k, v = pb.normal(T, heads, D), pb.normal(T, kvh, D), pb.normal(T, kvh, D)
    gain = lambda: (0.5 + torch.rand(D, generator=pb.g, device="cuda")).to(dt)  # noqa: E731
    qg, kg = (gain(), gain()) if norm else (None, None)
    q0 = q.clone()
    q_out = q if inplace else torch.full((T, heads, D), FILL, dtype=dt, device="cuda")
    if inplace:
        owned = torch.zeros(T, dtype=torch.bool, device="cuda")
        owned[pb.starts[0]:pb.starts[-1]] = True
        q[~owned] = FILL
    sess.append_kv(pb.layer(heads), q if with_q else None, k, v, pb.row_start, pb.kv_len, plan,
                   q_gain=qg if with_q else None, k_gain=kg, eps=eps,
                   q_out=q_out if with_q else None)
    assert sess.error() == 0
    check(pb, heads, plan, q0 if with_q else None, k, v, qg, kg, eps, q_out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rot", [0, 2, 10, 32, 64])
@pytest.mark.parametrize("inter", [False, True])
def test_layouts(sess, dtype, dim, rot, inter):
    pb = Paged([3, 0, 17, 1], [0, 5, 61, 200], kvh=2, dim=dim, dtype=dtype, seed=rot + dim, lead=2,
               trail=3, fill=FILL)
    run(sess, pb, 6, pkg.rope_plan(rot, 1e4, interleaved=inter), norm=rot != 32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads,kvh", [(1, 1), (5, 1), (32, 8), (64, 8), (40, 8), (128, 1)])
def test_heads_packed_rows(sess, dtype, heads, kvh):
    pb = Paged([16, 16, 1], [64, 8000, 63], kvh=kvh, dim=128, dtype=dtype, seed=heads, fill=FILL)
    run(sess, pb, heads, pkg.rope_plan(128, 1e6), packed=True)


@pytest.mark.parametrize("scaling", ["none", "linear", "bands", "yarn"])
def test_far_positions(sess, scaling):
    """Angles of positions up to 2^21: an fp32 product of position and frequency would be off by
    2^-3 radians there."""
    pb = Paged([5, 2], [2 ** 21 - 70, 1_000_003], kvh=1, dim=64, dtype=F32, seed=4, fill=FILL)
    run(sess, pb, 2, pkg.rope_plan(64, 1e6, scaling=scaling, factor=8, original_positions=8192))


@pytest.mark.parametrize("inplace,with_q", [(True, True), (False, False)])
def test_in_place_and_without_queries(sess, inplace, with_q):
    pb = Paged([4, 9], [10, 64], prefix=128, kvh=2, dim=128, seed=9, trail=1, fill=FILL)
    run(sess, pb, 8, pkg.rope_plan(128, 1e6), inplace=inplace, with_q=with_q)


def test_many_requests_single_rows(sess):
    lens = [1 if i % 7 else 0 for i in range(1024)]
    pb = Paged(lens, [i % 190 for i in range(1024)], kvh=1, dim=64, seed=2, fill=FILL)
    run(sess, pb, 2, pkg.rope_plan(64, 1e6))


def test_one_gain_only_and_large_eps(sess):
    pb = Paged([4], [3], kvh=2, dim=64, seed=3, fill=FILL)
    q, k, v = pb.normal(4, 4, 64), pb.normal(4, 2, 64), pb.normal(4, 2, 64)
    k[1] = 0                                   # a zero head: eps alone in the root
    out = torch.full_like(q, FILL)
    kg = pb.normal(64)
    plan = pkg.rope_plan(64, 1e4)
    sess.append_kv(pb.layer(4), q, k, v, pb.row_start, pb.kv_len, plan, k_gain=kg, eps=0.5, q_out=out)
    check(pb, 4, plan, q, k, v, None, kg, 0.5, out)


def bad_case(sess, word, survivors, prefix=0, **change):
    pb = Paged([3, 4, 2], [10, 60, 0], prefix=prefix, kvh=1, dim=64, seed=6, trail=2, fill=FILL)
    for name, f in change.items():
        setattr(pb, name, f(getattr(pb, name)))
    T = pb.rows
    q, k, v = pb.normal(T, 2, 64), pb.normal(T, 1, 64), pb.normal(T, 1, 64)
    out = torch.full_like(q, FILL)
    plan = pkg.rope_plan(64, 1e4)
    sess.append_kv(pb.layer(2), q, k, v, pb.row_start, pb.kv_len, plan, q_out=out)
    assert sess.error() == word
    check(pb, 2, plan, q, k, v, None, None, 1e-6, out, rows_of_requests=survivors)


def put(i, v):
    def f(t):
        t = t.clone()
        t.view(-1)[i] = v
        return t
    return f


def test_rows_without_a_place_are_flagged_and_skipped(sess):
    """Bad lengths, pages and ranges: checked by the kernel, never read or written through."""
    bad_case(sess, 0x1, [0, 2], kv_len=put(1, -1))
    bad_case(sess, 0x1, [0, 2], kv_len=put(1, 2 * PAGE))              # past the page table
    bad_case(sess, 0x1, [0, 2], kv_len=put(1, 2 ** 31 - 2))
    bad_case(sess, 0x1, [0, 2], prefix=128, kv_len=put(1, 127))       # inside the shared prefix
    bad_case(sess, 0x2, [1, 2], table=put(0, -3))
    bad_case(sess, 0x2, [1, 2], table=put(0, 10 ** 6))
    bad_case(sess, 0x40, [1, 2], row_start=put(0, -1))
    bad_case(sess, 0x40, [0, 1], row_start=put(3, 12))                # past total_rows
    bad_case(sess, 0x40, [2], row_start=put(1, 99))                   # 0..99, 99..7; 7..9 is one


def test_a_row_of_two_requests_is_skipped(sess):
    pb = Paged([2, 2, 2], [0, 0, 0], kvh=1, dim=64, seed=8, fill=FILL)
    pb.row_start = i32([0, 4, 2, 6])           # 0..3, (4..2: none), 2..5: rows 2 and 3 twice
    q, k, v = pb.normal(6, 2, 64), pb.normal(6, 1, 64), pb.normal(6, 1, 64)
    out = torch.full_like(q, FILL)
    sess.append_kv(pb.layer(2), q, k, v, pb.row_start, pb.kv_len, pkg.rope_plan(0, 1e4), q_out=out)
    assert sess.error() == 0x40
    assert bool((out[2:4] == FILL).all()) and torch.equal(out[:2], q[:2]) and torch.equal(out[4:], q[4:])


def test_python_checks(sess):
    pb = Paged([2], [0], kvh=1, dim=64, seed=1, fill=FILL)
    lay, plan = pb.layer(2), pkg.rope_plan(64, 1e4)
    q, k, v = pb.normal(2, 2, 64), pb.normal(2, 1, 64), pb.normal(2, 1, 64)
    out = torch.empty_like(q)
    args = dict(layer=lay, q=q, k=k, v=v, row_start=pb.row_start, kv_len=pb.kv_len, rope=plan, q_out=out)
    for bad in [dict(q=q.float()), dict(q=q[:1]), dict(k=k.transpose(0, 1)), dict(v=v.cpu()),
                dict(q_out=None), dict(q=pb.normal(2, 64, 2).transpose(1, 2)),
                dict(row_start=pb.row_start[:1]), dict(kv_len=pb.kv_len.long()),
                dict(k_gain=pb.normal(32)), dict(kv_len=i32([0, 0]), row_start=i32([0, 1, 2]))]:
        with pytest.raises(ValueError):
            sess.append_kv(**{**args, **bad})
    with pytest.raises(pkg.DFlashError):
        sess.append_kv(**{**args, "rope": pkg.rope_plan(128, 1e4)})


def test_graph_and_side_stream(sess):
    pb = Paged([5, 1], [7, 70], kvh=2, dim=128, seed=12, fill=FILL)
    lay, plan = pb.layer(4), pkg.rope_plan(128, 1e6)
    q, k, v = pb.normal(6, 4, 128), pb.normal(6, 2, 128), pb.normal(6, 2, 128)
    out = torch.full_like(q, FILL)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        sess.append_kv(lay, q, k, v, pb.row_start, pb.kv_len, plan, q_out=out)
    for seed in (1, 2):                        # replays read what the buffers hold then
        g2 = torch.Generator(device="cuda").manual_seed(seed)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g2, device="cuda"))
        pb.k.fill_(FILL), pb.v.fill_(FILL)
        g.replay()
        check(pb, 4, plan, q, k, v, None, None, 1e-6, out)
    assert sess.error() == 0
