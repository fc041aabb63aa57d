"""Plain 64-bit forms of the target-side operators, and a small session to call them through."""
from types import SimpleNamespace

import torch

PAGE = 64


def make_session(dev="cuda", block=2, vocab=256, max_batch=4):
    """A draft session of a tiny model: the handle that the target-side calls take."""
    import block_diffusion_speculative_fc_gb300 as pkg
    cfg = SimpleNamespace(dtype="f32", target_hidden=128, n_sel=1, hidden=128, n_layers=1,
                          n_heads=2, n_kv_heads=1, head_dim=64, intermediate=128, vocab=vocab,
                          mask_token_id=vocab - 1, block_size=block, page_size=PAGE,
                          sliding_window=(0,), rms_eps=1e-6, rope_theta=1e6)
    z = lambda *s: torch.zeros(s, device=dev)  # noqa: E731
    W = {"fc": z(128, 128), "hidden_norm": z(128), "final_norm": z(128), "embed": z(vocab, 128),
         "lm_head": z(vocab, 128),
         "layers": [{"qkv": z(256, 128), "o": z(128, 128), "gate_up": z(256, 128),
                     "down": z(128, 128), "in_norm": z(128), "post_norm": z(128), "q_norm": z(64),
                     "k_norm": z(64)}]}
    return pkg.DraftSession(cfg, W, max_batch=max_batch, max_rows=16, max_position=64)


def i32(v):
    return torch.as_tensor(v, dtype=torch.int32, device="cuda")


class Paged:
    """A random ragged batch over a paged cache: `lens` new rows and `ctx` own rows before them per
    request, a shared prefix of `prefix` rows, a pool with spare pages in a seeded order."""

    def __init__(self, lens, ctx, prefix=0, kvh=2, dim=64, dtype=torch.bfloat16, seed=0, lead=0,
                 trail=0, fill=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.lens, self.ctx, self.prefix, self.dtype = g, lens, ctx, prefix, dtype
        self.kvh, self.dim, B = kvh, dim, len(lens)
        starts = [lead]
        for n in lens:
            starts.append(starts[-1] + n)
        self.starts, self.rows = starts, starts[-1] + trail
        need = [-(-(c + n) // PAGE) for c, n in zip(ctx, lens)]
        self.width = max(1, max(need))
        pool = torch.randperm(sum(need) + prefix // PAGE + 2, generator=g, device="cuda").tolist()
        self.n_pages = len(pool)
        self.prefix_list = [pool.pop() for _ in range(prefix // PAGE)]
        self.lists = [[pool.pop() for _ in range(n)] for n in need]
        self.table = i32([p + [0] * (self.width - len(p)) for p in self.lists])
        self.prefix_pages = i32(self.prefix_list) if prefix else None
        self.row_start, self.kv_len = i32(starts), i32([prefix + c for c in ctx])
        shape = (self.n_pages, PAGE, kvh, dim)
        if fill is None:
            self.k, self.v = self.normal(*shape), self.normal(*shape)
        else:
            self.k, self.v = (torch.full(shape, fill, dtype=dtype, device="cuda") for _ in "kv")

    def normal(self, *shape, scale=1.0):
        return (torch.randn(shape, generator=self.g, device="cuda") * scale).to(self.dtype)

    def layer(self, heads):
        import block_diffusion_speculative_fc_gb300 as pkg
        return pkg.LayerKV(heads, self.k, self.v, self.table, self.prefix_pages)

    def slots(self, b, first, last):
        """(pages, rows) of positions first..last-1 of request b."""
        pages = self.prefix_list + self.lists[b]
        pos = range(first, last)
        return ([pages[p // PAGE] for p in pos], [p % PAGE for p in pos])


def rope64(x, pos, inv, amp, inter):
    """x [n, heads, D] float64; inv: angles per position, float64."""
    half = len(inv)
    ang = pos.double()[:, None] * inv
    cos, sin = (ang.cos() * amp)[:, None], (ang.sin() * amp)[:, None]
    y = x.clone()
    i0, i1 = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter else \
        (slice(0, half), slice(half, 2 * half))
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * cos - b * sin, b * cos + a * sin
    big = x.abs()
    big[..., i0] = big[..., i1] = amp * (a.abs() + b.abs())   # what an fp32 rounding is relative to
    return y, big


def norm64(x, gain, eps):
    x = x.double()
    return x if gain is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gain.double()


def attend64(pb, q, heads, scale, causal):
    """{row: (out, bound)}: out [heads, D] float64 and, per element, sum_p softmax |V| and the largest
    scale * sum_d |q_d k_d| (what the errors of P and of the scores are relative to)."""
    G, res = heads // pb.kvh, {}
    for b, n in enumerate(pb.lens):
        if n == 0:
            continue
        total = pb.prefix + pb.ctx[b] + n
        pages, rows = pb.slots(b, 0, total)
        k, v = pb.k[pages, rows].double(), pb.v[pages, rows].double()
        k, v = (t.repeat_interleave(G, 1) for t in (k, v))
        for i in range(n):
            t, m = pb.starts[b] + i, (total - n + i + 1) if causal else total
            x = q[t].double()
            s = torch.einsum("hd,phd->hp", x, k[:m]) * scale
            mag = torch.einsum("hd,phd->hp", x.abs(), k[:m].abs()).amax(1) * abs(scale)
            p = torch.softmax(s, -1)
            res[t] = (torch.einsum("hp,phd->hd", p, v[:m]),
                      torch.einsum("hp,phd->hd", p, v[:m].abs()), mag)
    return res


def sample64(x, T, k, p, mp):
    """One row: (weights [V] with dropped ones 0, exponents a >= 0, distance of the nearest top-p
    border to a token's cumulative share) in float64."""
    V = x.numel()
    big = torch.finfo(x.dtype).max
    x = x.double()
    x = torch.where(x.isnan(), -torch.inf, x).clamp(max=big)
    m = x.max()
    if m == -torch.inf:
        return torch.zeros_like(x), torch.zeros_like(x), 1.0
    sx, at = x.sort(descending=True, stable=True)
    keep = sx > -torch.inf
    rank = torch.arange(V, device=x.device)
    near = 1.0
    if T < 2.0 ** -126:
        keep &= rank == 0
        w = torch.ones_like(sx)
        a = torch.zeros_like(sx)
    else:
        a = (m - sx) / T
        w = torch.exp(-a)
        if k > 0:
            keep &= rank < k
        if p < 1:
            wk = torch.where(keep, w, 0.0)
            cum = wk.cumsum(0) - wk
            share = cum / wk.sum()
            near = float((share[keep] - p).abs().min())
            keep &= (share < p) | (rank == 0)
        keep &= w >= mp
    out = torch.zeros_like(x)
    out[at] = torch.where(keep, w, 0.0)
    full = torch.zeros_like(x)
    full[at] = torch.where(keep, a, 0.0)
    return out, full, near
