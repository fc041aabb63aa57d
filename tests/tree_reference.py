"""Plain 64-bit forms of the tree and eviction calls over tests.target_reference.Paged batches."""
import random

import torch


def random_parents(n, rng, back=6):
    """Row 0 the root; a later row's parent one of the `back` rows before it."""
    return [-1] + [max(0, i - 1 - rng.randrange(back)) for i in range(1, n)]


def closure(parents):
    """seen[i][j]: row j is row i or an ancestor of it."""
    n = len(parents)
    seen = torch.zeros((n, n), dtype=torch.bool)
    for i, p in enumerate(parents):
        if p >= 0:
            seen[i] = seen[p]
        seen[i, i] = True
    return seen


def pack(seen, rows, starts, words, fill=0):
    """Mask int32 [rows, words] of the requests' [n, n] truth values."""
    mask = torch.full((rows, words), fill, dtype=torch.int64)
    for s, m in zip(starts, seen):
        n = m.shape[0]
        bits = torch.zeros((n, 32 * words), dtype=torch.int64)
        bits[:, :n] = m.long()
        if fill:
            bits[:, n:] = 1          # bits past the request's rows count for nothing
        mask[s:s + n] = (bits.view(n, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to(torch.int32).cuda()


def causal(n):
    return torch.ones((n, n), dtype=torch.bool).tril()


def scores64(pb, q, heads, scale, b, seen, own_only=False):
    """(scores [n, heads, keys] with -inf where not seen, |scale| sum |q k|, keys, values, seen [n, keys])
    of request b in float64."""
    n, total = pb.lens[b], pb.prefix + pb.ctx[b] + pb.lens[b]
    first = pb.prefix if own_only else 0
    pages, rows = pb.slots(b, first, total)
    G = heads // pb.kvh
    k, v = (t[pages, rows].double().repeat_interleave(G, 1) for t in (pb.k, pb.v))
    vis = torch.ones((n, total - first), dtype=torch.bool, device="cuda")
    vis[:, total - first - n:] = seen.cuda()
    x = q[pb.starts[b]:pb.starts[b] + n].double()
    # a key that a row does not see has no part in it, whatever it holds
    some = vis.any(0)
    k = torch.where(some[:, None, None], k, 0.0)
    v = torch.where(some[:, None, None], v, 0.0)
    s = torch.einsum("nhd,phd->nhp", x, k) * scale
    mag = torch.einsum("nhd,phd->nhp", x.abs(), k.abs()) * abs(scale)
    return s.masked_fill(~vis[:, None], -torch.inf), mag, k, v, vis


def attend_tree64(pb, q, heads, scale, seen):
    """{row: (out, sum_p softmax |V|, largest |score| bound, lse)}; zeros and -inf where nothing is seen."""
    res = {}
    for b, n in enumerate(pb.lens):
        if n == 0:
            continue
        s, mag, k, v, vis = scores64(pb, q, heads, scale, b, seen[b])
        for i in range(n):
            t = pb.starts[b] + i
            at = vis[i].nonzero()[:, 0]
            if len(at) == 0:
                z = torch.zeros((heads, pb.dim), dtype=torch.float64, device="cuda")
                res[t] = (z, z, torch.zeros(heads, dtype=torch.float64, device="cuda"),
                          torch.full((heads,), -torch.inf, dtype=torch.float64, device="cuda"))
                continue
            si = s[i][:, at]
            p = torch.softmax(si, -1)
            res[t] = (torch.einsum("hp,phd->hd", p, v[at]), torch.einsum("hp,phd->hd", p, v[at].abs()),
                      mag[i][:, at].amax(1), torch.logsumexp(si, -1))
    return res


def weights64(pb, q, heads, scale, seen, lse, row_weight, decay, old):
    """(weights [B, KVH, width] in float64, bound of their error, live [B, width])."""
    want, tol = old.double().clone(), torch.zeros_like(old, dtype=torch.float64)
    live = torch.zeros((old.shape[0], old.shape[2]), dtype=torch.bool, device="cuda")
    G, D = heads // pb.kvh, pb.dim
    for b, n in enumerate(pb.lens):
        if n == 0:
            continue
        c = pb.ctx[b]
        live[b, :c + n] = True
        want[b, :, :c] = want[b, :, :c] * decay if decay else 0.0
        want[b, :, c:c + n] = 0.0
        # the old value: the factor rounded to float32, the product, the last addition, 2^-24 each
        tol[b] = 3 * 2.0 ** -24 * want[b].abs()
        rows = slice(pb.starts[b], pb.starts[b] + n)
        s, mag, _, _, _ = scores64(pb, q, heads, scale, b, seen[b], own_only=True)
        z = lse[rows].double()[..., None]
        rw = torch.ones(n, dtype=torch.float64, device="cuda") if row_weight is None else row_weight[rows].double()
        counts = z.isfinite() & (rw > 0)[:, None, None] & rw.isfinite()[:, None, None]
        p = torch.where(counts & (s > -torch.inf), torch.exp(s - z) * rw[:, None, None], 0.0)
        err = p * ((D + 8) * 2.0 ** -24 * mag + 2.0 ** -22 * z.abs().nan_to_num(0, 0, 0)
                   + 2.0 ** -22 * rw[:, None, None].clamp(min=1e-30).log().abs().nan_to_num(0, 0, 0) + 2.0 ** -20)
        add = p.sum(0).view(pb.kvh, G, -1).sum(1)
        want[b, :, :c + n] += add
        tol[b, :, :c + n] += (err.sum(0).view(pb.kvh, G, -1).sum(1) + (n * G + 8) * 2.0 ** -24 * add
                              + n * G * 2.0 ** -126)
    return want, tol, live


def choose(w, n, keep, first, last):
    """Kept rows of one list, from a list of floats."""
    if n <= keep:
        return list(range(n))
    a = min(first, keep)
    z = min(last, keep - a)
    key = [(-float("inf") if x != x else x) for x in w[:n]]
    mid = sorted(range(a, n - z), key=lambda i: (-key[i], i))[:keep - a - z]
    return sorted(list(range(a)) + mid + list(range(n - z, n)))


def walk(parents, tokens, posterior, most):
    """Rows of the path of one request."""
    path = [0]
    while len(path) < most:
        nxt = [c for c in range(1, len(parents)) if parents[c] == path[-1] and tokens[c] == posterior[path[-1]]]
        if not nxt:
            break
        path.append(nxt[0])
    return path


def rng_of(seed):
    return random.Random(seed)
