"""Measured operators of tree-shaped verification and of eviction from a target layer's cache.

plan     depths (as positions) and ancestor masks of the requests' draft trees (dflash_tree_plan)
tree     attention of the tree's rows over the paged cache and their own ancestors, with the log of
         each row's softmax sum (dflash_tree_attention)
accept   the walk down a tree along the target's tokens, and its commit (dflash_accept_commit_tree)
weights  the attention weight that falls on every cached row, accumulated (dflash_key_weights)
choose   the rows that a budget keeps: the first, the last, the heaviest (dflash_choose_rows)
keep     a list of rows moved together in the cache: an accepted path, or what an eviction keeps
         (dflash_keep_rows)

Shapes are those of this repository's workloads (32 or 64 query heads on 8 KV heads of 128) and
generic ones around them.
"""
import math

import torch

own = False

PAGE = 64
VOCAB = 8192


def _trees(name, op, batch, nodes):
    """nodes [lo, hi]: rows of a request's tree, the root among them."""
    return {"name": name, "op": op, "batch": batch, "n_lo": nodes[0], "n_hi": nodes[1]}


def _attend(name, op, batch, rows, ctx, prefix=0, heads=32, kvh=8, dim=128, dtype="bf16", tree=True,
            decay=0.0):
    """rows [lo, hi]: new rows per request; ctx [lo, hi]: own rows in the cache before them."""
    return {"name": name, "op": op, "batch": batch, "n_lo": rows[0], "n_hi": rows[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "prefix": prefix, "heads": heads, "kvh": kvh,
            "dim": dim, "dtype": dtype, "tree": tree, "decay": decay}


def _choose(name, batch, rows, keep, first, last, kvh=8):
    return {"name": name, "op": "choose", "batch": batch, "ctx_lo": rows[0], "ctx_hi": rows[1],
            "keep": keep, "first": first, "last": last, "kvh": kvh}


def _keep(name, batch, rows, keep, path, kvh=8, dim=128, dtype="bf16"):
    """path: one list a request, of at most `keep` of `rows` new rows behind a context; else a list a
    head, `keep` of the `rows` in the cache, and the heads' weights with it."""
    return {"name": name, "op": "keep", "batch": batch, "n_lo": rows[0], "n_hi": rows[1],
            "keep": keep, "path": path, "kvh": kvh, "dim": dim, "dtype": dtype}


def listed():
    return [
        # one request's tree of 64 drafted tokens: the smallest call of a step
        _trees("plan-b1", "plan", 1, [64, 64]),
        # a large batch of trees of uneven size
        _trees("plan-b128", "plan", 128, [17, 250]),
        # one request, a tree of 64, a short context: latency
        _attend("tree-b1", "tree", 1, [64, 64], [2000, 2000]),
        # 32 uneven trees over a system prompt of 8k rows and the requests' own
        _attend("tree-b32-shared", "tree", 32, [16, 64], [256, 4096], prefix=8192),
        # the walks of the same two batches
        _trees("accept-b1", "accept", 1, [64, 64]),
        _trees("accept-b128", "accept", 128, [17, 250]),
        # 32 requests decoding a token each: every step adds its weights
        _attend("weights-token-b32", "weights", 32, [1, 1], [500, 16000], tree=False, decay=1.0),
        # the last 64 rows of two long prompts judge the rows before them (64 query heads)
        _attend("weights-window-b2", "weights", 2, [64, 64], [8000, 30000], heads=64, tree=False),
        # one request over its budget
        _choose("choose-b1", 1, [4096, 4096], 2048, 4, 256),
        # 32 requests of uneven length, some below the budget
        _choose("choose-b32", 32, [2000, 32000], 4096, 4, 512),
        # accepted paths of 64 trees, moved to the end of the committed rows
        _keep("keep-path-b64", 64, [16, 64], 12, True),
        # eight requests cut to 4096 rows a head
        _keep("keep-evict-b8", 8, [5000, 16000], 4096, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "tree", "accept", "weights", "choose", "keep"])
    kvh = rng.choice([1, 2, 4, 8])
    if op in ("plan", "accept"):
        batch = _log(rng, 1, 128)
        hi = _log(rng, 1, min(900, 17000 // batch))
        return _trees(None, op, batch, [max(1, hi // rng.choice([1, 2, 7])), hi])
    if op in ("tree", "weights"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        group, dim = rng.choice([1, 4, 5, 8]), rng.choice([64, 128, 128])
        batch = _log(rng, 1, 32 if dtype == "bf16" else 8)
        hi = _log(rng, 1, max(1, min(300, (1200 if dtype == "bf16" else 200) // batch)))
        rows = [max(1, hi // rng.choice([1, 3])), hi]
        if op == "tree":
            c_hi = _log(rng, 10, 4000)
            prefix = PAGE * _log(rng, 1, 128) if rng.random() < 0.5 else 0
        else:
            c_hi = _log(rng, 10, max(20, min(30000, 250000 // batch, 2000000 // (batch * hi))))
            prefix = PAGE * _log(rng, 1, 8) if rng.random() < 0.3 else 0
        if dtype == "f32":
            c_hi, prefix = min(c_hi, 2000), min(prefix, 1024)
        return _attend(None, op, batch, rows, [rng.randint(0, c_hi), c_hi], prefix=prefix,
                       heads=kvh * group, kvh=kvh, dim=dim, dtype=dtype, tree=rng.random() < 0.7,
                       decay=rng.choice([0.0, 1.0, 0.95]) if op == "weights" else 0.0)
    if op == "choose":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 64, min(60000, 500000 // batch))
        keep = _log(rng, 8, hi - hi // 8)
        return _choose(None, batch, [max(1, hi // rng.choice([1, 3, 10])), hi], keep,
                       min(keep // 4, rng.choice([0, 4, 64])), min(keep // 4, rng.choice([0, 33, 512])),
                       kvh=kvh)
    path, dim, dtype = rng.random() < 0.4, rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "f32"])
    batch = _log(rng, 1, 64)
    hi = _log(rng, 2, 256 if path else min(30000, 60000 // batch))
    keep = min(hi, _log(rng, 1, 24)) if path else _log(rng, 1, hi)
    return _keep(None, batch, [max(1, hi // rng.choice([1, 2, 3])), hi], keep, path, kvh=kvh, dim=dim,
                 dtype=dtype)


# ---------------------------------------------------------------- inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _spread(lo, hi, n):
    """n whole numbers spread evenly over lo..hi: their sum does not go by the seed."""
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _session():
    """A draft session of a tiny model: what holds the handle that the calls take."""
    from types import SimpleNamespace

    import block_diffusion_speculative_fc_gb300 as pkg
    cfg = SimpleNamespace(dtype="f32", target_hidden=128, n_sel=1, hidden=128, n_layers=1,
                          n_heads=2, n_kv_heads=1, head_dim=64, intermediate=128, vocab=VOCAB,
                          mask_token_id=VOCAB - 1, block_size=2, page_size=PAGE,
                          sliding_window=(0,), rms_eps=1e-6, rope_theta=1e6)
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    W = {"fc": z(128, 128), "hidden_norm": z(128), "final_norm": z(128), "embed": z(VOCAB, 128),
         "lm_head": z(VOCAB, 128),
         "layers": [{"qkv": z(256, 128), "o": z(128, 128), "gate_up": z(256, 128),
                     "down": z(128, 128), "in_norm": z(128), "post_norm": z(128), "q_norm": z(64),
                     "k_norm": z(64)}]}
    return pkg, pkg.DraftSession(cfg, W, max_batch=1, max_rows=16, max_position=64)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    B = case["batch"]
    order = torch.randperm(B, generator=g, device="cuda").tolist()
    lists = {k: [_spread(case[k + "_lo"], case[k + "_hi"], B)[i] for i in order]
             for k in ("n", "ctx") if k + "_lo" in case}
    st = {"case": case, "g": g}
    {"plan": _prepare_trees, "accept": _prepare_trees, "tree": _prepare_attend,
     "weights": _prepare_attend, "choose": _prepare_choose, "keep": _prepare_keep}[case["op"]](
        st, case, g, **lists)
    if own:
        st["sess"] = _session()[1]
        if "k_pages" in st:
            import block_diffusion_speculative_fc_gb300 as pkg
            st["layer"] = pkg.LayerKV(case.get("heads", case["kvh"]), st["k_pages"], st["v_pages"],
                                      st["table"], prefix_pages=st.get("prefix_pages"))
        if case["op"] == "tree":
            st["ws"] = st["sess"].attention_workspace(st["layer"], B, st["T"])
    return st


def _starts(st, n):
    starts = [0]
    for v in n:
        starts.append(starts[-1] + v)
    st["T"], st["n_max"], st["row_start"] = starts[-1], max(n), _i32(starts)
    st["words"] = (max(n) + 31) // 32


def _parents(st, g):
    """Row 0 of a request is its root; a later row's parent is one of the eight rows before it."""
    b, i = _rows(st)
    u = torch.rand(st["T"], generator=g, device="cuda")
    back = (u * i.clamp(max=8)).long().clamp(max=7)
    return torch.where(i == 0, -1, (i - 1 - back).clamp(min=0)).int()


def _prepare_trees(st, case, g, n):
    _starts(st, n)
    T, B = st["T"], case["batch"]
    st["parent"] = _parents(st, g)
    st["root"] = torch.randint(0, 30000, (B,), generator=g, device="cuda", dtype=torch.int32)
    if case["op"] == "plan":
        st["mask"] = torch.zeros((T, st["words"]), dtype=torch.int32, device="cuda")
        st["positions"] = torch.zeros(T, dtype=torch.int32, device="cuda")
        return
    tok = torch.randint(0, VOCAB, (T,), generator=g, device="cuda", dtype=torch.int32)
    # three quarters of the nodes with children: the target's token is that of the last child
    b, i = _rows(st)
    at = st["row_start"].long()[b] + st["parent"].long()
    last = torch.full((T,), -1, dtype=torch.long, device="cuda")
    last.scatter_reduce_(0, at[i > 0], torch.arange(T, device="cuda")[i > 0], "amax")
    other = torch.randint(0, VOCAB, (T,), generator=g, device="cuda", dtype=torch.int32)
    hit = (torch.rand(T, generator=g, device="cuda") < 0.75) & (last >= 0)
    st["tokens"], st["posterior"] = tok, torch.where(hit, tok[last], other)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    # as long a path as the largest tree has rows
    st["outs"] = {"accept_len": z(B), "commit_len": z(B), "bonus": z(B), "out_tokens": z(B, st["n_max"]),
                  "path": z(B, st["n_max"])}
    st["seq"] = z(B)
    st["row_weight"] = torch.zeros(T, device="cuda")


def _pages(st, case, g, total, prefix=0, values=True):
    """Pages of `total` rows per request and of the shared prefix, in a seeded order."""
    dt, B, KVH, D = _dt(case), case["batch"], case["kvh"], case["dim"]
    need = [(t + PAGE - 1) // PAGE for t in total]
    width, used, n_prefix = max(need), sum(need), prefix // PAGE
    pool = torch.randperm(used + n_prefix, generator=g, device="cuda").to(torch.int32)
    mine = torch.arange(width, device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    st["table"] = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    st["table"][mine] = pool[:used]
    if prefix:
        st["prefix_pages"] = pool[used:]
    shape = (used + n_prefix, PAGE, KVH, D)
    normal = lambda: torch.randn(shape, generator=g, device="cuda").to(dt)  # noqa: E731
    st["k_pages"] = normal()
    st["v_pages"] = normal() if values else torch.zeros_like(st["k_pages"])


def _prepare_attend(st, case, g, n, ctx):
    _starts(st, n)
    T, H, D, prefix = st["T"], case["heads"], case["dim"], case["prefix"]
    _pages(st, case, g, [a + c for a, c in zip(n, ctx)], prefix, values=case["op"] == "tree")
    st["kv_len"] = _i32([prefix + c for c in ctx])
    # head-normed queries and keys: logits of a few units, a few keys that stand out
    st["q"] = (torch.randn((T, H, D), generator=g, device="cuda") * 1.5).to(_dt(case))
    st["parent"] = _parents(st, g) if case["tree"] else None
    if case["tree"]:
        st["mask"] = _plain_plan({**st, "root": st["kv_len"]})["mask"]
    if case["op"] == "tree":
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((T, H), device="cuda")
        return
    # what the attention has said of each row; the prefix, where there is one, has part of the sum
    b, i = _rows(st)
    s, _, _ = _own_scores(st)
    st["lse"] = torch.logsumexp(s, -1).view(len(n), case["kvh"], st["n_max"], -1)[b, :, i] \
        .reshape(T, H).contiguous() + (0.3 if prefix else 0.0)
    del s
    # some rows (rejected ones) do not count
    st["row_weight"] = (torch.rand(T, generator=g, device="cuda") < 0.7).float() if case["tree"] else None
    width = max(a + c for a, c in zip(n, ctx))
    st["weights"] = torch.rand((len(n), case["kvh"], width), generator=g, device="cuda")


def _prepare_choose(st, case, g, ctx):
    B, KVH = case["batch"], case["kvh"]
    # weights as attention leaves them: most of them small
    w = torch.randn((B, KVH, max(ctx)), generator=g, device="cuda")
    st["weights"] = torch.exp(2.5 * w).mul_(0.01)
    st["weights"][..., ::97] = 0.0    # rows that nothing has looked at: equal ones
    st["kv_len"] = _i32(ctx)
    st["keep"] = torch.full((B,), case["keep"], dtype=torch.int32, device="cuda")
    st["rows"] = torch.full((B, KVH, case["keep"]), -1, dtype=torch.int32, device="cuda")
    st["count"] = torch.zeros((B, KVH), dtype=torch.int32, device="cuda")
    # (the call takes the layer whose cache is to be cut: a page of it will do)
    if own:
        st["k_pages"], st["v_pages"] = (torch.zeros((1, PAGE, KVH, 64), device="cuda") for _ in "kv")
        st["table"] = torch.zeros((B, (max(ctx) + PAGE - 1) // PAGE), dtype=torch.int32, device="cuda")


def _prepare_keep(st, case, g, n):
    B, KVH, keep = case["batch"], case["kvh"], case["keep"]
    first = [(37 * v) % 300 for v in n] if case["path"] else [0] * B
    _pages(st, case, g, [a + f for a, f in zip(n, first)])
    st["first"] = _i32(first) if case["path"] else None
    L, width = 1 if case["path"] else KVH, max(n)
    key = torch.rand((B, L, width), generator=g, device="cuda")
    key.masked_fill_(torch.arange(width, device="cuda") >= torch.tensor(n, device="cuda")[:, None, None], 2.0)
    key[..., 0] = -1.0    # the root, or a first row that is always kept
    at = key.argsort(-1)[..., :keep]
    count = torch.tensor([min(keep, v) for v in n], device="cuda")
    at.masked_fill_(torch.arange(at.shape[-1], device="cuda") >= count[:, None, None], width)
    st["rows"] = at.sort(-1).values.int()
    st["count"] = count.int()[:, None].expand(B, L).contiguous()
    if not case["path"]:
        st["weights"] = torch.rand((B, KVH, width), generator=g, device="cuda")


# ---------------------------------------------------------------- one pass
def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "tree": _plain_tree, "accept": _plain_accept,
                "weights": _plain_weights, "choose": _plain_choose, "keep": _plain_keep}[op](st)
    s = st["sess"]
    if op == "plan":
        s.tree_plan(st["row_start"], st["parent"], st["mask"], st["positions"], root=st["root"])
        return {"mask": st["mask"], "positions": st["positions"]}
    if op == "tree":
        s.tree_attention(st["layer"], st["q"], st["row_start"], st["kv_len"], st["out"], st["ws"],
                         mask=st["mask"] if case["tree"] else None, lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "accept":
        o = st["outs"]
        st["seq"].copy_(st["root"])
        s.accept_tree(st["row_start"], st["parent"], st["tokens"], st["posterior"], st["seq"],
                      o["accept_len"], o["commit_len"], o["bonus"], o["out_tokens"], o["path"],
                      row_weight=st["row_weight"])
        return {**o, "seq_len": st["seq"], "row_weight": st["row_weight"]}
    if op == "weights":
        s.key_weights(st["layer"], st["q"], st["row_start"], st["kv_len"], st["lse"], st["weights"],
                      mask=st["mask"] if case["tree"] else None, row_weight=st["row_weight"],
                      decay=case["decay"])
        return {"weights": st["weights"]}
    if op == "choose":
        s.choose_rows(st["layer"], st["weights"], st["kv_len"], st["keep"], st["rows"], st["count"],
                      first=case["first"], last=case["last"])
        return {"rows": st["rows"], "count": st["count"]}
    s.keep_rows(st["layer"], st["rows"], st["count"], first=st["first"], weights=st.get("weights"))
    out = {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    return out if case["path"] else {**out, "weights": st["weights"]}


def _rows(st):
    """Request of every new row, and its number there."""
    rs = st["row_start"].long()
    b = torch.repeat_interleave(torch.arange(len(rs) - 1, device="cuda"), rs[1:] - rs[:-1],
                                output_size=st["T"])
    return b, torch.arange(st["T"], device="cuda") - rs[b]


def _ancestors(st):
    """[B, n, n]: row i's ancestors and itself, from the parents by repeated squaring."""
    b, i = _rows(st)
    B, n = len(st["row_start"]) - 1, st["n_max"]
    R = torch.eye(n, device="cuda").repeat(B, 1, 1)
    child = st["parent"] >= 0
    R[b[child], i[child], st["parent"].long()[child]] = 1.0
    for _ in range(max(1, (n - 1).bit_length())):
        R = (R @ R).clamp_(max=1.0)
    return R > 0, b, i


def _plain_plan(st):
    R, b, i = _ancestors(st)
    seen = torch.zeros((st["T"], 32 * st["words"]), dtype=torch.bool, device="cuda")
    seen[:, :st["n_max"]] = R[b, i]
    bit = torch.arange(32, device="cuda")
    words = (seen.view(st["T"], st["words"], 32).long() << bit).sum(-1)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words)
    return {"mask": words.int(), "positions": (st["root"].long()[b] + seen.sum(-1) - 1).int()}


def _plain_accept(st):
    R, b, i = _ancestors(st)
    B, n, rs = R.shape[0], st["n_max"], st["row_start"].long()
    T = st["T"]
    pad = lambda x, v: torch.full((B, n), v, dtype=torch.long, device="cuda").index_put((b, i), x.long())  # noqa: E731
    tok, post, par = pad(st["tokens"], -1), pad(st["posterior"], -2), pad(st["parent"], -2)
    right = (par >= 0) & (tok == post.gather(1, par.clamp(min=0)))
    # of equal children the first
    twin = (par[:, :, None] == par[:, None, :]) & right[:, None, :]
    twin &= torch.ones((n, n), dtype=torch.bool, device="cuda").tril(-1)
    good = (right & ~twin.any(-1)).clone()
    good[:, 0] = True
    on = (good[:, None, :] | ~R).all(-1) & (par > -2)
    on &= R[:, :, 0]    # down from the root
    commit = on.sum(-1)
    place = on.long().cumsum(-1) - 1
    node = torch.arange(n, device="cuda").expand(B, n)
    path = torch.full((B, n + 1), -1, dtype=torch.long, device="cuda")
    path.scatter_(1, torch.where(on, place, n), node)
    path = path[:, :n]
    path[torch.arange(n, device="cuda") >= commit[:, None]] = -1
    end = path.gather(1, commit[:, None] - 1)
    bonus = post.gather(1, end)[:, 0]
    nxt = torch.cat([path[:, 1:], torch.full((B, 1), -1, dtype=torch.long, device="cuda")], 1)
    out = torch.where(nxt >= 0, tok.gather(1, nxt.clamp(min=0)), 0)
    out.scatter_(1, commit[:, None] - 1, bonus[:, None])
    return {"accept_len": (commit - 1).int(), "commit_len": commit.int(), "bonus": bonus.int(),
            "out_tokens": out.int(), "path": path.int(), "seq_len": (st["root"].long() + commit).int(),
            "row_weight": on[b, i].float()}


def _own_scores(st):
    """Scores over the requests' own keys [B, KVH, n_max * group, keys], -inf where not seen; what is
    seen, and the requests' keys."""
    case, T, prefix = st["case"], st["T"], st["case"]["prefix"]
    H, KVH, D, B, n_max = case["heads"], case["kvh"], case["dim"], case["batch"], st["n_max"]
    G, rs = H // KVH, st["row_start"].long()
    b, i = _rows(st)
    q = torch.zeros((B, n_max, H, D), device="cuda")
    q[b, i] = st["q"].float() * D ** -0.5
    table = st["table"].long()
    k = st["k_pages"][table].float().flatten(1, 2)     # [B, keys, KVH, D]
    keys = torch.arange(k.shape[1], device="cuda")
    ctx, n = st["kv_len"].long() - prefix, rs[1:] - rs[:-1]
    new = keys[None] - ctx[:, None]                    # number of a key among the new rows
    if case["tree"]:
        bits = torch.zeros((B, n_max, 32 * st["words"]), dtype=torch.bool, device="cuda")
        bits[b, i] = ((st["mask"].long()[:, :, None] >> torch.arange(32, device="cuda")) & 1).flatten(1) > 0
        seen = bits.gather(2, new.clamp(0, 32 * st["words"] - 1)[:, None].expand(B, n_max, -1))
    else:
        seen = new[:, None] <= torch.arange(n_max, device="cuda")[:, None]
    seen = (seen & (new < n[:, None])[:, None]) | (new < 0)[:, None]
    seen = seen & (torch.arange(n_max, device="cuda") < n[:, None])[..., None]
    seen = seen.repeat_interleave(G, dim=1)[:, None]
    q = q.view(B, n_max, KVH, G, D).permute(0, 2, 1, 3, 4).reshape(B, KVH, n_max * G, D)
    s = q @ k.permute(0, 2, 3, 1)
    return s.masked_fill_(~seen, -math.inf), seen, keys


def _plain_tree(st):
    case, T, prefix = st["case"], st["T"], st["case"]["prefix"]
    H, KVH, D, B, n_max = case["heads"], case["kvh"], case["dim"], case["batch"], st["n_max"]
    G = H // KVH
    b, i = _rows(st)
    s, _, keys = _own_scores(st)
    rs = st["row_start"].long()
    behind = keys[None] >= (st["kv_len"].long() - prefix + rs[1:] - rs[:-1])[:, None]
    v = st["v_pages"][st["table"].long()].float().flatten(1, 2).masked_fill(behind[:, :, None, None], 0.0)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    if prefix:
        page = st["prefix_pages"].long()
        kp, vp = (st[x][page].float().flatten(0, 1).permute(1, 0, 2) for x in ("k_pages", "v_pages"))
        q = st["q"].float() * D ** -0.5
        sp = q.view(T, KVH, G, D).permute(1, 0, 2, 3).reshape(KVH, T * G, D) @ kp.transpose(1, 2)
        mo = m.view(B, KVH, n_max, G)
        mo[b, :, i] = torch.maximum(mo[b, :, i], sp.amax(-1).view(KVH, T, G).permute(1, 0, 2))
        m = mo.reshape(B, KVH, n_max * G, 1)
    e = torch.exp(s - m)
    den = e.sum(-1).view(B, KVH, n_max, G)[b, :, i]    # [T, KVH, G]
    out = (e @ v.permute(0, 2, 1, 3)).view(B, KVH, n_max, G, D)[b, :, i]
    mt = m.view(B, KVH, n_max, G)[b, :, i]
    if prefix:
        ep = torch.exp(sp - mt.permute(1, 0, 2).reshape(KVH, T * G, 1))
        den = den + ep.sum(-1).view(KVH, T, G).permute(1, 0, 2)
        out = out + (ep @ vp).view(KVH, T, G, D).permute(1, 0, 2, 3)
    return {"out": (out / den[..., None]).reshape(T, H, D).to(st["q"].dtype),
            "lse": (mt + den.log()).reshape(T, H)}


def _plain_weights(st):
    case, B, n_max = st["case"], st["case"]["batch"], st["n_max"]
    H, KVH = case["heads"], case["kvh"]
    b, i = _rows(st)
    s, _, keys = _own_scores(st)
    lse = torch.zeros((B, n_max, H), device="cuda")
    lse[b, i] = st["lse"]
    lse = lse.view(B, n_max, KVH, H // KVH).transpose(1, 2).reshape(B, KVH, -1, 1)
    w = torch.exp(s - lse)
    if st["row_weight"] is not None:
        rw = torch.zeros((B, n_max), device="cuda")
        rw[b, i] = st["row_weight"]
        w = w * rw.repeat_interleave(H // KVH, dim=1)[:, None, :, None]
    rs, width = st["row_start"].long(), st["weights"].shape[-1]
    add = w.sum(2)[..., :width]
    ctx = (st["kv_len"].long() - case["prefix"])[:, None]
    at = keys[None, :width]
    # rows of this call begin at 0; what lies behind a request's last row is left as it was
    old = st["weights"] * case["decay"] if case["decay"] else torch.zeros_like(st["weights"])
    new = torch.where((at < ctx)[:, None], old, 0.0) + add
    live = (at < ctx + (rs[1:] - rs[:-1])[:, None])[:, None]
    st["weights"].copy_(torch.where(live, new, st["weights"]))
    return {"weights": st["weights"]}


def _plain_choose(st):
    case, w = st["case"], st["weights"]
    n = st["kv_len"].long()[:, None, None]
    keep = st["keep"].long()[:, None, None]
    at = torch.arange(w.shape[-1], device="cuda")
    first = torch.clamp(keep, max=case["first"])
    last = torch.minimum(keep - first, torch.full_like(keep, case["last"]))
    key = w.double().nan_to_num(nan=-math.inf).clamp(min=-1e300, max=1e300)
    key = key.masked_fill((at < first) | (at >= n - last), 1e301).masked_fill(at >= n, -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, at.expand_as(order))
    kept = (rank < keep) & (at < n)
    place = torch.where(kept, kept.long().cumsum(-1) - 1, case["keep"])
    rows = torch.full((*w.shape[:2], case["keep"] + 1), -1, dtype=torch.long, device="cuda")
    rows.scatter_(-1, place, at.expand_as(order))
    rows[..., case["keep"]] = -1
    count = kept.sum(-1)
    return {"rows": rows[..., :case["keep"]].int(), "count": count.int()}


def _plain_keep(st):
    case, KVH, B = st["case"], st["case"]["kvh"], st["case"]["batch"]
    rows = st["rows"].long().expand(B, KVH, -1)
    i = torch.arange(rows.shape[-1], device="cuda").expand_as(rows)
    live = i < st["count"].long()[..., None]
    first = st["first"].long()[:, None, None] if case["path"] else 0
    b = torch.arange(B, device="cuda")[:, None, None].expand_as(rows)[live]
    h = torch.arange(KVH, device="cuda")[:, None].expand_as(rows)[live]
    src, dst = (rows + first)[live], (i + first)[live]
    table = st["table"].long()
    ps, pd = table[b, src // PAGE], table[b, dst // PAGE]
    k, v = st["k_pages"], st["v_pages"]
    k[pd, dst % PAGE, h], v[pd, dst % PAGE, h] = k[ps, src % PAGE, h], v[ps, src % PAGE, h]
    if case["path"]:
        return {"k_pages": k, "v_pages": v}
    w = st["weights"]
    w[b, h, dst] = w[b, h, src]
    return {"k_pages": k, "v_pages": v, "weights": w}


# ---------------------------------------------------------------- floors and 64-bit values
def work(case):
    B = case["batch"]
    n = _spread(case["n_lo"], case["n_hi"], B) if "n_lo" in case else []
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], B) if "ctx_lo" in case else []
    T, words = sum(n), (max(n) + 31) // 32 if n else 0
    es = 4 if case.get("dtype") == "f32" else 2
    op = case["op"]
    if op == "plan":
        return {"bytes": 4 * T * (2 + words) + 8 * B, "flops": T * words}
    if op == "accept":
        return {"bytes": 4 * (4 * T + B * (6 + 2 * max(n))), "flops": T}
    if op == "choose":
        kept = sum(min(c, case["keep"]) for c in ctx)
        return {"bytes": 4 * case["kvh"] * (sum(ctx) + kept), "flops": case["kvh"] * sum(ctx)}
    if op == "keep":
        kept = sum(min(v, case["keep"]) for v in n) * case["kvh"]
        lists = kept // case["kvh"] if case["path"] else kept
        return {"bytes": 4 * kept * case["dim"] * es + 4 * lists + (0 if case["path"] else 8 * kept),
                "flops": kept}
    H, KVH, D, prefix = case["heads"], case["kvh"], case["dim"], case["prefix"]
    own_keys = sum(n) + sum(ctx)
    if op == "tree":
        # (of the new rows each sees itself at least)
        seen = sum(v * (prefix + c + 1) for v, c in zip(n, ctx))
        return {"bytes": 2 * (prefix + own_keys) * KVH * D * es + 2 * T * H * D * es + 4 * T * H,
                "flops": 4 * seen * H * D}
    seen = sum(v * (c + 1) for v, c in zip(n, ctx))
    return {"bytes": own_keys * KVH * (D * es + 4) + T * H * (D * es + 4)
            + (4 * sum(ctx) * KVH if case["decay"] else 0), "flops": 2 * seen * H * D}


def exact(case, seed):
    if work(case)["flops"] > 1.5e12:
        return None
    st = prepare(case, seed)
    return {"plan": _exact_plan, "tree": _exact_attend, "accept": _exact_accept,
            "weights": _exact_attend, "choose": _exact_choose, "keep": _exact_keep}[case["op"]](st, case)


def _exact_plan(st, case):
    rs, root, parent = (st[x].tolist() for x in ("row_start", "root", "parent"))
    mask, pos = [], []
    for b in range(case["batch"]):
        seen = []
        for i, p in enumerate(parent[rs[b]:rs[b + 1]]):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
            pos.append(root[b] + bin(seen[i]).count("1") - 1)
            words = [seen[i] >> 32 * w & 0xffffffff for w in range(st["words"])]
            mask.append([w - (w >> 31 << 32) for w in words])
    return {"mask": _i32(mask), "positions": _i32(pos)}


def _exact_accept(st, case):
    rs, root, parent, tok, post = (st[x].tolist() for x in
                                   ("row_start", "root", "parent", "tokens", "posterior"))
    n_max, res, weight = st["n_max"], [], [0.0] * rs[-1]
    for b in range(case["batch"]):
        s, n = rs[b], rs[b + 1] - rs[b]
        path = [0]
        while True:
            nxt = [c for c in range(1, n) if parent[s + c] == path[-1] and tok[s + c] == post[s + path[-1]]]
            if not nxt:
                break
            path.append(nxt[0])
        bonus = post[s + path[-1]]
        for r in path:
            weight[s + r] = 1.0
        out = [tok[s + r] for r in path[1:]] + [bonus]
        res.append((len(path) - 1, len(path), bonus, out + [0] * (n_max - len(out)),
                    path + [-1] * (n_max - len(path)), root[b] + len(path)))
    names = ("accept_len", "commit_len", "bonus", "out_tokens", "path", "seq_len")
    return {**{k: _i32([r[j] for r in res]) for j, k in enumerate(names)},
            "row_weight": torch.tensor(weight, dtype=torch.float64, device="cuda")}


def _exact_attend(st, case):
    rs, kv = st["row_start"].tolist(), st["kv_len"].tolist()
    G, D, prefix = case["heads"] // case["kvh"], case["dim"], case["prefix"]
    tree = case["op"] == "tree"
    parent = st["parent"].tolist() if case["tree"] else None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    acc = None if tree else st["weights"].double()
    for b in range(case["batch"]):
        n, total = rs[b + 1] - rs[b], kv[b] + rs[b + 1] - rs[b]
        skip = 0 if tree else prefix
        pages = st["table"][b] if skip or not prefix else torch.cat([st["prefix_pages"], st["table"][b]])
        k = st["k_pages"][pages.long()].flatten(0, 1)[:total - skip].double()
        v = st["v_pages"][pages.long()].flatten(0, 1)[:total - skip].double()
        hide = [[True] * n for _ in range(n)]
        for i in range(n):
            j = i
            while j >= 0:
                hide[i][j] = False
                j = parent[rs[b] + j] if parent else j - 1
        hidden = torch.zeros((n, total - skip), dtype=torch.bool, device="cuda")
        hidden[:, total - skip - n:] = torch.tensor(hide, device="cuda")
        if not tree:
            c = kv[b] - prefix
            acc[b, :, :c] = acc[b, :, :c] * case["decay"] if case["decay"] else 0.0
            acc[b, :, c:c + n] = 0.0
        for h in range(case["heads"]):
            s = st["q"][rs[b]:rs[b + 1], h].double() @ k[:, h // G].T / math.sqrt(D)
            s[hidden] = -math.inf
            if tree:
                out[rs[b]:rs[b + 1], h] = torch.softmax(s, -1) @ v[:, h // G]
                lse[rs[b]:rs[b + 1], h] = torch.logsumexp(s, -1)
                continue
            p = torch.exp(s - st["lse"][rs[b]:rs[b + 1], h, None].double())
            if st["row_weight"] is not None:
                p = p * st["row_weight"][rs[b]:rs[b + 1], None].double()
            acc[b, h // G, :total - skip] += p.sum(0)
    return {"out": out, "lse": lse} if tree else {"weights": acc}


def _exact_choose(st, case):
    B, KVH, keep = case["batch"], case["kvh"], case["keep"]
    rows = torch.full((B, KVH, keep), -1, dtype=torch.long)
    count = torch.zeros((B, KVH), dtype=torch.long)
    for b, n in enumerate(st["kv_len"].tolist()):
        a = min(case["first"], keep)
        z = min(case["last"], keep - a)
        for h in range(KVH):
            at = list(range(n))
            if n > keep:
                w = st["weights"][b, h, :n].tolist()
                middle = sorted(range(a, n - z), key=lambda i: (-w[i], i))[:keep - a - z]
                at = at[:a] + sorted(middle) + at[n - z:]
            rows[b, h, :len(at)] = torch.tensor(at)
            count[b, h] = len(at)
    return {"rows": rows.int().cuda(), "count": count.int().cuda()}


def _exact_keep(st, case):
    k, v = st["k_pages"].double(), st["v_pages"].double()
    w = None if case["path"] else st["weights"].double()
    for b in range(case["batch"]):
        first = int(st["first"][b]) if case["path"] else 0
        for h in range(case["kvh"]):
            lst = 0 if case["path"] else h
            c = int(st["count"][b, lst])
            src = st["rows"][b, lst, :c].long() + first
            dst = torch.arange(first, first + c, device="cuda")
            ps, pd = st["table"][b].long()[src // PAGE], st["table"][b].long()[dst // PAGE]
            k[pd, dst % PAGE, h] = k[ps, src % PAGE, h]
            v[pd, dst % PAGE, h] = v[ps, src % PAGE, h]
            if w is not None:
                w[b, h, :c] = w[b, h, src]
    return {"k_pages": k, "v_pages": v} if case["path"] else {"k_pages": k, "v_pages": v, "weights": w}
