"""Measured operators of the target's side of a draft-verify cycle.

append  per-head RMSNorm of queries and keys, rotary positions, and the append of the new K/V rows
        to one layer's paged cache (dflash_append_kv)
attend  attention of the new rows over that cache, with a prefix that the whole batch shares
        (dflash_paged_attention)
probs   the target's sampling distribution from its logits: temperature, top-k, top-p, min-p
        (dflash_target_probs), the input of the sampled verification
sample  tokens drawn from that distribution with given Exp(1) variates (dflash_sample_tokens)

Shapes are those of this repository's workloads (32 or 64 query heads, 8 KV heads of 128, blocks
of 8 or 16, vocabularies 151936 and 163840) and generic ones around them.
"""
import math

import torch

own = False

PAGE = 64
EPS = 1e-6


def _append(name, lens, ctx, heads=32, kvh=8, dim=128, dtype="bf16", norm=True, rot=None,
            inter=False, scaling="none", packed=True):
    """lens [lo, hi, batch]: new rows per request; ctx [lo, hi]: rows already in the cache."""
    return {"name": name, "op": "append", "batch": lens[2], "n_lo": lens[0], "n_hi": lens[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "heads": heads, "kvh": kvh, "dim": dim,
            "dtype": dtype, "norm": norm, "rot": dim if rot is None else rot, "inter": inter,
            "scaling": scaling, "packed": packed}


def _attend(name, lens, ctx, prefix=0, heads=32, kvh=8, dim=128, causal=True, dtype="bf16"):
    return {"name": name, "op": "attend", "batch": lens[2], "n_lo": lens[0], "n_hi": lens[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "prefix": prefix, "heads": heads, "kvh": kvh,
            "dim": dim, "causal": causal, "dtype": dtype}


def _logits(name, op, batch, block, vocab, mode, dtype="bf16"):
    return {"name": name, "op": op, "batch": batch, "block": block, "vocab": vocab, "mode": mode,
            "dtype": dtype}


def listed():
    return [
        # one request decoding one token without drafting: the smallest call of every layer
        _append("append-token-b1", [1, 1, 1], [1024, 1024]),
        # the verify block of the largest benchmark workload, 128 requests x 16 rows
        _append("append-verify-b128", [16, 16, 128], [64, 8000]),
        # ragged prompts of 16k rows in all, 64 heads, long-context scaling, interleaved pairs on
        # half of the head, no head norms
        _append("append-prompts-16k", [40, 3999, 8], [0, 200], heads=64, norm=False, rot=64,
                inter=True, scaling="yarn", packed=False),
        # one request, one token, a short context: latency
        _attend("attend-token-b1", [1, 1, 1], [1000, 1000]),
        # verification of 32 requests x 16 rows that share a system prompt of 8k rows
        _attend("attend-verify-b32-shared", [16, 16, 32], [256, 4096], prefix=8192),
        # 64 samples of one 16k prompt decoded a token at a time (64 query heads)
        _attend("attend-token-b64-shared", [1, 1, 64], [33, 2048], prefix=16384, heads=64),
        # two ragged prompts, causal prefill, no cache before them
        _attend("attend-prompts", [2500, 4096, 2], [0, 0]),
        # one request's verify block of 16 rows: top-k and top-p
        _logits("probs-b1-s16", "probs", 1, 16, 151936, "topk_topp"),
        # the largest workload's verify block, every kind of request in one batch
        _logits("probs-b128-s16", "probs", 128, 16, 151936, "mix"),
        # an odd vocabulary in fp32, nucleus only
        _logits("probs-odd-fp32", "probs", 12, 8, 50257, "topp", dtype="f32"),
        # the first token after one prompt
        _logits("sample-b1", "sample", 1, 1, 151936, "topk_topp"),
        # the first tokens of 128 prompts, every kind of request
        _logits("sample-b128", "sample", 128, 1, 163840, "mix"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "probs", "sample"])
    if op == "append":
        dim = rng.choice([64, 128, 128])
        kvh = rng.choice([1, 2, 4, 8])
        batch = _log(rng, 1, 128)
        top = max(1, min(4000, 16000 // batch))
        hi = _log(rng, 1, top)
        return _append(None, [max(1, hi // rng.choice([1, 2, 5])), hi, batch],
                       [rng.randint(0, 100), _log(rng, 100, 20000)],
                       heads=kvh * rng.choice([1, 4, 5, 8]), kvh=kvh, dim=dim,
                       dtype=rng.choice(["bf16", "bf16", "f32"]), norm=rng.random() < 0.6,
                       rot=rng.choice([dim, dim, dim // 2, dim // 4, 10]),
                       inter=rng.random() < 0.4,
                       scaling=rng.choice(["none", "linear", "bands", "yarn"]),
                       packed=rng.random() < 0.5)
    if op == "attend":
        kvh = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 4, 5, 8])
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, min(1024, 2048 // batch)))
        prefix = PAGE * _log(rng, 1, 256) if rng.random() < 0.5 else 0
        c_hi = _log(rng, 10, 4000)
        return _attend(None, [max(1, hi // rng.choice([1, 3])), hi, batch],
                       [rng.randint(0, c_hi), c_hi], prefix=prefix, heads=kvh * group, kvh=kvh,
                       dim=rng.choice([64, 128, 128]), causal=rng.random() < 0.8)
    batch = _log(rng, 1, 128)
    vocab = rng.choice([151936, 163840, _log(rng, 500, 160000), _log(rng, 500, 160000)])
    dtype = rng.choice(["bf16", "f32"])
    block = rng.choice([1, 8, 16]) if op == "probs" else 1
    if dtype == "f32":      # no dearer than the largest bf16 call
        batch = max(1, min(batch, 1400 * 163840 // (block * vocab)))
    if dtype == "bf16" and block == 16:
        vocab = min(vocab, 151936)
    return _logits(None, op, batch, block, vocab,
                   rng.choice(["topk_topp", "topp", "minp", "none", "mix"]), dtype=dtype)


# ---------------------------------------------------------------- inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _spread(lo, hi, n):
    """n whole numbers spread evenly over lo..hi: their sum does not go by the seed."""
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _lens(case):
    return _spread(case["n_lo"], case["n_hi"], case["batch"]), \
        _spread(case["ctx_lo"], case["ctx_hi"], case["batch"])


def _frequencies(rot, scaling):
    """Angles per position in 64 bits: base 1e6; scaled ones stretch 8192 positions 8 times."""
    n = rot // 2
    inv = [1e6 ** (-2.0 * i / rot) for i in range(n)]
    factor, orig, amp = 8.0, 8192.0, 1.0
    if scaling == "linear":
        inv = [f / factor for f in inv]
    elif scaling == "bands":    # low factor 1, high factor 4
        out = []
        for f in inv:
            turns = orig * f / (2 * math.pi)
            s = min(1.0, max(0.0, (turns - 1.0) / 3.0))
            out.append(f * ((1 - s) / factor + s))
        inv = out
    elif scaling == "yarn":     # fast 32, slow 1
        def at(r):
            return rot * math.log(orig / (r * 2 * math.pi)) / (2 * math.log(1e6))
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        out = []
        for i, f in enumerate(inv):
            ramp = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            out.append(f * (ramp / factor + (1 - ramp)))
        inv = out
        amp = 0.1 * math.log(factor) + 1.0
    return inv, amp


def _session():
    """A draft session of a tiny model: what holds the handle that the calls take."""
    from types import SimpleNamespace

    import block_diffusion_speculative_fc_gb300 as pkg
    cfg = SimpleNamespace(dtype="f32", target_hidden=128, n_sel=1, hidden=128, n_layers=1,
                          n_heads=2, n_kv_heads=1, head_dim=64, intermediate=128, vocab=256,
                          mask_token_id=255, block_size=2, page_size=PAGE, sliding_window=(0,),
                          rms_eps=EPS, rope_theta=1e6)
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    W = {"fc": z(128, 128), "hidden_norm": z(128), "final_norm": z(128), "embed": z(256, 128),
         "lm_head": z(256, 128),
         "layers": [{"qkv": z(256, 128), "o": z(128, 128), "gate_up": z(256, 128),
                     "down": z(128, 128), "in_norm": z(128), "post_norm": z(128), "q_norm": z(64),
                     "k_norm": z(64)}]}
    return pkg, pkg.DraftSession(cfg, W, max_batch=1, max_rows=16, max_position=64)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    if case["op"] in ("probs", "sample"):
        return _prepare_logits(case, g)
    dt, B, D, H, KVH = _dt(case), case["batch"], case["dim"], case["heads"], case["kvh"]
    n, ctx = _lens(case)
    order = torch.randperm(B, generator=g, device="cuda").tolist()
    n, ctx = [n[i] for i in order], [ctx[i] for i in order]
    prefix = case.get("prefix", 0)
    starts = [0]
    for v in n:
        starts.append(starts[-1] + v)
    T = starts[-1]
    need = [(c + v + PAGE - 1) // PAGE for c, v in zip(ctx, n)]
    width = max(need)
    used, n_prefix = sum(need), prefix // PAGE
    pool = torch.randperm(used + n_prefix, generator=g, device="cuda").to(torch.int32)
    rank = torch.arange(width, device="cuda")
    need_t = torch.tensor(need, device="cuda")
    mine = rank[None] < need_t[:, None]
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    table[mine] = pool[:used]
    st = {"case": case, "T": T, "prefix": prefix, "table": table, "prefix_pages": pool[used:],
          "row_start": torch.tensor(starts, dtype=torch.int32, device="cuda"),
          "kv_len": torch.tensor([prefix + c for c in ctx], dtype=torch.int32, device="cuda"),
          "n_max": max(n)}

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)

    pages = (used + n_prefix, PAGE, KVH, D)
    if case["op"] == "append":
        st["k_pages"], st["v_pages"] = (torch.zeros(pages, dtype=dt, device="cuda") for _ in "kv")
        if case["packed"]:      # the rows of one fused projection
            qkv = normal(T, (H + 2 * KVH) * D)
            st["q"], st["k"], st["v"] = (
                t.unflatten(1, (-1, D)) for t in qkv.split([H * D, KVH * D, KVH * D], dim=1))
        else:
            st["q"], st["k"], st["v"] = normal(T, H, D), normal(T, KVH, D), normal(T, KVH, D)
        gain = lambda: (0.5 + torch.rand(D, generator=g, device="cuda")).to(dt)  # noqa: E731
        st["q_gain"], st["k_gain"] = (gain(), gain()) if case["norm"] else (None, None)
        inv, amp = _frequencies(case["rot"], case["scaling"])
        st["inv"], st["amp"] = torch.tensor(inv, dtype=torch.float64, device="cuda"), amp
        st["q_out"] = torch.empty((T, H, D), dtype=dt, device="cuda")
    else:
        # head-normed queries and keys: logits of a few units, a few keys that stand out
        st["q"] = normal(T, H, D, scale=1.5)
        st["k_pages"], st["v_pages"] = normal(*pages), normal(*pages)
        st["out"] = torch.empty((T, H, D), dtype=dt, device="cuda")
    if own:
        pkg, sess = _session()
        st["sess"] = sess
        st["layer"] = pkg.LayerKV(H, st["k_pages"], st["v_pages"], table,
                                  prefix_pages=st["prefix_pages"] if prefix else None)
        if case["op"] == "append":
            st["rope"] = pkg.rope_plan(case["rot"], 1e6, interleaved=case["inter"],
                                       scaling=case["scaling"], factor=8.0,
                                       original_positions=8192)
        else:
            st["ws"] = sess.attention_workspace(st["layer"], B, T)
    return st


def _prepare_logits(case, g):
    B, S, V = case["batch"], case["block"], case["vocab"]
    R = B * S
    x = torch.empty((R, V), dtype=_dt(case), device="cuda")
    step = max(1, (1 << 27) // V)
    for r in range(0, R, step):
        m = min(step, R - r)
        y = torch.randn((m, V), generator=g, device="cuda") * 2.5
        # a model's logits: a few tokens stand out of the bulk
        top = torch.randint(0, V, (m, 32), generator=g, device="cuda")
        y.scatter_add_(1, top, 14 * torch.rand((m, 32), generator=g, device="cuda"))
        x[r:r + m] = y.to(x.dtype)
    x[:, V - V // 100:] = torch.finfo(x.dtype).min    # the padding rows of the output head
    kinds = {"topk_topp": [0], "topp": [1], "minp": [2], "none": [3], "mix": [0, 1, 2, 3, 4]}
    kind = [kinds[case["mode"]][b % len(kinds[case["mode"]])] for b in range(B)]
    f = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    st = {"case": case, "logits": x,
          "temperature": f([(0.6, 0.8, 1.0, 1.0, 0.0)[k] for k in kind]),
          "top_k": torch.tensor([(20 + b % 40, 0, 0, 0, 0)[k] for b, k in enumerate(kind)],
                                dtype=torch.int32, device="cuda"),
          "top_p": f([(0.95, 0.9, 1.0, 1.0, 1.0)[k] for k in kind]),
          "min_p": f([(0.0, 0.0, 0.05, 0.0, 0.0)[k] for k in kind])}
    if case["op"] == "probs":
        st["probs"] = torch.empty((R, V), dtype=torch.float32, device="cuda")
    else:
        st["noise"] = torch.empty((R, V), device="cuda").exponential_(generator=g)
        st["noise"].clamp_(min=1e-30)
        st["ids"] = torch.empty(R, dtype=torch.int32, device="cuda")
        st["prob"] = torch.empty(R, dtype=torch.float32, device="cuda")
    if own:
        st["sess"] = _session()[1]
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        s = st["sess"]
        if op == "append":
            s.append_kv(st["layer"], st["q"], st["k"], st["v"], st["row_start"], st["kv_len"],
                        st["rope"], q_gain=st["q_gain"], k_gain=st["k_gain"], eps=EPS,
                        q_out=st["q_out"])
            return {"q": st["q_out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
        if op == "attend":
            s.paged_attention(st["layer"], st["q"], st["row_start"], st["kv_len"], st["out"],
                              st["ws"], causal=st["case"]["causal"])
            return {"out": st["out"]}
        params = {k: st[k] for k in ("temperature", "top_k", "top_p", "min_p")}
        if op == "probs":
            s.target_probs(st["logits"], st["probs"], **params)
            return {"probs": st["probs"]}
        s.sample_tokens(st["logits"], st["noise"], st["ids"], prob=st["prob"], **params)
        return {"ids": st["ids"], "prob": st["prob"]}
    if op == "append":
        return _plain_append(st)
    if op == "attend":
        return {"out": _plain_attend(st)}
    return _plain_probs(st)


def _rows(st):
    """Request and position of every new row."""
    rs = st["row_start"].long()
    b = torch.repeat_interleave(torch.arange(len(rs) - 1, device="cuda"), rs[1:] - rs[:-1],
                                output_size=st["T"])
    return b, st["kv_len"].long()[b] + torch.arange(st["T"], device="cuda") - rs[b]


def _plain_rope(x, gain, cos, sin, case):
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.float()
    rot, half = case["rot"], case["rot"] // 2
    if case["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_append(st):
    case = st["case"]
    b, pos = _rows(st)
    ang = pos.double()[:, None] * st["inv"]
    cos, sin = (ang.cos() * st["amp"]).float()[:, None], (ang.sin() * st["amp"]).float()[:, None]
    q = _plain_rope(st["q"], st["q_gain"], cos, sin, case).to(st["q"].dtype)
    k = _plain_rope(st["k"], st["k_gain"], cos, sin, case).to(st["k"].dtype)
    page = st["table"].long()[b, pos // PAGE]
    st["k_pages"][page, pos % PAGE] = k
    st["v_pages"][page, pos % PAGE] = st["v"]
    return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _plain_attend(st):
    case, T, prefix = st["case"], st["T"], st["prefix"]
    H, KVH, D = case["heads"], case["kvh"], case["dim"]
    G, B, n_max = H // KVH, case["batch"], st["n_max"]
    rs = st["row_start"].long()
    b, pos = _rows(st)
    i = torch.arange(T, device="cuda") - rs[b]
    last = pos if case["causal"] else (st["kv_len"].long() + rs[1:] - rs[:-1] - 1)[b]
    q = st["q"].float() * D ** -0.5
    # the requests' own rows: queries padded to the longest block, keys to the longest context
    qo = torch.zeros((B, n_max, H, D), device="cuda")
    qo[b, i] = q
    lo = torch.full((B, n_max), -1, device="cuda", dtype=torch.long)
    lo[b, i] = last
    table = st["table"].long()
    k = st["k_pages"][table].float().flatten(1, 2)     # [B, keys, KVH, D]
    v = st["v_pages"][table].float().flatten(1, 2)
    keys = torch.arange(k.shape[1], device="cuda") + prefix
    qo = qo.view(B, n_max, KVH, G, D).permute(0, 2, 1, 3, 4).reshape(B, KVH, n_max * G, D)
    s = qo @ k.permute(0, 2, 3, 1)
    seen = (keys <= lo[:, :, None]).repeat_interleave(G, dim=1)[:, None]
    s = s.masked_fill(~seen, -math.inf)
    v = v.masked_fill((keys > lo.amax(1)[:, None])[:, :, None, None], 0.0)
    m = s.amax(-1, keepdim=True)
    if prefix:
        page = st["prefix_pages"].long()
        kp, vp = (st[n][page].float().flatten(0, 1).permute(1, 0, 2) for n in ("k_pages", "v_pages"))
        sp = q.view(T, KVH, G, D).permute(1, 0, 2, 3).reshape(KVH, T * G, D) @ kp.transpose(1, 2)
        mp = sp.amax(-1).view(KVH, T, G)
        mo = m.view(B, KVH, n_max, G)
        mo[b, :, i] = torch.maximum(mo[b, :, i], mp.permute(1, 0, 2))
        m = mo.reshape(B, KVH, n_max * G, 1)
    e = torch.exp(s - m.clamp(min=-1e30))
    den = e.sum(-1).view(B, KVH, n_max, G)[b, :, i]    # [T, KVH, G]
    out = (e @ v.permute(0, 2, 1, 3)).view(B, KVH, n_max, G, D)[b, :, i]
    if prefix:
        mt = m.view(B, KVH, n_max, G)[b, :, i].permute(1, 0, 2).reshape(KVH, T * G, 1)
        ep = torch.exp(sp - mt)
        den = den + ep.sum(-1).view(KVH, T, G).permute(1, 0, 2)
        out = out + (ep @ vp).view(KVH, T, G, D).permute(1, 0, 2, 3)
    return (out / den[..., None]).reshape(T, H, D).to(st["q"].dtype)


def _plain_probs(st):
    x = st["logits"].float()
    R, V = x.shape
    per = lambda t: t.repeat_interleave(R // len(t))[:, None]  # noqa: E731
    T, k = per(st["temperature"]), per(st["top_k"]).long()
    p, mp = per(st["top_p"]).double(), per(st["min_p"]).double()
    x = x.masked_fill(x.isnan(), -math.inf).clamp_(max=torch.finfo(torch.float32).max)
    sx, at = x.sort(dim=-1, descending=True, stable=True)
    rank = torch.arange(V, device="cuda")
    # borders (mass before a token against p, weight against min-p) in 64 bits
    w64 = torch.exp((sx.double() - sx[:, :1].double()) / T.double().clamp(min=1e-30))
    w64.masked_fill_(sx == -math.inf, 0.0)
    w64.masked_fill_((rank >= k) & (k > 0), 0.0)
    before = w64.cumsum(-1)
    total = before[:, -1:].clone()
    before -= w64
    keep = ((before < p * total) | (p >= 1) | (rank == 0)) & (w64 >= mp) & (sx > -math.inf)
    keep &= ((rank < k) | (k <= 0)) & ((rank == 0) | (T > 0))
    del before
    w = torch.where(keep, w64, 0.0).float()
    del w64
    prob = w / w.sum(-1, keepdim=True)
    if st["case"]["op"] == "probs":
        return {"probs": torch.zeros_like(x).scatter_(1, at, prob)}
    won = (torch.zeros_like(x).scatter_(1, at, w) / st["noise"]).argmax(-1, keepdim=True)
    drawn = torch.zeros_like(x).scatter_(1, at, prob).gather(1, won)
    return {"ids": won[:, 0].int(), "prob": drawn[:, 0]}


# ---------------------------------------------------------------- floors and 64-bit values
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("probs", "sample"):
        R, V = case["batch"] * case["block"], case["vocab"]
        if case["op"] == "probs":
            return {"bytes": R * V * (es + 4), "flops": 4 * R * V}
        # the variates of unfiltered requests are read whole, the others' only where kept
        whole = {"none": R, "mix": sum(b % 5 == 3 for b in range(case["batch"]))}.get(case["mode"], 0)
        return {"bytes": R * V * es + whole * V * 4 + R * 8, "flops": 4 * R * V}
    n, ctx = _lens(case)
    H, KVH, D = case["heads"], case["kvh"], case["dim"]
    T = sum(n)
    if case["op"] == "append":
        return {"bytes": 2 * T * (H + 2 * KVH) * D * es, "flops": 8 * T * (H + KVH) * D}
    keys = case["prefix"] + sum(n) + sum(ctx)
    if case["causal"]:
        seen = sum(v * (case["prefix"] + c) + v * (v + 1) // 2 for v, c in zip(n, ctx))
    else:
        seen = sum(v * (case["prefix"] + c + v) for v, c in zip(n, ctx))
    return {"bytes": 2 * keys * KVH * D * es + 2 * T * H * D * es, "flops": 4 * seen * H * D}


def exact(case, seed):
    if case["op"] == "attend" and work(case)["flops"] > 1.5e12:
        return None
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "probs": _exact_probs,
            "sample": _exact_probs}[case["op"]](st, case)


def _exact_append(st, case):
    rs, kv = st["row_start"].tolist(), st["kv_len"].tolist()
    rot, half = case["rot"], case["rot"] // 2
    if case["inter"]:
        i0 = torch.arange(half, device="cuda") * 2
        i1 = i0 + 1
    else:
        i0 = torch.arange(half, device="cuda")
        i1 = i0 + half
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    q_out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        rows = slice(rs[b], rs[b + 1])
        pos = torch.arange(kv[b], kv[b] + rs[b + 1] - rs[b], device="cuda")
        turn = torch.polar(torch.full((len(pos), half), st["amp"], dtype=torch.float64, device="cuda"),
                           torch.outer(pos.double(), st["inv"]))[:, None]

        def turned(x, gain):
            x = x[rows].double()
            if gain is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * gain.double()
            z = torch.complex(x[..., i0], x[..., i1]) * turn
            x = x.clone()
            x[..., i0], x[..., i1] = z.real, z.imag
            return x

        q_out[rows] = turned(st["q"], st["q_gain"])
        page = st["table"][b].long()[torch.div(pos, PAGE, rounding_mode="floor")]
        kp[page, pos % PAGE] = turned(st["k"], st["k_gain"])
        vp[page, pos % PAGE] = st["v"][rows].double()
    return {"q": q_out, "k_pages": kp, "v_pages": vp}


def _exact_attend(st, case):
    rs, kv = st["row_start"].tolist(), st["kv_len"].tolist()
    G, D, prefix = case["heads"] // case["kvh"], case["dim"], st["prefix"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        n = rs[b + 1] - rs[b]
        pages = torch.cat([st["prefix_pages"], st["table"][b]]).long()
        total = kv[b] + n
        k = st["k_pages"][pages].flatten(0, 1)[:total].double()
        v = st["v_pages"][pages].flatten(0, 1)[:total].double()
        row = torch.arange(n, device="cuda") + kv[b] if case["causal"] else \
            torch.full((n,), total - 1, device="cuda")
        hidden = torch.arange(total, device="cuda")[None] > row[:, None]
        for h in range(case["heads"]):
            s = st["q"][rs[b]:rs[b + 1], h].double() @ k[:, h // G].T / math.sqrt(D)
            s[hidden] = -math.inf
            out[rs[b]:rs[b + 1], h] = torch.softmax(s, -1) @ v[:, h // G]
    return {"out": out}


def _exact_probs(st, case):
    x = st["logits"]
    R, V = x.shape
    per = R // len(st["top_k"])
    probs = torch.zeros((R, V), dtype=torch.float64, device="cuda")
    temps, ks, ps, ms = (st[n].tolist() for n in ("temperature", "top_k", "top_p", "min_p"))
    for r in range(R):
        e = r // per
        row = x[r].double()
        idx = torch.argsort(row, descending=True, stable=True)
        if temps[e] == 0:
            probs[r, idx[0]] = 1.0
            continue
        if ks[e] > 0:
            idx = idx[:ks[e]]
        q = torch.softmax(row[idx] / temps[e], 0)
        if ps[e] < 1:
            idx = idx[:max(1, int((q.cumsum(0) - q < ps[e]).sum()))]
        q = torch.softmax(row[idx] / temps[e], 0)
        idx = idx[q >= ms[e] * q[0]]
        probs[r, idx] = torch.softmax(row[idx] / temps[e], 0)
    if case["op"] == "probs":
        return {"probs": probs}
    won = (probs / st["noise"].double()).argmax(-1)
    return {"ids": None, "prob": probs.gather(1, won[:, None])[:, 0]}
