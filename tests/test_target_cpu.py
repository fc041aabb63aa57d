"""Host side of the target-side calls: rotary plans against their formulas, and refusals before
any device work (arguments are checked before the handle's workspace)."""
import ctypes
import math

import pytest

import block_diffusion_speculative_fc_gb300 as pkg
from block_diffusion_speculative_fc_gb300 import _build
from synth import WORKLOADS

FAKE = 0x10000  # never dereferenced by host-side code


@pytest.fixture(scope="module")
def handle():
    _build.build()
    cfg = WORKLOADS["tiny"].cfg
    win = (ctypes.c_int32 * cfg.n_layers)(*cfg.sliding_window)
    c = pkg.DflashConfig(pkg.DFLASH_F32, cfg.target_hidden, cfg.n_sel, cfg.hidden, cfg.n_layers,
                         cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, cfg.intermediate, cfg.vocab,
                         cfg.mask_token_id, cfg.block_size, cfg.page_size,
                         ctypes.cast(win, ctypes.POINTER(ctypes.c_int32)), cfg.rms_eps,
                         cfg.rope_theta, 4, 256, 4096)
    arr = (ctypes.c_void_p * cfg.n_layers)(*([FAKE] * cfg.n_layers))
    P = ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))
    w = pkg.DflashWeights(FAKE, FAKE, FAKE, FAKE, FAKE, P, P, P, P, P, P, P, P)
    h = pkg.dflash_create(c, w)
    yield h
    pkg.dflash_destroy(h)


def plain_frequencies(rd, theta, scaling, factor, orig, low, high):
    out = []
    for i in range(rd // 2):
        f = theta ** (-2.0 * i / rd)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            s = min(1.0, max(0.0, (orig * f / (2 * math.pi) - low) / (high - low)))
            f *= (1 - s) / factor + s
        elif scaling == "yarn":
            c = lambda r: rd * math.log(orig / (2 * math.pi * r)) / (2 * math.log(theta))  # noqa: E731
            lo, hi = max(math.floor(c(high)), 0), min(math.ceil(c(low)), rd - 1)
            a = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f *= a / factor + 1 - a
        out.append(f)
    return out


@pytest.mark.parametrize("rd,theta", [(128, 1e6), (64, 1e4), (10, 5e5), (2, 2.0), (0, 1e6)])
@pytest.mark.parametrize("scaling,factor,orig,low,high",
                         [("none", 1.0, 0, 0, 0), ("linear", 4.0, 0, 0, 0),
                          ("bands", 8.0, 8192, 1, 4), ("yarn", 40.0, 4096, 1, 32),
                          ("yarn", 4.0, 32768, 2, 16)])
def test_rope_plan_frequencies(rd, theta, scaling, factor, orig, low, high):
    _build.build()
    r = pkg.rope_plan(rd, theta, scaling=scaling, factor=factor, original_positions=orig, low=low,
                      high=high)
    want = plain_frequencies(rd, theta, scaling, factor, orig, low, high)
    got = [t * 2 * math.pi / 2 ** 64 for t in r.turns[:rd // 2]]
    # both in double; a frequency is then cut to 2^-64 turn
    for g, w in zip(got, want):
        assert abs(g - w) <= 1e-13 * w + 2 ** -60
    assert list(r.turns[rd // 2:]) == [0] * (64 - rd // 2)
    amp = 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0
    assert abs(r.amplitude - amp) <= 2 ** -23 * amp


def test_rope_defaults_and_refusals():
    _build.build()
    assert list(pkg.rope_plan(64, 1e4, scaling="bands", factor=8, original_positions=8192).turns) == \
        list(pkg.rope_plan(64, 1e4, scaling="bands", factor=8, original_positions=8192, low=1,
                           high=4).turns)
    good = dict(rotary_dim=64, theta=1e4, scaling="yarn", factor=4.0, original_positions=4096)
    for bad in [dict(rotary_dim=63), dict(rotary_dim=130), dict(rotary_dim=-2), dict(theta=1.0),
                dict(theta=math.nan), dict(theta=math.inf), dict(factor=0.5), dict(factor=math.nan),
                dict(original_positions=0), dict(low=4, high=2), dict(low=-1)]:
        with pytest.raises(pkg.DFlashError):
            pkg.rope_plan(**{**good, **bad})
    with pytest.raises(KeyError):
        pkg.rope_plan(64, 1e4, scaling="other")


def layer(**over):
    kv = dict(dtype=pkg.DFLASH_BF16, n_heads=8, n_kv_heads=2, head_dim=128, k_pages=FAKE,
              v_pages=FAKE, n_pages=4, page_table=FAKE, pages_per_req=2, prefix_pages=None,
              prefix_len=0)
    return pkg.DflashLayerKV(*{**kv, **over}.values())


BAD_LAYERS = [dict(dtype=7), dict(head_dim=96), dict(head_dim=256), dict(n_heads=7), dict(n_heads=0),
              dict(n_heads=258), dict(n_heads=2048, n_kv_heads=1024), dict(n_kv_heads=0),
              dict(k_pages=None), dict(v_pages=None), dict(k_pages=FAKE + 8), dict(v_pages=FAKE + 2),
              dict(n_pages=0), dict(n_pages=1 << 26), dict(page_table=None), dict(pages_per_req=0),
              dict(prefix_len=64), dict(prefix_len=63, prefix_pages=FAKE),
              dict(prefix_len=-64, prefix_pages=FAKE)]


def refused(status, f, *a, **k):
    with pytest.raises(pkg.DFlashError) as e:
        f(*a, **k)
    assert e.value.status in (status if isinstance(status, tuple) else (status,)), e.value


def call_append(h, kv=None, batch=2, rows=4, row_start=FAKE, kv_len=FAKE, q=FAKE, qs=1024, k=FAKE,
                ks=256, v=FAKE, vs=256, qg=None, kg=None, eps=1e-6, rope=None, out=FAKE, os_=1024):
    rope = pkg.rope_plan(128, 1e6) if rope is None else rope
    pkg.dflash_append_kv(h, layer() if kv is None else kv, batch, rows, row_start, kv_len, q, qs, k,
                         ks, v, vs, qg, kg, eps, rope, out, os_, None)


def test_append_refusals(handle):
    refused(-6, call_append, handle)                       # every argument right: no workspace yet
    refused(-6, call_append, handle, rows=0)
    refused(-6, call_append, handle, q=None, out=None)
    for bad in BAD_LAYERS:
        refused((-1, -2), call_append, handle, kv=layer(**bad))
    for bad in [dict(row_start=None), dict(kv_len=None), dict(k=None), dict(v=None), dict(q=None),
                dict(out=None), dict(qs=1023), dict(ks=255), dict(vs=8), dict(os_=1000),
                dict(qs=1028), dict(ks=260), dict(vs=257), dict(os_=1025), dict(q=FAKE + 2),
                dict(k=FAKE + 8), dict(v=FAKE + 4), dict(out=FAKE + 8), dict(qg=FAKE + 2),
                dict(kg=FAKE + 8), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
                dict(batch=-1), dict(rows=-1), dict(q=None, out=None, qg=FAKE),
                dict(kv=layer(head_dim=64))]:
        refused(-1, call_append, handle, **bad)
    refused(-3, call_append, handle, batch=1025)
    refused(-3, call_append, handle, rows=1 << 28)
    refused(-1, call_append, None)
    assert pkg.load_library().dflash_append_kv(handle, None, 1, 1, FAKE, FAKE, None, 0, FAKE, 256,
                                               FAKE, 256, None, None, 0.0, pkg.rope_plan(64, 1e4),
                                               None, 0, None) == -1


def call_attend(h, kv=None, batch=2, rows=4, row_start=FAKE, kv_len=FAKE, q=FAKE, qs=1024, scale=0.1,
                causal=1, out=2 * FAKE, os_=1024, ws=FAKE, nbytes=1 << 40):
    pkg.dflash_paged_attention(h, layer() if kv is None else kv, batch, rows, row_start, kv_len, q,
                               qs, scale, causal, out, os_, ws, nbytes, None)


def test_attention_refusals(handle):
    refused(-6, call_attend, handle)
    refused(-6, call_attend, handle, rows=0)
    for bad in BAD_LAYERS:
        refused((-1, -2), call_attend, handle, kv=layer(**bad))
        refused((-1, -2), pkg.dflash_paged_attention_workspace_size, layer(**bad), 2, 4)
    for bad in [dict(row_start=None), dict(kv_len=None), dict(q=None), dict(out=None),
                dict(out=FAKE), dict(qs=1000), dict(os_=8), dict(qs=1028), dict(os_=1025),
                dict(q=FAKE + 4), dict(out=2 * FAKE + 8), dict(ws=None), dict(ws=FAKE + 16),
                dict(scale=math.nan), dict(scale=math.inf), dict(causal=2), dict(batch=-1)]:
        refused(-1, call_attend, handle, **bad)
    need = pkg.dflash_paged_attention_workspace_size(layer(), 2, 4)
    refused(-3, call_attend, handle, nbytes=need - 1)
    refused(-3, call_attend, handle, batch=1025)
    refused(-1, call_attend, None)


def call_probs(h, rows=4, vocab=100, logits=FAKE, dtype=pkg.DFLASH_BF16, ld=100, sp=None,
               probs=1 << 30):
    sp = pkg.DflashSampling(None, None, None, None, 2) if sp is None else sp
    pkg.dflash_target_probs(h, rows, vocab, logits, dtype, ld, sp, probs, None)


def call_sample(h, rows=4, vocab=100, logits=FAKE, dtype=pkg.DFLASH_BF16, ld=100, sp=None,
                noise=FAKE, ids=FAKE):
    sp = pkg.DflashSampling(None, None, None, None, 2) if sp is None else sp
    pkg.dflash_sample_tokens(h, rows, vocab, logits, dtype, ld, sp, noise, ids, None, None)


def test_sampling_refusals(handle):
    for call in (call_probs, call_sample):
        refused(-6, call, handle)
        refused(-6, call, handle, rows=0)
        for bad in [dict(rows=-1), dict(vocab=0), dict(logits=None), dict(logits=FAKE + 1),
                    dict(ld=99), dict(sp=pkg.DflashSampling(None, None, None, None, 0)),
                    dict(sp=pkg.DflashSampling(None, None, None, None, 3))]:
            refused(-1, call, handle, **bad)
        refused(-2, call, handle, dtype=2)
        refused(-2, call, handle, vocab=524289, ld=1 << 20)
        refused(-2, call, handle, vocab=262145, ld=1 << 20, dtype=pkg.DFLASH_F32)
        refused(-3, call, handle, rows=(1 << 24) + 2)
        refused(-1, call, None)
    for bad in [dict(probs=None), dict(probs=(1 << 30) + 2), dict(probs=FAKE),
                dict(probs=FAKE - 1600 + 4)]:
        refused(-1, call_probs, handle, **bad)
    refused(-6, call_probs, handle, probs=FAKE - 1600)     # ends where the logits begin
    refused(-1, call_sample, handle, noise=None)
    refused(-1, call_sample, handle, ids=None)


def test_misaligned_arrays_and_overlapping_outputs_are_refused(handle):
    for bad in [dict(row_start=FAKE + 2), dict(kv_len=FAKE + 1), dict(os_=1032),
                dict(kv=layer(page_table=FAKE + 2)),
                dict(kv=layer(prefix_len=64, prefix_pages=FAKE + 1))]:
        refused(-1, call_append, handle, **bad)
    refused(-6, call_append, handle, os_=1032, rows=1)      # one row: the stride is not used
    for bad in [dict(row_start=FAKE + 2), dict(kv_len=FAKE + 1), dict(kv=layer(page_table=FAKE + 2)),
                dict(kv=layer(prefix_len=64, prefix_pages=FAKE + 1))]:
        refused(-1, call_attend, handle, **bad)
    for call in (call_probs, call_sample):
        for i in range(4):
            sp = pkg.DflashSampling(*[FAKE + 2 * (i == j) for j in range(4)], 2)
            refused(-1, call, handle, sp=sp)
    refused(-1, call_sample, handle, noise=FAKE + 2)
    refused(-1, call_sample, handle, ids=FAKE + 1)
