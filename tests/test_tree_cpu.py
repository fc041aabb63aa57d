"""Refusals of the tree and eviction calls before any device work, and the exported names."""
import math

import pytest

import block_diffusion_speculative_fc_gb300 as pkg
from tests.test_target_cpu import BAD_LAYERS, FAKE, handle, layer, refused  # noqa: F401

BIG = 1 << 40


def plan(h, batch=2, rows=8, row_start=FAKE, parent=FAKE, root=FAKE, words=1, mask=FAKE, positions=FAKE):
    pkg.dflash_tree_plan(h, batch, rows, row_start, parent, root, words, mask, positions, None)


def append(h, kv=None, batch=2, rows=4, row_start=FAKE, kv_len=FAKE, positions=FAKE, q=FAKE, k=FAKE):
    pkg.dflash_append_kv_at(h, layer() if kv is None else kv, batch, rows, row_start, kv_len, positions, q, 1024, k,
                            256, FAKE, 256, None, None, 1e-6, pkg.rope_plan(128, 1e6), FAKE, 1024, None)


def attend(h, kv=None, batch=2, rows=4, row_start=FAKE, kv_len=FAKE, mask=FAKE, words=1, q=FAKE, qs=1024, scale=0.1,
           out=2 * FAKE, os_=1024, lse=FAKE, ws=FAKE, nbytes=BIG):
    pkg.dflash_tree_attention(h, layer() if kv is None else kv, batch, rows, row_start, kv_len, mask, words, q, qs,
                              scale, out, os_, lse, ws, nbytes, None)


def accept(h, batch=2, rows=8, row_start=FAKE, parent=FAKE, tokens=FAKE, posterior=FAKE, most=4, seq=FAKE, acc=FAKE,
           com=FAKE, bonus=FAKE, out=FAKE, path=FAKE, weight=None, ids=None, stride=0):
    pkg.dflash_accept_commit_tree(h, batch, rows, row_start, parent, tokens, posterior, most, seq, acc, com, bonus, out,
                                  path, weight, ids, stride, None)


def weigh(h, kv=None, batch=2, rows=4, row_start=FAKE, kv_len=FAKE, mask=None, words=0, q=FAKE, qs=1024, scale=0.1,
          lse=FAKE, row_weight=None, decay=1.0, weights=FAKE, width=100):
    pkg.dflash_key_weights(h, layer() if kv is None else kv, batch, rows, row_start, kv_len, mask, words, q, qs, scale,
                           lse, row_weight, decay, weights, width, None)


def choose(h, kv=None, batch=2, kv_len=FAKE, weights=FAKE, width=100, keep=FAKE, first=0, last=0, most=10, rows=FAKE,
           count=FAKE):
    pkg.dflash_choose_rows(h, layer() if kv is None else kv, batch, kv_len, weights, width, keep, first, last, most,
                           rows, count, None)


def keep(h, kv=None, batch=2, first=None, lists=1, most=10, rows=FAKE, count=FAKE, weights=None, width=0):
    pkg.dflash_keep_rows(h, layer() if kv is None else kv, batch, first, lists, most, rows, count, weights, width, None)


CALLS = [plan, append, attend, accept, weigh, choose, keep]


def test_good_arguments_ask_for_the_workspace(handle):  # noqa: F811
    for call in CALLS:
        refused(-6, call, handle)
        refused(-6, call, handle, batch=0)
        refused(-1, call, None)
        refused(-1, call, handle, batch=-1)
        refused(-3, call, handle, batch=1025)
    for call in (plan, append, attend, accept, weigh):
        refused(-6, call, handle, rows=0)
        refused(-1, call, handle, rows=-1)
        refused(-3, call, handle, rows=(1 << 28) + 1)
    for call in (append, attend, weigh, choose, keep):
        for bad in BAD_LAYERS:
            refused((-1, -2), call, handle, kv=layer(**bad))


def test_pointers(handle):  # noqa: F811
    need = {plan: ["row_start", "parent", "root", "mask"], append: ["row_start", "kv_len", "positions", "k"],
            attend: ["row_start", "kv_len", "q", "out", "ws"],
            accept: ["row_start", "parent", "tokens", "posterior", "seq", "acc", "com", "bonus", "out", "path"],
            weigh: ["row_start", "kv_len", "q", "lse", "weights"],
            choose: ["kv_len", "weights", "keep", "rows", "count"], keep: ["rows", "count"]}
    more = {plan: ["positions"], attend: ["lse", "mask"], accept: ["weight"], weigh: ["row_weight"], keep: ["first"]}
    for call, names in need.items():
        for n in names:
            refused(-1, call, handle, **{n: None})
        for n in names + more.get(call, []):
            refused(-1, call, handle, **{n: FAKE + 2})
    refused(-1, weigh, handle, mask=FAKE + 2, words=1)
    refused(-1, accept, handle, ids=FAKE + 2, stride=9)
    refused(-1, keep, handle, weights=FAKE + 2, width=9)
    refused(-6, plan, handle, positions=None)
    refused(-6, attend, handle, lse=None)


def test_sizes(handle):  # noqa: F811
    for words in (0, -1, 33):
        refused(-2, plan, handle, words=words)
        refused(-1, attend, handle, words=words)
        refused(-1, weigh, handle, mask=FAKE, words=words)
    refused(-6, attend, handle, words=32)
    refused(-1, attend, handle, mask=None)                  # words without a mask
    refused(-6, attend, handle, mask=None, words=0)
    refused(-1, attend, handle, out=FAKE)
    for call in (attend, weigh):
        for bad in [dict(scale=math.nan), dict(scale=math.inf), dict(qs=1000), dict(qs=1028), dict(q=FAKE + 8)]:
            refused(-1, call, handle, **bad)
    for bad in [dict(os_=8), dict(os_=1025), dict(out=2 * FAKE + 8), dict(ws=FAKE + 16)]:
        refused(-1, attend, handle, **bad)
    need = pkg.dflash_paged_attention_workspace_size(layer(), 2, 4)
    refused(-3, attend, handle, nbytes=need - 1)
    refused(-6, attend, handle, nbytes=need)
    for most in (0, -1, 1025):
        refused(-2, accept, handle, most=most)
    refused(-1, accept, handle, ids=FAKE, stride=0)
    refused(-2, weigh, handle, scale=2.0 ** -101)
    refused(-2, weigh, handle, scale=-2.0 ** 101)
    for scale in (0.0, 2.0 ** -100, -2.0 ** 100):
        refused(-6, weigh, handle, scale=scale)
    for bad in [dict(decay=-0.1), dict(decay=1.1), dict(decay=math.nan), dict(width=0)]:
        refused(-1, weigh, handle, **bad)
    for bad in [dict(width=0), dict(most=0), dict(first=-1), dict(last=-1)]:
        refused(-1, choose, handle, **bad)
    for bad in [dict(lists=0), dict(lists=3), dict(most=0), dict(weights=FAKE, width=0)]:
        refused(-1, keep, handle, **bad)
    refused(-6, keep, handle, lists=2)


def test_error_bits_have_names():
    assert pkg.decode_error(0x600) == ["TREE", "ROW_LIST"]
