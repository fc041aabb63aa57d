"""Tensors of the target-side calls that are not on the session's device are refused by the session,
before a pointer reaches the library (no GPU needed)."""
from types import SimpleNamespace

import pytest
import torch

import block_diffusion_speculative_fc_gb300 as pkg


class Reached(Exception):
    pass


@pytest.fixture(params=["cuda:0", "cuda:1"])
def sess(request, monkeypatch):
    """A session's Python side alone; a call that would reach the library raises Reached."""
    from block_diffusion_speculative_fc_gb300 import session

    def reached(*a, **k):
        raise Reached

    for name in ("dflash_append_kv", "dflash_paged_attention", "dflash_paged_attention_workspace_size",
                 "dflash_target_probs", "dflash_sample_tokens"):
        monkeypatch.setattr(session, name, reached)
    monkeypatch.setattr(session, "_stream", lambda: 0)
    s = pkg.DraftSession.__new__(pkg.DraftSession)
    s.h, s.device = None, torch.device(request.param)
    return s


def layer(device):
    """What the calls read of a LayerKV, on any device."""
    return SimpleNamespace(device=torch.device(device), dtype=torch.bfloat16, n_heads=4, n_kv_heads=1,
                           head_dim=64, batch=2, struct=None)


def calls(sess, lay):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 1, 64, dtype=torch.bfloat16)
    x, f = torch.zeros(3, 50, dtype=torch.bfloat16), torch.zeros(3, 50)
    ws = torch.zeros(256, dtype=torch.uint8)
    yield lambda: sess.append_kv(lay, q, k, k, i32(0, 1, 3), i32(5, 6), None, q_out=q)
    yield lambda: sess.paged_attention(lay, q, i32(0, 1, 3), i32(5, 6), q, ws)
    yield lambda: sess.attention_workspace(lay, 2, 3)
    yield lambda: sess.target_probs(x, f)
    yield lambda: sess.sample_tokens(x, f, i32(0, 0, 0))


def test_tensors_elsewhere_are_refused(sess):
    for lay in (layer("cpu"), layer("cuda:2")):
        for call in calls(sess, lay):
            with pytest.raises(ValueError):
                call()


def test_tensors_of_the_session_pass(sess):
    sess.device = torch.device("cpu")
    for call in calls(sess, layer("cpu")):
        with pytest.raises(Reached):
            call()


def test_a_layer_of_host_tensors_is_refused():
    pages = torch.zeros(2, 64, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkg.LayerKV(4, pages, pages.clone(), torch.zeros(1, 2, dtype=torch.int32))
