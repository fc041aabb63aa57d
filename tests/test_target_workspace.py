"""Sizes of the paged attention's workspace (host only)."""
import pytest

import block_diffusion_speculative_fc_gb300 as pkg
from block_diffusion_speculative_fc_gb300 import _build

FAKE = 0x10000  # never dereferenced by host-side code


def size(batch, rows, heads=32, kvh=8, dim=128, prefix=0, dtype=pkg.DFLASH_BF16):
    _build.build()
    kv = pkg.DflashLayerKV(dtype, heads, kvh, dim, FAKE, FAKE, 1 << 20, FAKE, 1 << 16,
                           FAKE if prefix else None, prefix)
    return pkg.dflash_paged_attention_workspace_size(kv, batch, rows)


def test_a_call_of_few_rows_needs_little():
    """A split of a token's keys holds a partial row a head: 1024 splits of 4 heads of 128 at most."""
    assert size(1, 1) < 4 << 20
    assert size(1, 1, prefix=8192) < 4 << 20
    assert size(1, 16) < 48 << 20
    assert size(1, 1, dtype=pkg.DFLASH_F32) <= 256


@pytest.mark.parametrize("heads,kvh,dim,prefix", [(32, 8, 128, 0), (64, 8, 128, 16384), (5, 1, 64, 64),
                                                  (128, 1, 128, 0), (2, 2, 64, 128)])
def test_a_larger_call_never_needs_less(heads, kvh, dim, prefix):
    rows = [1, 2, 3, 7, 16, 31, 32, 33, 64, 255, 256, 257, 1000, 16384]
    for batch in (1, 3, 128, 1024):
        sizes = [size(batch, r, heads, kvh, dim, prefix) for r in rows]
        assert sizes == sorted(sizes)
    for r in rows:
        sizes = [size(b, r, heads, kvh, dim, prefix) for b in (0, 1, 2, 60, 1024)]
        assert sizes == sorted(sizes)
        # the partial rows that any plan may lay out: one of every segment, and the items beyond it
        group = heads // kvh
        tokens = 2 * (128 // group)
        most = r * heads * (2 if prefix else 1) + 1024 * min(tokens, r) * group
        assert sizes[0] >= most * (dim + 1) * 4
