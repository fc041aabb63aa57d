"""Host objects of the target-side calls: one layer's paged cache, a rotary plan.

The calls themselves are DraftSession methods (append_kv, paged_attention,
target_probs, sample_tokens); semantics in include/dflash.h.
"""
from __future__ import annotations

import torch

from . import DFLASH_BF16, DFLASH_F32, DflashLayerKV, dflash_rope_init

_DTYPES = {torch.float32: DFLASH_F32, torch.bfloat16: DFLASH_BF16}
_SCALING = {"none": 0, "linear": 1, "bands": 2, "yarn": 3}


def dtype_code(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: float32 or bfloat16, not {t.dtype}")
    return code


def check(t, name, dtype, device, shape=None):
    """A contiguous device tensor of one type (and shape), or ValueError."""
    if t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor on {device} is needed")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} is needed, not {tuple(t.shape)}")
    return t


def rows_of(t, name, heads, dim, dtype, device, rows=None):
    """Row stride of a [rows, heads, dim] tensor whose rows are whole."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name}: shape [rows, {heads}, {dim}] is needed, not {tuple(shape)}")
    if t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name}: a {dtype} tensor on {device} is needed")
    stride = t.stride()
    if stride[2] != 1 or (heads > 1 and stride[1] != dim):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return stride[0] if shape[0] > 1 else heads * dim


def rope_plan(rotary_dim, theta, interleaved=False, scaling="none", factor=1.0,
              original_positions=0, low=0.0, high=0.0):
    """Rotary plan (include/dflash.h, dflash_rope): scaling "none", "linear", "bands" or "yarn"."""
    return dflash_rope_init(rotary_dim, 1 if interleaved else 0, theta, _SCALING[scaling], factor,
                            float(original_positions), low, high)


class LayerKV:
    """One target layer's paged cache: k_pages and v_pages [n_pages, 64, KVH, D], page_table int32
    [batch, pages_per_req], prefix_pages int32 [prefix_len / 64] of a prefix that the whole batch
    shares (or None)."""

    def __init__(self, n_heads, k_pages, v_pages, page_table, prefix_pages=None):
        if k_pages.dim() != 4 or k_pages.shape[1] != 64:
            raise ValueError(f"k_pages: shape [n_pages, 64, KVH, D] is needed, not {tuple(k_pages.shape)}")
        self.device, self.dtype = k_pages.device, k_pages.dtype
        if self.device.type != "cuda":
            raise ValueError(f"k_pages: a CUDA tensor is needed, not one on {self.device}")
        code = dtype_code(k_pages, "k_pages")
        check(k_pages, "k_pages", self.dtype, self.device)
        check(v_pages, "v_pages", self.dtype, self.device, k_pages.shape)
        check(page_table, "page_table", torch.int32, self.device)
        if page_table.dim() != 2:
            raise ValueError("page_table: shape [batch, pages_per_req] is needed")
        if prefix_pages is not None:
            check(prefix_pages, "prefix_pages", torch.int32, self.device)
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, k_pages.shape[2], k_pages.shape[3]
        self.prefix_len = 64 * prefix_pages.numel() if prefix_pages is not None else 0
        self.batch = page_table.shape[0]
        self._keep = (k_pages, v_pages, page_table, prefix_pages)
        self.struct = DflashLayerKV(code, n_heads, self.n_kv_heads, self.head_dim,
                                    k_pages.data_ptr(), v_pages.data_ptr(), k_pages.shape[0],
                                    page_table.data_ptr(), page_table.shape[1],
                                    prefix_pages.data_ptr() if self.prefix_len else None,
                                    self.prefix_len)
