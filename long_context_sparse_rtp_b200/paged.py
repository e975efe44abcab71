"""Python entry points of the paged-cache calls of librtp.so.

The signatures users see; checks, allocation and marshalling are in C++
(csrc/paged_binding.cpp, built as _paged.so), the work is in librtp.so: see
include/rtp.h for the exact contracts.  Wrong tensors raise ValueError, what the
library refuses RtpError.  Work runs on `stream` (default: the current stream of
the tensors' device), and what a call allocates, outputs and workspace, belongs to
that stream: each call has its own workspace, inside a stream capture from the
graph's own memory.

If the libraries are not built this module raises on first use -- there is no
fallback implementation.
"""
from __future__ import annotations

import importlib
import os

from .rtp import RtpError, lib

_HERE = os.path.dirname(os.path.abspath(__file__))
EXT_PATH = os.path.join(_HERE, "_paged.so")
_SCALE = 1.0 / (128 ** 0.5)
_PLAN = ("seq_lens", "cu_new", "slot_map", "spans", "free_count", "admitted")

_ext = None


def _native():
    global _ext
    if _ext is None:
        lib()
        if not os.path.exists(EXT_PATH):
            raise RuntimeError(
                f"{EXT_PATH} is not built; run `python -m long_context_sparse_rtp_b200.build`")
        import torch  # noqa: F401  (the extension links against its libraries)
        from . import build
        if build.binding_built_for() not in ("", build.binding_tag()):
            raise RuntimeError(
                f"{EXT_PATH} was built for {build.binding_built_for()}, this is "
                f"{build.binding_tag()}; run `python -m long_context_sparse_rtp_b200.build`")
        ext = importlib.import_module(__package__ + "._paged")
        ext.set_error(RtpError)
        _ext = ext
    return _ext


def rtp_paged_plan(seq_lens, n_new, block_table, free_pages, free_count, *, page_size, max_tokens,
                   row_tokens=0, release=None, out=None, stream=None):
    """Block-table entries, slots and spans of a step, from lengths on the GPU.

    seq_lens, n_new [B] int32 (present and new tokens per request), block_table
    [B, width] int32 (new entries are written), free_pages int32 and free_count
    [1] int32 (a stack), release [B] bool or uint8 (pages that go back first) or
    None.  The batch of max_tokens tokens is packed, or padded to row_tokens per
    request.  Returns dict(seq_lens [B], cu_new [B + 1], slot_map [max_tokens],
    spans [n, 4], free_count [1], admitted [B]); `out` may hold buffers for any of
    them (seq_lens and free_count themselves included)."""
    if out is None:
        bufs = (None,) * 6
    elif set(out) <= set(_PLAN):
        bufs = [out.get(name) for name in _PLAN]
    else:
        raise ValueError(f"out: expected some of {list(_PLAN)}")
    return (_ext or _native()).plan(seq_lens, n_new, block_table, free_pages, free_count, page_size,
                                    max_tokens, row_tokens, release, *bufs, stream)


def rtp_paged_kv_write(k, v, slot_map, k_pages, v_pages, *, k_scale=None, v_scale=None,
                       stream=None):
    """Rows k, v [T, Hkv, 128] bf16 into the pages [n_pages, page_size, Hkv, 128] (bf16
    or e4m3) at slot_map [T] int32; slots outside the pool skip their token."""
    (_ext or _native()).kv_write(k, v, slot_map, k_pages, v_pages, k_scale, v_scale, stream)


def rtp_paged_kv_append(k, v, spans, k_pages, v_pages, kv_role, bounds, bound_scale, *,
                        k_scale=None, v_scale=None, stream=None):
    """Rows k, v [T, Hkv, 128] bf16 into the pages by spans [n, 4] int32
    (rtp_paged_plan), and the touched pages' bounds [n_pages, retrieval kv heads, 2,
    128] int8 and bound_scale [n_pages, retrieval kv heads] fp32."""
    (_ext or _native()).kv_append(k, v, spans, k_pages, v_pages, kv_role, bounds, bound_scale,
                                  k_scale, v_scale, stream)


def rtp_paged_block_select(q, bounds, bound_scale, block_table, seq_lens, kv_role, *, page_size,
                           n_sel, n_first=1, n_recent=1, sel=None, sel_count=None, stream=None):
    """The n_sel pages each retrieval kv head of each request attends to, by the integer
    score of their bounds.  q [B, 1, H, 128].  Returns (sel [B, retrieval kv heads,
    n_sel] int32 block-table columns, ascending, -1 behind the last, and sel_count
    [B, retrieval kv heads] int32)."""
    return (_ext or _native()).block_select(q, bounds, bound_scale, block_table, seq_lens, kv_role,
                                            page_size, n_sel, n_first, n_recent, sel, sel_count,
                                            stream)


def rtp_paged_attn_decode(q, k_pages, v_pages, block_table, seq_lens, kv_role, *, window=None,
                          n_sink=0, sel=None, sel_count=None, k_scale=None, v_scale=None,
                          scale=None, o=None, lse=None, stream=None):
    """Attention of one new token per request over its pages, every head: retrieval
    heads over every key (or the pages of sel, sel_count), local heads over sinks and
    window.  q [B, 1, H, 128], seq_lens [B] int32 (the new token counted).  Returns
    (o like q, lse [B, H, 1])."""
    return (_ext or _native()).attn_decode(q, k_pages, v_pages, block_table, seq_lens, kv_role,
                                           window, n_sink, sel, sel_count, k_scale, v_scale,
                                           _SCALE if scale is None else scale, o, lse, stream)


def check_rows(k, v, k_pages, v_pages, kv_role, *, k_scale=None, v_scale=None):
    """Raises what rtp_paged_kv_append or rtp_paged_kv_write would raise for these rows and
    pages; enqueues nothing."""
    (_ext or _native()).check_rows(k, v, k_pages, v_pages, kv_role, k_scale, v_scale)


def check_block_select(q, bounds, bound_scale, block_table, seq_lens, kv_role, *, page_size,
                       n_sel, n_first=1, n_recent=1):
    """Raises what rtp_paged_block_select would raise; enqueues nothing."""
    (_ext or _native()).check_block_select(q, bounds, bound_scale, block_table, seq_lens, kv_role,
                                           page_size, n_sel, n_first, n_recent, None, None, None)


def check_attn_decode(q, k_pages, v_pages, block_table, seq_lens, kv_role, *, window=None, n_sink=0,
                      n_sel=None, k_scale=None, v_scale=None, scale=None, o=None, lse=None):
    """Raises what rtp_paged_attn_decode would raise, with lists of n_sel pages where that
    is given; enqueues nothing."""
    (_ext or _native()).check_attn_decode(q, k_pages, v_pages, block_table, seq_lens, kv_role,
                                          window, n_sink, n_sel, None, k_scale, v_scale,
                                          _SCALE if scale is None else scale, o, lse, None)
