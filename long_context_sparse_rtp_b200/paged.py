"""Thin Python binding of the paged-cache entry points of librtp.so (ctypes).

Argument checks and marshalling only; see include/rtp.h for the exact contracts.
Work runs on `stream` (default: the current stream of the tensors' device), and
what a call allocates, outputs and workspace, belongs to that stream: each call
has its own workspace, inside a stream capture from the graph's own memory.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from .rtp import Pages, _check, lib

PAGED_PLAN, PAGED_SELECT, PAGED_ATTN = range(3)
_KV_TYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}


def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _tensor(t, name, dtype, shape, dev, contiguous=True):
    """`t` is a tensor of this type and shape (None: any size) on `dev`."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != dev or \
            t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name}: expected {dtype} {list(shape)} on {dev}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t


def _device(t, name):
    _need(isinstance(t, torch.Tensor) and t.is_cuda, f"{name}: expected a CUDA tensor")
    return t.device


@contextlib.contextmanager
def _elsewhere(dev, stream):
    with torch.cuda.device(dev):
        if stream is None:
            yield ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
        else:
            with torch.cuda.stream(stream):
                yield ctypes.c_void_p(stream.cuda_stream)


def _on(dev, stream):
    """Context in which `dev` is current and allocations belong to the call's stream,
    which it gives as a C handle."""
    if stream is not None:
        _need(stream.device == dev, "stream: expected a stream of the tensors' device")
    elif torch.cuda.current_device() == dev.index:
        return contextlib.nullcontext(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    return _elsewhere(dev, stream)


@functools.lru_cache(maxsize=64)
def _role_array(kv_role):
    return (ctypes.c_uint8 * len(kv_role))(*kv_role)


def _roles(kv_role):
    role = tuple(int(x) for x in kv_role)
    _need(len(role) > 0 and set(role) <= {0, 1}, "kv_role: expected one 0 or 1 per kv head")
    return role, _role_array(role)


def _p(t):
    return None if t is None else t.data_ptr()


def _pages(t, name, dev):
    """[n_pages, page_size, Hkv, 128] (any order of strides) -> rtp_pages."""
    _need(isinstance(t, torch.Tensor) and t.dtype in _KV_TYPES and t.device == dev and t.dim() == 4
          and t.shape[3] == 128 and t.stride(3) == 1,
          f"{name}: expected bfloat16 or float8_e4m3fn [n_pages, page_size, Hkv, 128] on {dev}, "
          "rows of 128 contiguous")
    n, ps, h, _ = t.shape
    st = [s if m > 1 else 128 for s, m in zip(t.stride(), t.shape)]  # a size of 1 has no stride
    return Pages(t.data_ptr(), st[0], st[1], st[2], n, ps, _KV_TYPES[t.dtype])


def _cache(k_pages, v_pages, k_scale, v_scale, Hkv, dev):
    kp, vp = _pages(k_pages, "k_pages", dev), _pages(v_pages, "v_pages", dev)
    _need(k_pages.shape == v_pages.shape and k_pages.dtype == v_pages.dtype,
          "k_pages and v_pages differ in shape or type")
    _need(k_pages.shape[2] == Hkv, f"pages: expected {Hkv} kv heads")
    for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if s is not None:
            _need(kp.type == 1, f"{name}: bfloat16 pages have no scales")
            _tensor(s, name, torch.float32, (Hkv,), dev)
    return kp, vp


def _rows(x, name, T, Hkv, dev):
    """[T, Hkv, 128] bf16 with contiguous heads -> elements between rows."""
    _tensor(x, name, torch.bfloat16, (T, Hkv, 128), dev, contiguous=False)
    _need(x.stride(2) == 1 and (Hkv == 1 or x.stride(1) == 128),
          f"{name}: expected contiguous heads x 128 per row")
    return x.stride(0) if T > 1 else Hkv * 128


def _query(q, name, B, H, dev):
    """[B, 1, H, 128] bf16 with contiguous heads -> elements between requests."""
    _tensor(q, name, torch.bfloat16, (B, 1, H, 128), dev, contiguous=False)
    _need(q.stride(3) == 1 and (H == 1 or q.stride(2) == 128),
          f"{name}: expected contiguous heads x 128 per request")
    return q.stride(0) if B > 1 else H * 128


def _table(block_table, B, dev):
    _tensor(block_table, "block_table", torch.int32, (B, None), dev, contiguous=False)
    width = block_table.shape[1]
    _need(width <= 1 or block_table.stride(1) == 1, "block_table: expected contiguous rows")
    return width, block_table.stride(0) if B > 1 else width


def _workspace(op, B, H, Hkv, role, width, dev):
    return torch.empty(lib().rtp_paged_workspace_size(op, B, H, Hkv, role, width),
                       dtype=torch.uint8, device=dev)


def rtp_paged_plan(seq_lens, n_new, block_table, free_pages, free_count, *, page_size, max_tokens,
                   row_tokens=0, release=None, out=None, stream=None):
    """Block-table entries, slots and spans of a step, from lengths on the GPU.

    seq_lens, n_new [B] int32 (present and new tokens per request), block_table
    [B, width] int32 (new entries are written), free_pages int32 and free_count
    [1] int32 (a stack), release [B] bool or uint8 (pages that go back first) or
    None.  The batch of max_tokens tokens is packed, or padded to row_tokens per
    request.  Returns dict(seq_lens, cu_new, slot_map, spans, free_count,
    admitted); `out` may hold buffers for any of them (seq_lens and free_count
    themselves included)."""
    dev = _device(seq_lens, "seq_lens")
    i32 = torch.int32
    _tensor(seq_lens, "seq_lens", i32, (None,), dev)
    B = seq_lens.shape[0]
    _tensor(n_new, "n_new", i32, (B,), dev)
    width, stride = _table(block_table, B, dev)
    _tensor(free_pages, "free_pages", i32, (None,), dev)
    _tensor(free_count, "free_count", i32, (1,), dev)
    if release is not None:
        _need(isinstance(release, torch.Tensor) and release.dtype in (torch.bool, torch.uint8),
              "release: expected a bool or uint8 tensor")
        _tensor(release, "release", release.dtype, (B,), dev)
    max_tokens, row_tokens = int(max_tokens), int(row_tokens)
    _need(max_tokens >= 0 and row_tokens >= 0 and page_size > 0,
          "page_size, max_tokens and row_tokens are not negative")
    n_spans = min(max_tokens, max_tokens // page_size + 2 * B)
    shapes = dict(seq_lens=(B,), cu_new=(B + 1,), slot_map=(max_tokens,), spans=(n_spans, 4),
                  free_count=(1,), admitted=(B,))
    out = {} if out is None else out
    _need(set(out) <= set(shapes), f"out: expected some of {list(shapes)}")
    with _on(dev, stream) as s:
        r = {name: _tensor(out[name], name, i32, (None, 4) if name == "spans" else shape, dev)
             if name in out else torch.empty(shape, dtype=i32, device=dev)
             for name, shape in shapes.items()}
        if B == 0:  # no request: an empty batch
            r["slot_map"].fill_(-1)
            r["spans"].copy_(torch.tensor([-1, 0, 0, 0], dtype=i32, device=dev).expand_as(r["spans"]))
            r["cu_new"].zero_()
            r["free_count"].copy_(free_count)
            return r
        ws = _workspace(PAGED_PLAN, B, 0, 0, None, 0, dev)
        _check("rtp_paged_plan", lib().rtp_paged_plan(
            B, page_size, row_tokens, _p(seq_lens), _p(n_new), _p(release), _p(block_table),
            stride, width, _p(free_pages), free_pages.shape[0], _p(free_count), max_tokens,
            r["spans"].shape[0], _p(r["seq_lens"]), _p(r["cu_new"]), _p(r["slot_map"]),
            _p(r["spans"]), _p(r["free_count"]), _p(r["admitted"]), _p(ws), ws.numel(), s))
    return r


def rtp_paged_kv_write(k, v, slot_map, k_pages, v_pages, *, k_scale=None, v_scale=None,
                       stream=None):
    """Rows k, v [T, Hkv, 128] bf16 into the pages [n_pages, page_size, Hkv, 128] (bf16
    or e4m3) at slot_map [T] int32; slots outside the pool skip their token."""
    dev = _device(k, "k")
    _need(k.dim() == 3, "k: expected [T, Hkv, 128]")
    T, Hkv = k.shape[0], k.shape[1]
    ks, vs = _rows(k, "k", T, Hkv, dev), _rows(v, "v", T, Hkv, dev)
    _tensor(slot_map, "slot_map", torch.int32, (T,), dev)
    kp, vp = _cache(k_pages, v_pages, k_scale, v_scale, Hkv, dev)
    with _on(dev, stream) as s:
        _check("rtp_paged_kv_write", lib().rtp_paged_kv_write(
            T, Hkv, _p(k), ks, _p(v), vs, _p(slot_map), kp, vp, _p(k_scale), _p(v_scale), s))


def rtp_paged_kv_append(k, v, spans, k_pages, v_pages, kv_role, bounds, bound_scale, *,
                        k_scale=None, v_scale=None, stream=None):
    """Rows k, v [T, Hkv, 128] bf16 into the pages by spans [n, 4] int32
    (rtp_paged_plan), and the touched pages' bounds [n_pages, retrieval kv heads, 2,
    128] int8 and bound_scale [n_pages, retrieval kv heads] fp32."""
    dev = _device(k, "k")
    _need(k.dim() == 3, "k: expected [T, Hkv, 128]")
    T, Hkv = k.shape[0], k.shape[1]
    role, arr = _roles(kv_role)
    _need(len(role) == Hkv, f"kv_role: expected {Hkv} kv heads")
    ks, vs = _rows(k, "k", T, Hkv, dev), _rows(v, "v", T, Hkv, dev)
    _tensor(spans, "spans", torch.int32, (None, 4), dev)
    kp, vp = _cache(k_pages, v_pages, k_scale, v_scale, Hkv, dev)
    n, n_rkv = k_pages.shape[0], sum(role)
    _tensor(bounds, "bounds", torch.int8, (n, n_rkv, 2, 128), dev)
    _tensor(bound_scale, "bound_scale", torch.float32, (n, n_rkv), dev)
    with _on(dev, stream) as s:
        _check("rtp_paged_kv_append", lib().rtp_paged_kv_append(
            T, Hkv, arr, _p(k), ks, _p(v), vs, _p(spans), spans.shape[0], kp, vp, _p(k_scale),
            _p(v_scale), _p(bounds), _p(bound_scale), s))


def rtp_paged_block_select(q, bounds, bound_scale, block_table, seq_lens, kv_role, *, page_size,
                           n_sel, n_first=1, n_recent=1, sel=None, sel_count=None, stream=None):
    """The n_sel pages each retrieval kv head of each request attends to, by the integer
    score of their bounds.  q [B, 1, H, 128].  Returns (sel [B, retrieval kv heads,
    n_sel] int32 block-table columns, ascending, -1 behind the last, and sel_count
    [B, retrieval kv heads] int32)."""
    dev = _device(q, "q")
    _need(q.dim() == 4, "q: expected [B, 1, H, 128]")
    B, H = q.shape[0], q.shape[2]
    qs = _query(q, "q", B, H, dev)
    role, arr = _roles(kv_role)
    n_rkv, n_sel = sum(role), int(n_sel)
    _need(n_sel >= 1, "n_sel: expected at least 1")
    _tensor(bounds, "bounds", torch.int8, (None, n_rkv, 2, 128), dev)
    n_pages = bounds.shape[0]
    _tensor(bound_scale, "bound_scale", torch.float32, (n_pages, n_rkv), dev)
    width, stride = _table(block_table, B, dev)
    _tensor(seq_lens, "seq_lens", torch.int32, (B,), dev)
    with _on(dev, stream) as s:
        sel = torch.empty(B, n_rkv, n_sel, dtype=torch.int32, device=dev) if sel is None else \
            _tensor(sel, "sel", torch.int32, (B, n_rkv, n_sel), dev)
        sel_count = torch.empty(B, n_rkv, dtype=torch.int32, device=dev) if sel_count is None else \
            _tensor(sel_count, "sel_count", torch.int32, (B, n_rkv), dev)
        ws = _workspace(PAGED_SELECT, B, H, len(role), arr, width, dev)
        _check("rtp_paged_block_select", lib().rtp_paged_block_select(
            B, H, len(role), arr, _p(q), qs, _p(bounds), _p(bound_scale), n_pages, page_size,
            _p(block_table), stride, width, _p(seq_lens), n_sel, n_first, n_recent, _p(sel),
            _p(sel_count), _p(ws), ws.numel(), s))
    return sel, sel_count


def rtp_paged_attn_decode(q, k_pages, v_pages, block_table, seq_lens, kv_role, *, window=None,
                          n_sink=0, sel=None, sel_count=None, k_scale=None, v_scale=None,
                          scale=None, o=None, lse=None, stream=None):
    """Attention of one new token per request over its pages, every head: retrieval
    heads over every key (or the pages of sel, sel_count), local heads over sinks and
    window.  q [B, 1, H, 128], seq_lens [B] int32 (the new token counted).  Returns
    (o like q, lse [B, H, 1])."""
    dev = _device(q, "q")
    _need(q.dim() == 4, "q: expected [B, 1, H, 128]")
    B, H = q.shape[0], q.shape[2]
    qs = _query(q, "q", B, H, dev)
    role, arr = _roles(kv_role)
    Hkv, n_rkv = len(role), sum(role)
    _need(n_rkv == Hkv or window is not None, "window: expected with local heads")
    kp, vp = _cache(k_pages, v_pages, k_scale, v_scale, Hkv, dev)
    width, stride = _table(block_table, B, dev)
    _tensor(seq_lens, "seq_lens", torch.int32, (B,), dev)
    _need((sel is None) == (sel_count is None), "sel and sel_count come together")
    n_sel = 0
    if sel is not None:
        _tensor(sel, "sel", torch.int32, (B, n_rkv, None), dev)
        _tensor(sel_count, "sel_count", torch.int32, (B, n_rkv), dev)
        n_sel = sel.shape[2]
    scale = 1.0 / (128 ** 0.5) if scale is None else scale
    with _on(dev, stream) as s:
        o = torch.empty(B, 1, H, 128, dtype=torch.bfloat16, device=dev) if o is None else o
        os_ = _query(o, "o", B, H, dev)
        lse = torch.empty(B, H, 1, dtype=torch.float32, device=dev) if lse is None else \
            _tensor(lse, "lse", torch.float32, (B, H, 1), dev)
        ws = _workspace(PAGED_ATTN, B, H, Hkv, arr, width, dev)
        _check("rtp_paged_attn_decode", lib().rtp_paged_attn_decode(
            B, H, Hkv, arr, 0 if window is None else window, n_sink, _p(q), qs, kp, vp,
            _p(k_scale), _p(v_scale), _p(block_table), stride, width, _p(seq_lens),
            _p(sel) if n_rkv else None, _p(sel_count) if n_rkv else None, n_sel, scale, _p(o),
            os_, _p(lse), _p(ws), ws.numel(), s))
    return o, lse
