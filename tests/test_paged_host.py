"""The paged-cache entry points without a GPU: refusals before any CUDA call, and
the tests' own plain implementations against hand-worked values."""
import ctypes

import numpy as np
import pytest
import torch

import paged_ref as ref
from long_context_sparse_rtp_b200 import PagedCache, build, rtp, rtp_paged_plan

OK, INVALID, UNSUPPORTED, ALIGN, WS = 0, 1, 2, 3, 4
P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    build.build()
    return rtp.lib()


def pages(ptr=P, sp=64 * 4 * 128, sr=4 * 128, sh=128, n=10, ps=64, type=0):
    return rtp.Pages(ptr, sp, sr, sh, n, ps, type)


def role(*x):
    return (ctypes.c_uint8 * len(x))(*x)


def plan(L, **kw):
    a = dict(B=2, ps=64, row_tokens=0, lens=P, n_new=P, release=None, table=P, stride=8, width=8,
             free=P, cap=16, count=P, max_tokens=4, max_spans=4, out=P, cu=P, slots=P, spans=P,
             fc=P, adm=P, ws=P, ws_bytes=BIG)
    a.update(kw)
    return L.rtp_paged_plan(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(row_tokens=-1), INVALID), (dict(width=-1, stride=0), INVALID),
    (dict(stride=7), INVALID), (dict(cap=-1), INVALID), (dict(max_tokens=-1), INVALID),
    (dict(max_spans=-1), INVALID), (dict(ps=8), UNSUPPORTED), (dict(ps=48), UNSUPPORTED),
    (dict(ps=512), UNSUPPORTED), (dict(ps=0), UNSUPPORTED),
    (dict(width=1 << 27, stride=1 << 27), UNSUPPORTED), (dict(lens=None), INVALID),
    (dict(n_new=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
    (dict(count=None), INVALID), (dict(out=None), INVALID), (dict(cu=None), INVALID),
    (dict(slots=None), INVALID), (dict(spans=None), INVALID), (dict(fc=None), INVALID),
    (dict(adm=None), INVALID), (dict(spans=ODD), ALIGN), (dict(ws=ODD), ALIGN),
    (dict(ws=None), WS), (dict(ws_bytes=511), WS), (dict(B=0, lens=None), OK)])
def test_plan_refusals(L, kw, code):
    assert plan(L, **kw) == code


def write(L, **kw):
    a = dict(T=3, Hkv=4, k=P, ks=512, v=P, vs=512, slots=P, kp=pages(), vp=pages(), k_scale=None,
             v_scale=None)
    a.update(kw)
    return L.rtp_paged_kv_write(*a.values(), None)


def append(L, **kw):
    a = dict(T=3, Hkv=4, role=role(1, 0, 0, 1), k=P, ks=512, v=P, vs=512, spans=P, n=5, kp=pages(),
             vp=pages(), k_scale=None, v_scale=None, bounds=P, scale=P)
    a.update(kw)
    return L.rtp_paged_kv_append(*a.values(), None)


CACHE = [
    (dict(kp=pages(ptr=None)), INVALID), (dict(vp=pages(n=0)), INVALID),
    (dict(kp=pages(type=2), vp=pages(type=2)), UNSUPPORTED), (dict(kp=pages(ps=24)), UNSUPPORTED),
    (dict(kp=pages(n=1 << 26), vp=pages(n=1 << 26)), UNSUPPORTED),
    (dict(kp=pages(sp=0)), INVALID), (dict(kp=pages(sr=64)), INVALID),
    (dict(vp=pages(sh=-128)), INVALID), (dict(kp=pages(ptr=ODD)), ALIGN),
    (dict(kp=pages(sr=516)), ALIGN), (dict(vp=pages(sh=132)), ALIGN),
    (dict(kp=pages(type=1, sr=520), vp=pages(type=1)), ALIGN), (dict(vp=pages(n=9)), INVALID),
    (dict(vp=pages(ps=32)), INVALID), (dict(vp=pages(type=1)), INVALID),
    (dict(k_scale=P), INVALID), (dict(v_scale=P), INVALID)]


@pytest.mark.parametrize("call", [write, append])
@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(T=-1), INVALID), (dict(Hkv=0), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(ks=511), INVALID), (dict(vs=516), ALIGN), (dict(k=ODD), ALIGN), (dict(T=0, k=None), OK)])
def test_write_refusals(L, call, kw, code):
    assert call(L, **kw) == code


@pytest.mark.parametrize("call,kw,code", [
    (write, dict(slots=None), INVALID), (write, dict(Hkv=257), UNSUPPORTED),
    (append, dict(spans=None), INVALID), (append, dict(spans=ODD), ALIGN),
    (append, dict(bounds=None), INVALID), (append, dict(scale=None), INVALID),
    (append, dict(bounds=ODD), ALIGN), (append, dict(n=-1), INVALID), (append, dict(n=0), OK),
    (append, dict(role=None), INVALID), (append, dict(role=role(1, 0, 2, 1)), INVALID)])
def test_write_only_refusals(L, call, kw, code):
    assert call(L, **kw) == code


def select(L, **kw):
    a = dict(B=2, H=32, Hkv=4, role=role(1, 0, 0, 1), q=P, qs=4096, bounds=P, scale=P, n_pages=10,
             ps=64, table=P, stride=8, width=8, lens=P, n_sel=4, n_first=1, n_recent=1, sel=P,
             count=P, ws=P, ws_bytes=BIG)
    a.update(kw)
    return L.rtp_paged_block_select(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(H=30), INVALID), (dict(H=0), INVALID), (dict(H=512), UNSUPPORTED),
    (dict(H=68, Hkv=4), UNSUPPORTED), (dict(role=None), INVALID), (dict(ps=20), UNSUPPORTED),
    (dict(n_pages=0), INVALID), (dict(width=0), INVALID), (dict(stride=7), INVALID),
    (dict(width=1 << 25, stride=1 << 25), UNSUPPORTED), (dict(n_sel=0, n_first=0, n_recent=0), INVALID),
    (dict(n_first=-1), INVALID), (dict(n_recent=-1), INVALID), (dict(n_first=2, n_recent=3), INVALID),
    (dict(n_first=2 ** 31 - 1, n_recent=2 ** 31 - 1), INVALID), (dict(B=40000), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(bounds=None), INVALID), (dict(scale=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(sel=None), INVALID),
    (dict(count=None), INVALID), (dict(qs=4095), INVALID), (dict(qs=4100), ALIGN),
    (dict(q=ODD), ALIGN), (dict(bounds=ODD), ALIGN), (dict(ws=ODD), ALIGN), (dict(ws=None), WS),
    (dict(ws_bytes=256), WS), (dict(B=0), OK), (dict(role=role(0, 0, 0, 0), q=None), OK)])
def test_select_refusals(L, kw, code):
    assert select(L, **kw) == code


def attn(L, **kw):
    a = dict(B=2, H=32, Hkv=4, role=role(1, 0, 0, 1), window=64, n_sink=4, q=P, qs=4096, kp=pages(),
             vp=pages(), k_scale=None, v_scale=None, table=P, stride=8, width=8, lens=P, sel=None,
             count=None, n_sel=0, scale=0.1, o=P, os=4096, lse=None, ws=P, ws_bytes=BIG)
    a.update(kw)
    return L.rtp_paged_attn_decode(*a.values(), None)


@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(B=-1), INVALID), (dict(H=30), INVALID), (dict(H=68), UNSUPPORTED), (dict(role=None), INVALID),
    (dict(window=0), INVALID), (dict(n_sink=-1), INVALID), (dict(width=0), INVALID),
    (dict(stride=7), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(sel=P), INVALID), (dict(count=P), INVALID),
    (dict(sel=P, count=P), INVALID), (dict(sel=P, count=P, n_sel=1 << 25), UNSUPPORTED),
    (dict(width=1 << 25, stride=1 << 25), UNSUPPORTED), (dict(B=1 << 28), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(qs=4095), INVALID), (dict(os=4000), INVALID),
    (dict(q=ODD), ALIGN), (dict(o=ODD), ALIGN), (dict(qs=4100), ALIGN), (dict(os=4100), ALIGN),
    (dict(ws=ODD), ALIGN), (dict(ws=None), WS), (dict(ws_bytes=1 << 16), WS), (dict(B=0), OK)])
def test_attn_refusals(L, kw, code):
    assert attn(L, **kw) == code


def test_workspace_sizes(L):
    size = L.rtp_paged_workspace_size
    r = role(1, 0, 0, 1)
    assert size(0, 100, 0, 0, None, 0) >= 256 + 100 * 32
    assert size(1, 8, 32, 4, r, 2048) >= 8 * 2 * 2048 * 4
    # two partial results per CTA, 2 x 148 CTAs, one row per query head of a group
    assert size(2, 8, 32, 4, r, 2048) >= 2 * 296 * 8 * 132 * 4
    assert size(2, -1, 32, 4, r, 2048) == 256
    assert size(2, 8, 30, 4, r, 2048) == 256
    assert size(9, 8, 32, 4, r, 2048) == 256


def test_python_refuses_host_tensors():
    t = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        rtp_paged_plan(t, t, torch.zeros(2, 4, dtype=torch.int32), t, t[:1], page_size=64,
                       max_tokens=2)


def test_cache_layout_on_the_host():
    c = PagedCache(5, 32, [1, 0, 1], batch=2, max_len=100, device="cpu")
    assert c.k_pages.shape == (5, 32, 3, 128) and c.block_table.shape == (2, 4)
    assert c.bounds.shape == (5, 2, 2, 128) and int(c.free_pages[-1]) == 0
    assert PagedCache(5, 32, [0, 0], batch=2, max_len=100, device="cpu").bounds is None


def test_plan_by_hand():
    """Two requests, pages of 16: 15 + 2 tokens cross into a new page, 0 + 1 take one; a
    third finds no page left."""
    table = np.array([[7, -1], [-1, -1], [-1, -1]])
    r = ref.plan([15, 0, 0], [2, 1, 5], table, np.array([3, 4]), 2, page_size=16, max_tokens=8,
                 n_spans=8)
    assert r["block_table"].tolist() == [[7, 4], [3, -1], [-1, -1]]
    assert r["slot_map"].tolist() == [7 * 16 + 15, 4 * 16, 3 * 16, -1, -1, -1, -1, -1]
    assert r["admitted"].tolist() == [1, 1, 0] and r["seq_lens"].tolist() == [17, 1, 0]
    assert r["free_count"].tolist() == [0] and r["cu_new"].tolist() == [0, 2, 3, 8]
    assert r["spans"][:4].tolist() == [[7, 16, 15, 0], [4, 1, 0, 1], [3, 1, 0, 2], [-1, 0, 0, 0]]


def test_bounds_and_score_by_hand():
    rows = np.zeros((2, 128), dtype=np.float32)
    rows[0, 0], rows[1, 0], rows[1, 1] = 127.0, -63.5, 0.25
    lo, hi, s = ref.bounds(rows)
    assert abs(s - 1) < 1e-6 and hi[0] == 127 and lo[0] == -64 and hi[1] == 1 and lo[1] == 0
    q = np.zeros((1, 128), dtype=np.float32)
    q[0, 0] = -2.0  # q8 = -127: the page's bound is 127 * 64 against another's 127 * 3
    one = np.zeros(128, dtype=np.int64)
    three = one.copy()
    three[0] = -3
    got = ref.select(q, np.stack([three, lo, one]), np.stack([one, hi, one]),
                     np.array([1, s, 1], dtype=np.float32), 1, 0, 0)
    assert got == [1]


def test_e4m3_values():
    x = [0.0, 1.0, 1.0625, 1.1875, 447.0, 1e6, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -17.0]
    want = [0.0, 1.0, 1.0, 1.25, 448.0, 448.0, 2.0 ** -9, 0.0, 2.0 ** -8, -16.0]
    assert ref.e4m3(x).tolist() == want
    t = torch.randn(4000, generator=torch.Generator().manual_seed(1)) * 30
    assert np.array_equal(ref.e4m3(t.double().numpy()),
                          t.to(torch.float8_e4m3fn).double().numpy())
