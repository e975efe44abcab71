"""The paged-cache operators on the GPU against plain implementations in 64 bits
(paged_ref.py).

Tolerances of attention, per output element (u16 the half step of the 16-bit
type that P is rounded to: bf16 2^-8, fp16 2^-11):
  |o - exact| <= 2^-8 |o|                       the output's own rounding to bf16
               + (u16 + 2 e + 2^-20) sum p |v|  P's rounding, the scores' error e on
                                                both sides of the quotient, exp2
               + n 2^-24 sum p |v|              fp32 sums over n keys
with e = (128 2^-24 + 2^-22) max sum |q k| scale: fp32 sums of 128 products, and
the scores' multiplication.  lse: e + n 2^-24 + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest
import torch

import paged_ref as ref
from long_context_sparse_rtp_b200 import (PagedCache, RtpError, rtp_dense_attn,
                                          rtp_layer_decode_paged, rtp_local_attn,
                                          rtp_paged_attn_decode, rtp_paged_block_select,
                                          rtp_paged_kv_append, rtp_paged_kv_write, rtp_paged_plan)

pytestmark = pytest.mark.gpu
DEV, D = "cuda", 128
SCALE = D ** -0.5
I32 = torch.int32


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from long_context_sparse_rtp_b200 import build
    build.build()


def ints(x, **kw):
    return torch.tensor(x, dtype=I32, device=DEV, **kw)


class Made:
    """A filled paged cache: pages in random order, NaN wherever nothing is stored."""

    def __init__(self, lens, ps, H, roles, kv="bf16", layout="row", seed=0, width=None, tail=2):
        g = torch.Generator(device=DEV).manual_seed(seed)
        B, Hkv = len(lens), len(roles)
        need = [ref.up(n, ps) for n in lens]
        width = max(1, max(need, default=1)) + 1 if width is None else width
        n_pages = sum(need) + tail
        self.lens, self.ps, self.H, self.Hkv, self.roles, self.kv = lens, ps, H, Hkv, roles, kv
        self.G = H // Hkv
        ids = torch.randperm(n_pages, generator=g, device=DEV).to(I32)
        self.table = torch.full((B, width), n_pages + 7, dtype=I32, device=DEV)
        self.k_scale = self.v_scale = None
        dtype = torch.bfloat16
        if kv == "e4m3":
            dtype = torch.float8_e4m3fn
            self.k_scale = torch.rand(Hkv, generator=g, device=DEV) * 0.02 + 0.005
            self.v_scale = torch.rand(Hkv, generator=g, device=DEV) * 0.02 + 0.005
        shape = (n_pages, ps, Hkv, D) if layout == "row" else (n_pages, Hkv, ps, D)
        if layout == "padded":
            shape = (n_pages, ps, Hkv + 1, D)
        store = [torch.full(shape, float("nan"), device=DEV).to(dtype) for _ in range(2)]
        if layout == "head":
            store = [s.transpose(1, 2) for s in store]
        if layout == "padded":
            store = [s[:, :, :Hkv] for s in store]
        self.k_pages, self.v_pages = store
        self.k, self.v = [], []  # per request, values in 64 bits [n, Hkv, D]
        at = 0
        for b, n in enumerate(lens):
            mine = ids[at:at + need[b]].long()
            at += need[b]
            self.table[b, :need[b]] = mine.to(I32)
            pos = torch.arange(n, device=DEV)
            for pages, vals, scale in ((self.k_pages, self.k, self.k_scale),
                                       (self.v_pages, self.v, self.v_scale)):
                x = torch.randn((n, Hkv, D), generator=g, device=DEV, dtype=torch.bfloat16)
                if kv == "e4m3":
                    x = (x.float() / scale[:, None]).clamp(-448, 448).to(dtype)
                pages[mine[pos // ps], pos % ps] = x
                x = x.double()
                vals.append(x if scale is None else x * scale.double()[:, None])
        self.seq_lens = ints(lens)
        self.q = torch.randn((B, 1, H, D), generator=g, device=DEV, dtype=torch.bfloat16)

    def attn(self, **kw):
        a = dict(k_scale=self.k_scale, v_scale=self.v_scale)
        a.update(kw)
        return rtp_paged_attn_decode(self.q, self.k_pages, self.v_pages, self.table, self.seq_lens,
                                     self.roles, **a)

    def check(self, o, lse, window=None, n_sink=0, scale=SCALE, sel=None, count=None, drop=()):
        """Every head of every request against 64 bits; drop: (request, position)s that count
        as absent."""
        u16 = 2.0 ** -11 if self.kv == "e4m3" else 2.0 ** -8
        G = self.G
        for b, n in enumerate(self.lens):
            for g, role in enumerate(self.roles):
                pages = None
                if role and sel is not None:
                    r = sum(self.roles[:g])
                    pages = sel[b, r, :int(count[b, r])].tolist()
                keys = [j for j in ref.keys_of(n, role, self.ps, window, n_sink, pages)
                        if (b, j) not in drop]
                idx = torch.tensor(keys, dtype=torch.long, device=DEV)
                h = slice(g * G, (g + 1) * G)
                eo, el, mag, sqk = ref.attend(self.q[b, 0, h], self.k[b][idx, g], self.v[b][idx, g],
                                              scale)
                e = (128 * 2.0 ** -24 + 2.0 ** -22) * sqk * scale
                nn = len(keys) * 2.0 ** -24
                tol = 2.0 ** -8 * eo.abs() + (u16 + 2 * e + 2.0 ** -20 + nn) * mag
                err = (o[b, 0, h].double() - eo).abs()
                assert bool((err <= tol).all()), (b, g, float((err - tol).max()))
                gl = lse[b, h, 0].double()
                if not keys:
                    assert bool((gl == float("-inf")).all()) and bool((o[b, 0, h] == 0).all())
                else:
                    lt = e + nn + 2.0 ** -20 * (1 + el.abs().max())
                    assert float((gl - el.to(gl.device)).abs().max()) <= lt, (b, g)


RAGGED = [0, 1, 15, 16, 17, 63, 64, 65, 129, 300, 0, 1000]


# ------------------------------------------------------------------------------------ attention
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H,roles", [(4, (1, 1)), (8, (1, 0)), (6, (0, 1))])
def test_attn_ragged(kv, ps, H, roles):
    m = Made(RAGGED, ps, H, roles, kv, seed=ps)
    o, lse = m.attn(window=37, n_sink=5)
    m.check(o, lse, 37, 5)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (8, 1), (16, 1), (32, 4), (16, 16), (10, 2), (64, 4)])
def test_attn_head_layouts(kv, H, Hkv):
    m = Made([77, 400, 33], 32, H, [1] * Hkv, kv, seed=H)
    m.check(*m.attn())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["head", "padded"])
def test_attn_page_strides(kv, layout):
    m = Made([77, 400, 33], 16, 8, (1, 0, 1, 1), kv, layout, seed=3)
    m.check(*m.attn(window=20, n_sink=0), window=20)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (16, 16), (17, 40), (100, 3), (999, 1),
                                           (5000, 0), (1, 5000), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_attn_windows(window, n_sink):
    m = Made(RAGGED, 32, 8, (0, 0), seed=window % 97)
    m.check(*m.attn(window=window, n_sink=n_sink), window, n_sink)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [20011, 70001])
def test_attn_long(kv, n):
    """One request over every CTA, and three beside short ones: the joins of many parts."""
    m = Made([n], 64, 8, (1, 0), kv, seed=1)
    m.check(*m.attn(window=4096, n_sink=4), 4096, 4)
    m = Made([3, n // 3, 0, n // 2, 1, 100], 16, 8, (1, 1), kv, seed=2)
    m.check(*m.attn())


def test_attn_many_requests():
    """More requests than a CTA scans at once (128), more rows than CTAs."""
    lens = [(37 * i) % 90 for i in range(300)]
    m = Made(lens, 16, 4, (1, 0), seed=5)
    m.check(*m.attn(window=9, n_sink=2), 9, 2)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("B", [3, 30, 60, 120])
@pytest.mark.parametrize("H", [4, 32])
def test_attn_clusters(kv, B, H):
    """Row counts that give a row 16, 8, 4, 2 and 1 CTAs; one long request, the others ragged."""
    lens = [(53 * i) % 400 for i in range(B)]
    lens[B // 2] = 9001 if B == 3 else 1000
    m = Made(lens, 16, H, (1, 0), kv, seed=B)
    m.check(*m.attn(window=300, n_sink=3), 300, 3)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("H", [4, 16])
def test_attn_long_selection(kv, H):
    """Selected pages beyond what clusters take, beside short and unused rows."""
    m = Made([30000, 500, 0, 19500], 64, H, (1,), kv, seed=H)
    g = torch.Generator().manual_seed(H)
    sel = torch.full((4, 1, 300), -1, dtype=I32)
    count = torch.zeros(4, 1, dtype=I32)
    for b, n in enumerate(m.lens):
        nb = ref.up(n, 64)
        k = min(300, nb)
        sel[b, 0, :k] = torch.randperm(nb, generator=g)[:k].sort().values.to(I32)
        count[b, 0] = k
    sel, count = sel.to(DEV), count.to(DEV)
    m.check(*m.attn(sel=sel, sel_count=count), sel=sel, count=count)


def test_attn_selection_that_cannot_be_meant():
    """Columns outside the table or behind the request, and counts outside the list, name no
    keys."""
    m = Made([100, 40], 16, 4, (1,), seed=3)
    sel = ints([[[0, -1, 3, 99]], [[2 ** 31 - 1, 1, 5, 2]]])
    count = ints([[9], [-2]])
    o, lse = m.attn(sel=sel, sel_count=count)
    m.check(o, lse, sel=ints([[[0, 3]], [[0, 0]]]), count=ints([[2], [0]]))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,H", [(50, 4), (200, 4), (200, 32)])
def test_attn_one_long_among_many(kv, B, H):
    """The split over all CTAs with many rows, some of them empty, more requests than a CTA
    scans at once, and joins of rows that many CTAs and that two CTAs share."""
    lens = [(37 * i) % 90 for i in range(B)]
    lens[B // 3], lens[B - 1] = 9001, 1500
    m = Made(lens, 16, H, (1, 0), kv, seed=B)
    m.check(*m.attn(window=70, n_sink=3), 70, 3)


def test_attn_scale_outputs_and_strided_q():
    m = Made([100, 7], 16, 8, (1, 1), seed=6)
    big = torch.zeros(2, 1, 3, 8, D, dtype=torch.bfloat16, device=DEV)
    big[:, :, 1] = m.q
    m.q = big[:, :, 1]  # a slice of one projection's output
    out = torch.full((2, 1, 2, 8, D), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(2, 8, 1, device=DEV)
    o, l2 = m.attn(scale=0.5, o=out[:, :, 0], lse=lse)
    assert l2 is lse and bool((out[:, :, 1] == 5).all())
    m.check(out[:, :, 0], lse, scale=0.5)


def test_attn_large_scores_and_offsets():
    """Logits of +-100 and keys that share a large offset: the running maximum carries it."""
    m = Made([500], 16, 4, (1,), seed=7)
    m.q = m.q * 10
    m.check(*m.attn())


def test_attn_bad_pages_and_lengths():
    """Table entries outside the pool hide their keys; lengths beyond the table stop at it,
    negative ones are zero."""
    m = Made([200, 90, 64], 32, 4, (1, 0), seed=8)
    m.table[0, 2] = -1
    m.table[1, 0] = 10 ** 9
    m.table[1, 2] = m.k_pages.shape[0]
    drop = {(0, j) for j in range(64, 96)} | {(1, j) for j in range(32)} | \
        {(1, j) for j in range(64, 90)}
    m.check(*m.attn(window=50, n_sink=8), 50, 8, drop=drop)
    width = m.table.shape[1]
    m = Made([width * 32, 90], 32, 4, (1, 0), seed=9, width=width)
    m.seq_lens = ints([10 ** 9, -5])
    m.lens = [width * 32, 0]
    m.check(*m.attn(window=50, n_sink=8), 50, 8)


def test_attn_all_empty():
    m = Made([0, 0], 16, 8, (1, 0), seed=1)
    m.check(*m.attn(window=4), window=4)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attn_nan_stays_with_its_head(kv):
    """A NaN key in one request's kv head reaches that head's outputs and no others."""
    m = Made([70, 70], 16, 4, (1, 1), kv, seed=10)
    page = int(m.table[1, 1])
    m.k_pages[page, 3, 0, 5] = float("nan")
    o, lse = m.attn()
    assert bool(o[1, 0, :2].isnan().all()) and bool(lse[1, :2].isnan().all())
    assert not bool(o[0].isnan().any()) and not bool(o[1, 0, 2:].isnan().any())


def test_attn_infinite_scores():
    """A key of score -inf is absent; a V of infinity gives infinity."""
    m = Made([40], 16, 1, (1,), seed=11)
    m.q = m.q.abs() + 0.1
    page = int(m.table[0, 0])
    m.k_pages[page, 2, 0] = float("-inf")
    o, lse = m.attn()
    m.k[0][2] = 0
    m.check(o, lse, drop={(0, 2)})
    m.v_pages[page, 4, 0, 9] = float("inf")
    o, _ = m.attn()
    assert float(o[0, 0, 0, 9]) == float("inf") and bool(o[0, 0, 0, :9].isfinite().all())


def test_attn_repeats_and_sees_only_its_request():
    m = Made([5000, 301, 17], 16, 8, (1, 0), seed=12)
    a, b = m.attn(window=100), m.attn(window=100)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attn_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements: the request lies at its end."""
    ps, Hkv = 256, 8
    n_pages = (2 ** 31) // (ps * Hkv * D) + 40
    pool = torch.empty(n_pages, ps, Hkv, D, dtype=torch.bfloat16, device=DEV)
    m = Made([700, 5], ps, 8, [1] * Hkv, seed=13)
    old = m.table.clone()
    for b in range(2):
        for c in range(ref.up(m.lens[b], ps)):
            to = n_pages - 1 - (b * 3 + c)
            pool[to] = m.k_pages[int(old[b, c])]
            m.table[b, c] = to
    m.v = m.k
    m.k_pages = m.v_pages = pool
    m.check(*m.attn())
    # and the writes: the last page's last row
    slot = ints([n_pages * ps - 1])
    row = torch.randn(1, Hkv, D, device=DEV, dtype=torch.bfloat16)
    rtp_paged_kv_write(row, row, slot, pool, pool)
    assert torch.equal(pool[-1, -1], row[0])


# ------------------------------------------------------------------------------------ selection
def random_bounds(n_pages, n_rkv, seed, ties=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    a = torch.randint(-127, 128, (2, n_pages, n_rkv, D), generator=g, device=DEV)
    b = torch.stack([a.amin(0), a.amax(0)], 2).to(torch.int8)
    s = torch.rand(n_pages, n_rkv, generator=g, device=DEV)
    if ties:
        b[:] = b[:1]
        s = torch.floor(s * 3)
    return b.contiguous(), s


def check_select(q, b, s, table, lens, roles, ps, n_sel, n_first, n_recent):
    sel, count = rtp_paged_block_select(q, b, s, table, ints(lens), roles, page_size=ps,
                                        n_sel=n_sel, n_first=n_first, n_recent=n_recent)
    heads = [g for g, r in enumerate(roles) if r]
    G = q.shape[2] // len(roles)
    qc, bc, sc, tc = (x.float().cpu().numpy() if x.is_floating_point() else x.cpu().numpy()
                      for x in (q, b, s, table))
    for i, n in enumerate(lens):
        nb = min(table.shape[1], ref.up(max(n, 0), ps))
        for r, g in enumerate(heads):
            t = tc[i, :nb]
            bad = (t < 0) | (t >= b.shape[0])
            t = np.where(bad, 0, t)
            lo, hi = bc[t, r, 0].astype(np.int64), bc[t, r, 1].astype(np.int64)
            want = ref.select(qc[i, 0, g * G:(g + 1) * G], lo, hi, np.where(bad, -1, sc[t, r]),
                              n_sel, n_first, n_recent)
            assert int(count[i, r]) == len(want)
            assert sel[i, r].tolist() == want + [-1] * (n_sel - len(want)), (i, r)


def tables(lens, ps, width, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n_pages = sum(ref.up(n, ps) for n in lens) + 3
    ids = torch.randperm(n_pages, generator=g, device=DEV).to(I32)
    table = torch.full((len(lens), width), -1, dtype=I32, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        k = ref.up(n, ps)
        table[b, :k] = ids[at:at + k]
        at += k
    return table, n_pages


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("H,roles", [(4, (1,)), (16, (1,)), (6, (1, 0, 1)), (1, (1,)), (32, (0, 1, 1, 1))])
@pytest.mark.parametrize("n_sel,n_first,n_recent", [(1, 0, 0), (5, 1, 1), (20, 3, 9), (64, 0, 64), (7, 7, 0)])
def test_select(ties, H, roles, n_sel, n_first, n_recent):
    lens = [0, 1, 16, 17, 16 * 20, 16 * 21, 16 * 64, 16 * 65, 1900]
    table, n_pages = tables(lens, 16, 125, seed=H)
    b, s = random_bounds(n_pages, sum(roles), n_sel, ties)
    q = torch.randn(len(lens), 1, H, D, device=DEV, dtype=torch.bfloat16)
    check_select(q, b, s, table, lens, roles, 16, n_sel, n_first, n_recent)


@pytest.mark.parametrize("width,n_sel", [(1024, 100), (1025, 1000), (4096, 31), (4097, 256),
                                         (16384, 2049), (16385, 300), (33000, 5000)])
@pytest.mark.parametrize("ties", [False, True])
def test_select_long_rows(width, n_sel, ties):
    lens = [width * 16, width * 16 - 5 * 16 - 3]
    table, n_pages = tables(lens, 16, width, seed=width)
    b, s = random_bounds(n_pages, 1, n_sel, ties)
    q = torch.randn(2, 1, 2, D, device=DEV, dtype=torch.bfloat16)
    check_select(q, b, s, table, lens, (1,), 16, n_sel, 1, 2)


def test_select_special_values():
    """Zero and non-finite queries, infinite page scales, huge scales, bad pages, zero scales."""
    lens = [16 * 40] * 5
    table, n_pages = tables(lens, 16, 40, seed=1)
    b, s = random_bounds(n_pages, 1, 5)
    s[3::7] = float("inf")
    s[4::7] = 3e38
    s[5::7] = 0
    q = torch.randn(5, 1, 2, D, device=DEV, dtype=torch.bfloat16)
    q[0] = 0
    q[1, 0, 0, 3] = float("nan")
    q[2, 0, :, 3] = float("inf")
    q[3] *= 1e30
    table[4, ::3] = -1
    table[4, 1] = n_pages
    for n_sel in (1, 6, 33, 39):
        check_select(q, b, s, table, lens, (1,), 16, n_sel, 0, 1)


# ------------------------------------------------------------------------------------- plan
def check_plan(lens, news, *, ps, width, free, max_tokens=None, row_tokens=0, release=None, seed=0,
               in_place=False, cap=None):
    g = np.random.default_rng(seed)
    B = len(lens)
    cap = cap or 4096
    ids = g.permutation(100000).astype(np.int32)
    table = np.full((B, width), -1, dtype=np.int32)
    for b in range(B):
        k = min(width, ref.up(max(0, lens[b]), ps))
        table[b, :k], ids = ids[:k], ids[k:]
    stack = ids[:cap].copy()
    if max_tokens is None:
        max_tokens = (B * row_tokens if row_tokens else sum(max(0, n) for n in news)) + 3
    n_spans = min(max_tokens, max_tokens // ps + 2 * B)
    want = ref.plan(lens, news, table, stack, free, page_size=ps, max_tokens=max_tokens,
                    n_spans=n_spans, row_tokens=row_tokens, release=release)
    wide = torch.full((B, width + 3), -9, dtype=I32, device=DEV)
    t = wide[:, :width]
    t.copy_(torch.from_numpy(table))
    seq, fc, pool = ints(lens), ints([free]), torch.from_numpy(stack).to(DEV)
    rel = None if release is None else torch.tensor(release, dtype=torch.bool, device=DEV)
    out = dict(seq_lens=seq, free_count=fc) if in_place else None
    got = rtp_paged_plan(seq, ints(news), t, pool, fc, page_size=ps, max_tokens=max_tokens,
                         row_tokens=row_tokens, release=rel, out=out)
    if in_place:
        assert got["seq_lens"] is seq and got["free_count"] is fc
    else:
        assert seq.tolist() == list(lens) and fc.tolist() == [free]
    for name in ("seq_lens", "cu_new", "slot_map", "spans", "free_count", "admitted"):
        assert np.array_equal(got[name].cpu().numpy(), want[name]), name
    assert np.array_equal(t.cpu().numpy(), want["block_table"])
    assert bool((wide[:, width:] == -9).all())
    assert np.array_equal(pool.cpu().numpy(), want["free_pages"])
    return got


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ps", [16, 64, 256])
def test_plan_steps(ps, in_place):
    lens = [0, 1, ps - 1, ps, ps + 1, 7 * ps - 1, 7 * ps, 333]
    check_plan(lens, [1] * 8, ps=ps, width=30, free=50, in_place=in_place)
    check_plan(lens, [0, 1, 0, 1, 2, 3, 0, 5], ps=ps, width=30, free=50, in_place=in_place)
    check_plan(lens, [0] * 8, ps=ps, width=30, free=0, in_place=in_place)


@pytest.mark.parametrize("B", [1, 31, 64, 1023, 1024, 1025, 2500])
@pytest.mark.parametrize("big", [0, 700])
def test_plan_many(B, big):
    g = np.random.default_rng(B + big)
    lens = g.integers(0, 200, B).tolist()
    news = (g.integers(0, 3, B) + (g.random(B) < 0.05) * big).tolist()
    check_plan(lens, news, ps=16, width=70, free=9000, cap=20000, seed=B)


def test_plan_prompts():
    check_plan([0, 100, 0, 7], [5000, 3001, 1, 20000], ps=64, width=400, free=600)


@pytest.mark.parametrize("big", [0, 3000])  # one launch, and two
def test_plan_refusals_on_the_device(big):
    """Free pages, table width and batch that do not suffice; requests behind a refused one."""
    lens, ps = [15, 0, 16, 30, 100, 0], 16
    news = [2, 40 + big, 16, 1, 1, 0]
    for free in (0, 1, 2, 3, 4, 5, 60):
        check_plan(lens, news, ps=ps, width=300, free=free)
    check_plan(lens, news, ps=ps, width=7, free=300)
    for cut in (0, 1, 2, 41 + big, 43 + big, 59 + big):
        check_plan(lens, news, ps=ps, width=300, free=300, max_tokens=cut)
    check_plan([-3, 10 ** 9, 5], [4, 1, -2], ps=ps, width=30, free=5)
    check_plan([5, 5], [2 ** 31 - 1, 2 ** 31 - 1], ps=ps, width=30, free=5, max_tokens=10)


@pytest.mark.parametrize("big", [0, 3000])
def test_plan_release(big):
    lens = [33, 0, 160, 5, 400]
    for release in ([1, 0, 0, 0, 0], [0, 1, 1, 0, 1], [1] * 5, [0] * 5):
        for free in (0, 3, 40):
            check_plan(lens, [3, 1, 0, 40 + big, 1], ps=16, width=250, free=free, release=release,
                       in_place=True)
    check_plan(lens, [0] * 5, ps=16, width=250, free=10, cap=20, release=[1] * 5)  # a full stack


@pytest.mark.parametrize("row_tokens", [1, 2, 5, 700])
def test_plan_padded(row_tokens):
    lens = [0, 15, 16, 31, 100, 0]
    news = [min(row_tokens, n) for n in (1, 1, 0, 700, 3, 0)]
    check_plan(lens, news, ps=16, width=99, free=99, row_tokens=row_tokens)
    check_plan(lens, [n + 1 for n in news], ps=16, width=99, free=99, row_tokens=row_tokens)
    check_plan(lens, news, ps=16, width=99, free=99, row_tokens=row_tokens,
               max_tokens=3 * row_tokens + 1)


def test_plan_of_nothing():
    e = torch.empty(0, dtype=I32, device=DEV)
    r = rtp_paged_plan(e, e, torch.empty(0, 4, dtype=I32, device=DEV), e, ints([0]), page_size=16,
                       max_tokens=5)
    assert r["slot_map"].tolist() == [-1] * 5 and r["cu_new"].tolist() == [0]


# ------------------------------------------------------------------------------------- writes
def written(kv, x, scale):
    """What the pages hold for rows x, as fp64."""
    if kv == "bf16":
        return x.double().cpu().numpy()
    # fp32 division, as the pages' definition has it; then the nearest e4m3 value
    y = (x.float() / scale[:, None]).double().cpu().numpy()
    return ref.e4m3(y)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["row", "head"])
@pytest.mark.parametrize("T,Hkv", [(1, 1), (1, 8), (5, 3), (257, 4), (33, 17), (3, 256), (0, 2)])
def test_kv_write(kv, layout, T, Hkv):
    g = torch.Generator(device=DEV).manual_seed(T)
    ps, n_pages = 16, 40
    dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    shape = (n_pages, ps, Hkv, D) if layout == "row" else (n_pages, Hkv, ps, D)
    kp, vp = (torch.full(shape, 3.0, device=DEV).to(dtype) for _ in range(2))
    if layout == "head":
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    qkv = torch.randn(T, 3, Hkv, D, generator=g, device=DEV, dtype=torch.bfloat16) * 4
    k, v = qkv[:, 1], qkv[:, 2]
    sc = torch.rand(2, Hkv, generator=g, device=DEV) * 0.1 + 0.001 if kv == "e4m3" else (None, None)
    slot = torch.randperm(n_pages * ps, generator=g, device=DEV)[:T].to(I32)
    slot[T // 2:T // 2 + 1] = -1
    if T > 4:
        slot[1] = n_pages * ps
        slot[3] = 2 ** 31 - 1
    rtp_paged_kv_write(k, v, slot, kp, vp, k_scale=sc[0], v_scale=sc[1])
    for pages, x, s in ((kp, k, sc[0]), (vp, v, sc[1])):
        want = np.full((n_pages * ps, Hkv, D), 3.0)
        rows = written(kv, x, s)
        for t, p in enumerate(slot.tolist()):
            if 0 <= p < n_pages * ps:
                want[p] = rows[t]
        got = pages.double().cpu().numpy().reshape(n_pages * ps, Hkv, D)
        assert np.array_equal(got, want)


def test_kv_write_rounds_the_fp32_quotient():
    """Scales for which many quotients lie within a unit in the last place of the middle of
    two e4m3 values, powers of two, subnormal quotients, and scales at the ends of fp32:
    always the e4m3 value nearest to the fp32 quotient, as torch divides."""
    g = torch.Generator(device=DEV).manual_seed(5)
    H = 256
    x = torch.randn(96, H, D, generator=g, device=DEV, dtype=torch.bfloat16)
    mid = 2.0 ** torch.randint(-7, 9, (H,), generator=g, device=DEV) * \
        (1 + (2 * torch.randint(0, 8, (H,), generator=g, device=DEV) + 1) / 16)
    scale = x[0, :, 0].abs().float() / mid.float()  # x[0] / scale is next to mid
    scale[:32] = 2.0 ** torch.arange(-16, 16, device=DEV).float()
    special = [0.0, float("inf"), float("nan"), 1e-45, 1e-38, 2e-38, 3e38, 1.7e38, -0.3, -1e-40,
               2.0 ** -126, 2.0 ** 127, 2.0 ** -125, 2.0 ** 125]
    scale[32:32 + len(special)] = torch.tensor(special, device=DEV)
    x[1:65, :, 0] = x[0, :, 0]  # and its neighbours in bf16
    x[1:65, :, 0].view(torch.int16).add_(torch.arange(-32, 32, device=DEV, dtype=torch.int16)[:, None])
    x[65], x[66, :, :4] = 0, torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0])
    x[67:80] *= 1e-5
    kp, vp = (torch.zeros(6, 16, H, D, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    rtp_paged_kv_write(x, x, torch.arange(96, device=DEV, dtype=I32), kp, vp, k_scale=scale,
                       v_scale=scale)
    want = (x.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    for got in (kp, vp):
        a, b = got.view(96, H, D).float(), want.float()
        assert torch.equal(a.isnan(), b.isnan())
        assert torch.equal(a.nan_to_num(1.0), b.nan_to_num(1.0))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("ps", [16, 64, 256])
@pytest.mark.parametrize("roles", [(1,), (0, 1, 0, 1), (0, 0)])
def test_append_matches_write_and_bounds(kv, ps, roles):
    """Plan, append in three uneven steps: pages as kv_write leaves them, bounds of every
    touched page by their definition, nothing else touched."""
    g = torch.Generator(device=DEV).manual_seed(ps)
    Hkv, B = len(roles), 4
    dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    sc = torch.rand(2, Hkv, generator=g, device=DEV) * 0.1 + 0.01 if kv == "e4m3" else (None, None)
    c = PagedCache(60, ps, roles, batch=B, max_len=8 * ps, device=DEV, dtype=dtype, k_scale=sc[0],
                   v_scale=sc[1], bounds=True)
    n_rkv = sum(roles)
    # the bounds too are checked where no head has any: an empty array is legal
    bounds = torch.full((60, n_rkv, 2, D), 99, dtype=torch.int8, device=DEV)
    scale = torch.full((60, n_rkv), -5.0, device=DEV)
    kp, vp = torch.zeros_like(c.k_pages), torch.zeros_like(c.v_pages)
    touched = set()
    for news in ([ps + 3, 1, 0, 2 * ps], [1, 0, 5, 1], [ps, ps - 1, 1, 0]):
        T = sum(news)
        k, v = (torch.randn(T, Hkv, D, generator=g, device=DEV, dtype=torch.bfloat16)
                for _ in range(2))
        k[0, :, 7] = 0
        plan = rtp_paged_plan(c.seq_lens, ints(news), c.block_table, c.free_pages, c.free_count,
                              page_size=ps, max_tokens=T, out=dict(seq_lens=c.seq_lens,
                                                                   free_count=c.free_count))
        rtp_paged_kv_append(k, v, plan["spans"], c.k_pages, c.v_pages, roles, bounds, scale,
                            k_scale=sc[0], v_scale=sc[1])
        rtp_paged_kv_write(k, v, plan["slot_map"], kp, vp, k_scale=sc[0], v_scale=sc[1])
        assert torch.equal(c.k_pages.view(torch.uint8), kp.view(torch.uint8))
        assert torch.equal(c.v_pages.view(torch.uint8), vp.view(torch.uint8))
        for page, rows, _, _ in plan["spans"].tolist():
            if page < 0:
                continue
            touched.add(page)
            for r, h in enumerate([h for h, x in enumerate(roles) if x]):
                lo, hi, s = ref.bounds(kp[page, :rows, h].float().cpu().numpy())
                assert np.float32(scale[page, r].item()) == s
                assert bounds[page, r, 0].tolist() == lo.tolist()
                assert bounds[page, r, 1].tolist() == hi.tolist()
    rest = [p for p in range(60) if p not in touched]
    assert bool((bounds[rest] == 99).all()) and bool((scale[rest] == -5).all())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_append_special_values(kv):
    """Zero pages, one NaN, infinities: scale 0, inf, and inf (8 bits saturate instead)."""
    dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    c = PagedCache(4, 16, (1,), batch=3, max_len=32, device=DEV, dtype=dtype)
    k = torch.zeros(9, 1, D, dtype=torch.bfloat16, device=DEV)
    k[4, 0, 77] = float("nan")
    k[7, 0, 3] = float("-inf")
    plan = c.append(k, k, ints([3, 3, 3]))
    pages = plan["spans"][:3, 0].long()
    want = [0.0, float("inf"), float("inf") if kv == "bf16" else
            float(np.float32(448) * (np.float32(1) / np.float32(127)))]
    assert c.bound_scale[pages, 0].tolist() == want
    b = c.bounds[pages].cpu()
    assert bool((b[:2] == 0).all())
    assert int(b[2, 0, 0, 3]) == (0 if kv == "bf16" else -127)
    sat = c.k_pages[pages[2], 1, 0, 3]
    assert float(sat) == (float("-inf") if kv == "bf16" else -448.0)


def test_append_skips_spans_that_cannot_be_meant():
    c = PagedCache(4, 16, (1,), batch=1, max_len=64, device=DEV)
    k = torch.ones(4, 1, D, dtype=torch.bfloat16, device=DEV)
    spans = ints([[-1, 16, 0, 0], [4, 16, 0, 0], [2 ** 31 - 1, 16, 0, 0], [1, 99, 0, 0],
                  [2, 3, 0, -1], [3, -4, 0, 0]])
    rtp_paged_kv_append(k, k, spans, c.k_pages, c.v_pages, (1,), c.bounds, c.bound_scale)
    got = c.k_pages[:, :, 0, 0].float().cpu()
    want = torch.zeros(4, 16)
    want[1, :4] = 1  # rows past the page and tokens past the batch are left out
    want[2, 1:3] = 1
    assert torch.equal(got, want)


# ------------------------------------------------------------------------------------- together
def run_cache(dtype, roles, H, steps, n_sel=None, use=None, seed=0, ps=16, window=40, n_sink=4):
    """Prompts, then decode steps of a padded batch; every step against 64 bits.  Rows: two
    requests, an unused one, one that joins late in place of the first."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    Hkv, B = len(roles), 4
    sc = torch.full((2, Hkv), 0.02, device=DEV) if dtype != torch.bfloat16 else (None, None)
    c = PagedCache(300, ps, roles, batch=B, max_len=1500, device=DEV, dtype=dtype, k_scale=sc[0],
                   v_scale=sc[1])
    m = Made([0] * B, ps, H, roles, "bf16" if dtype == torch.bfloat16 else "e4m3", seed=seed)
    m.k = [torch.zeros(0, Hkv, D, dtype=torch.float64, device=DEV) for _ in range(B)]
    m.v = list(m.k)

    def stored(x, s):
        if s is None:
            return x.double()
        return (x.float() / s[:, None]).clamp(-448, 448).to(dtype).double() * s.double()[:, None]

    def rows(n):
        return torch.randn(n, Hkv, D, generator=g, device=DEV, dtype=torch.bfloat16)

    def note(b, k, v):
        m.k[b] = torch.cat([m.k[b], stored(k, sc[0])])
        m.v[b] = torch.cat([m.v[b], stored(v, sc[1])])
        m.lens[b] = m.k[b].shape[0]

    news = [700, 33, 0, 1001]
    k, v = rows(sum(news)), rows(sum(news))
    plan = c.append(k, v, ints(news))
    assert plan["admitted"].tolist() == [1] * 4
    at = 0
    for b, n in enumerate(news):
        note(b, k[at:at + n], v[at:at + n])
        at += n
    for s in range(steps):
        n_new = [1, 1, 0, 1]
        release = None
        if s == 2:
            release = torch.tensor([1, 0, 0, 0], dtype=torch.uint8, device=DEV)
            m.k[0], m.v[0] = m.k[0][:0], m.v[0][:0]
        q = torch.randn(B, 1, H, D, generator=g, device=DEV, dtype=torch.bfloat16)
        k, v = rows(B)[:, None], rows(B)[:, None]
        r = rtp_layer_decode_paged(q, k, v, c, ints(n_new), window=window, n_sink=n_sink,
                                   n_sel=n_sel, release=release)
        for b in range(B):
            if n_new[b]:
                note(b, k[b], v[b])
        assert c.seq_lens.tolist() == m.lens
        m.q = q
        sel = r["sel"] if r["sel"] is not None else (None, None)
        m.check(r["o"], r["lse"], window, n_sink, sel=sel[0], count=sel[1])
    return c, m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("roles,H,n_sel", [((1, 0), 8, None), ((1, 0), 8, 6), ((1, 1, 1), 6, 12),
                                           ((0, 0), 8, None)])
def test_cache_steps(dtype, roles, H, n_sel):
    run_cache(dtype, roles, H, 5, n_sel)


def test_selection_of_every_page_is_the_whole_cache():
    c, m = run_cache(torch.bfloat16, (1, 0), 8, 1)
    a = c.attend(m.q, window=40, n_sink=4)
    b = c.attend(m.q, window=40, n_sink=4, n_sel=100)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_against_the_contiguous_kernels():
    """One length for the whole batch, where rtp_dense_attn and rtp_local_attn apply: both
    are within their rounding of the same 64-bit result."""
    m = Made([900, 900], 64, 8, (1, 0), seed=4)
    o, lse = m.attn(window=128, n_sink=4)
    k = torch.stack([x.to(torch.bfloat16) for x in m.k])
    v = torch.stack([x.to(torch.bfloat16) for x in m.v])
    d, dl = rtp_dense_attn(m.q, k, v, q_pos0=899)
    loc, ll = rtp_local_attn(m.q, k, v, (1, 0), window=128, n_sink=4, q_pos0=899)
    d[:, :, 4:], dl[:, 4:] = loc[:, :, 4:], ll[:, 4:]
    assert float((d.float() - o.float()).abs().max()) <= 2e-2
    assert float((dl - lse).abs().max()) <= 1e-2


def test_step_in_a_graph():
    """A captured step replays while the cache grows: lengths, pages and bounds advance on
    the device as in the eager run, over page borders."""
    B, H, roles, steps = 3, 8, (1, 0), 40

    def fresh():
        c = PagedCache(80, 16, roles, batch=B, max_len=400, device=DEV)
        g = torch.Generator(device=DEV).manual_seed(9)
        k = torch.randn(150, 2, D, generator=g, device=DEV, dtype=torch.bfloat16)
        c.append(k, -k, ints([30, 0, 120]))
        data = [torch.randn(B, 1, n, D, generator=g, device=DEV, dtype=torch.bfloat16)
                for _ in range(steps) for n in (H, 2, 2)]
        return c, [data[3 * i:3 * i + 3] for i in range(steps)]

    n_new = ints([1, 0, 1])
    kw = dict(window=50, n_sink=3, n_sel=4)
    c, data = fresh()
    eager = []
    for q, k, v in data:
        r = rtp_layer_decode_paged(q, k, v, c, n_new, **kw)
        eager.append((r["o"].clone(), r["lse"].clone(), r["sel"][0].clone(), c.seq_lens.tolist()))
    c2, data = fresh()
    bufs = [torch.empty_like(x) for x in data[0]]
    for x, y in zip(bufs, data[0]):
        x.copy_(y)
    warm = fresh()[0]
    rtp_layer_decode_paged(*bufs, warm, n_new, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        r = rtp_layer_decode_paged(*bufs, c2, n_new, **kw)
    for (q, k, v), (o, lse, sel, lens) in zip(data, eager):
        for x, y in zip(bufs, (q, k, v)):
            x.copy_(y)
        graph.replay()
        assert torch.equal(r["o"], o) and torch.equal(r["lse"], lse)
        assert torch.equal(r["sel"][0], sel) and c2.seq_lens.tolist() == lens
    assert torch.equal(c.k_pages, c2.k_pages) and torch.equal(c.bounds, c2.bounds)


def test_two_graphs_and_two_streams_at_once():
    """Calls that run at the same time have workspaces of their own: two captured steps on
    two streams, and eager calls beside them, give what they give alone."""
    ms = [Made([3000 + i, 5, 700], 16, 8, (1, 0), seed=i) for i in range(3)]
    kw = dict(window=64, n_sink=2)
    alone = [m.attn(**kw) for m in ms]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for m in ms[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            outs.append(m.attn(**kw))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        third = ms[2].attn(stream=streams[2], **kw)
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for (o, l), (o2, l2) in zip(outs + [third], alone):
            assert torch.equal(o, o2) and torch.equal(l, l2)


def test_calls_run_on_the_given_stream():
    """Work queued behind a long copy on the given stream sees that copy's result."""
    m = Made([500], 16, 4, (1,), seed=2)
    want = m.attn()
    src, s = m.q.clone(), torch.cuda.Stream()
    torch.cuda.synchronize()
    m.q.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.zeros(1 << 28, device=DEV)
        for _ in range(4):
            big += 1
        m.q.copy_(src)
    got = m.attn(stream=s)
    s.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_tensors_may_go_while_another_stream_uses_them():
    """Inputs that the caller drops, and outputs it drops, right after a call on another
    stream: their memory is not handed out before that stream is done with them."""
    m = Made([500], 16, 4, (1,), seed=2)
    want = m.attn()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        q, table = m.q.clone(), m.table.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            big = torch.zeros(1 << 28, device=DEV)
            for _ in range(4):
                big += 1
        got = rtp_paged_attn_decode(q, m.k_pages, m.v_pages, table, m.seq_lens, m.roles, stream=s)
        del q, table
        junk = [torch.full_like(m.q, float("nan")) for _ in range(8)]
        junk += [torch.full_like(m.table, 10 ** 6) for _ in range(8)]
        s.synchronize()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        # the outputs: read here behind a long queue, dropped, then s allocates again
        torch.cuda.current_stream().wait_stream(s)
        slow = torch.zeros(1 << 28, device=DEV)
        for _ in range(4):
            slow += 1
        copy = got[0].clone()
        del got
        with torch.cuda.stream(s):
            junk += [torch.full((m.q.numel() + 8,), 7.0, dtype=torch.bfloat16, device=DEV)
                     for _ in range(8)]
        torch.cuda.synchronize()
        assert torch.equal(want[0], copy)
        del junk


# ------------------------------------------------------------------------------------- refusals
def test_python_refusals():
    m = Made([40, 3], 16, 4, (1, 0), "e4m3", seed=1)
    a = dict(window=5)
    bad = [dict(q=m.q.float()), dict(q=m.q[:, 0]), dict(q=m.q[:1]), dict(q=m.q.cpu()),
           dict(q=m.q[..., :64]), dict(k_pages=m.k_pages.to(torch.bfloat16)),
           dict(v_pages=m.v_pages[:1]), dict(k_pages=m.k_pages[:, :, :1]),
           dict(k_pages=m.k_pages.transpose(2, 3)), dict(table=m.table.long()),
           dict(table=m.table[:1]), dict(table=m.table.t()), dict(seq_lens=m.seq_lens.long()),
           dict(seq_lens=m.seq_lens[:1]), dict(roles=(1, 2)), dict(roles=()), dict(roles=(1,)),
           dict(roles=(1, 0, 1))]
    for kw in bad:
        args = dict(q=m.q, k_pages=m.k_pages, v_pages=m.v_pages, table=m.table,
                    seq_lens=m.seq_lens, roles=m.roles)
        args.update(kw)
        with pytest.raises(ValueError):
            rtp_paged_attn_decode(*args.values(), **a)
    sel = ints([[[0]], [[0]]])
    one = ints([[1], [1]])
    for kw in (dict(), dict(window=5, k_scale=m.k_scale[:1]), dict(window=5, v_scale=m.v_scale.double()),
               dict(window=5, sel=sel), dict(window=5, sel=sel[:1], sel_count=one),
               dict(window=5, sel=sel, sel_count=one[:1]), dict(window=5, o=m.q[:1]),
               dict(window=5, lse=torch.zeros(2, 4, device=DEV))):
        with pytest.raises(ValueError):
            rtp_paged_attn_decode(m.q, m.k_pages, m.v_pages, m.table, m.seq_lens, m.roles, **kw)
    with pytest.raises(RtpError):
        m.attn(window=0)
    with pytest.raises(RtpError):
        m.attn(window=5, scale=-1.0)
    bf = Made([40, 3], 16, 4, (1, 0), seed=1)
    with pytest.raises(ValueError):
        bf.attn(window=5, k_scale=m.k_scale)
    with pytest.raises(RtpError):
        Made([40], 16, 34, (1, 1), seed=1).attn()
    with pytest.raises(ValueError):
        PagedCache(4, 16, (1,), batch=1, max_len=16, device=DEV, bounds=False).attend(
            m.q[:1, :, :1], n_sel=4)


def test_python_refusals_of_plan_write_and_select():
    m = Made([40, 3], 16, 4, (1, 0), seed=1)
    fp, fc, lens = ints([0, 1]), ints([2]), m.seq_lens
    for args, kw in [((lens.long(), lens, m.table, fp, fc), {}), ((lens, lens[:1], m.table, fp, fc), {}),
                     ((lens, lens, m.table[:1], fp, fc), {}), ((lens, lens, m.table, fp.long(), fc), {}),
                     ((lens, lens, m.table, fp, ints([1, 2])), {}),
                     ((lens, lens, m.table, fp, fc), dict(max_tokens=-1)),
                     ((lens, lens, m.table, fp, fc), dict(row_tokens=-1)),
                     ((lens, lens, m.table, fp, fc), dict(page_size=0)),
                     ((lens, lens, m.table, fp, fc), dict(release=lens)),
                     ((lens, lens, m.table, fp, fc), dict(out=dict(x=lens))),
                     ((lens, lens, m.table, fp, fc), dict(out=dict(slot_map=lens)))]:
        with pytest.raises(ValueError):
            rtp_paged_plan(*args, **dict(dict(page_size=16, max_tokens=5), **kw))
    with pytest.raises(RtpError):
        rtp_paged_plan(lens, lens, m.table, fp, fc, page_size=24, max_tokens=5)
    k = torch.zeros(3, 2, D, dtype=torch.bfloat16, device=DEV)
    slot = ints([0, 1, 2])
    for args in [(k.float(), k, slot), (k, k[:2], slot), (k, k, slot[:2]), (k[:, :1], k, slot),
                 (k, k, slot.long()), (k[0], k, slot), (k.transpose(0, 1), k, slot)]:
        with pytest.raises(ValueError):
            rtp_paged_kv_write(*args, m.k_pages, m.v_pages)
    b, s = random_bounds(m.k_pages.shape[0], 1, 1)
    spans = ints([[0, 1, 0, 0]])
    for args in [(spans[0], (1, 0), b, s), (spans, (1,), b, s), (spans, (1, 1), b, s),
                 (spans, (1, 0), b.float(), s), (spans, (1, 0), b, s[:1])]:
        with pytest.raises(ValueError):
            rtp_paged_kv_append(k, k, args[0], m.k_pages, m.v_pages, *args[1:])
    for kw in (dict(n_sel=0), dict(q=m.q[:1]), dict(b=b[:1]), dict(lens=lens.long())):
        a = dict(q=m.q, b=b, s=s, t=m.table, lens=lens, roles=(1, 0), n_sel=4)
        a.update(kw)
        with pytest.raises(ValueError):
            rtp_paged_block_select(a["q"], a["b"], a["s"], a["t"], a["lens"], a["roles"],
                                   page_size=16, n_sel=a["n_sel"])
    with pytest.raises(RtpError):
        rtp_paged_block_select(m.q, b, s, m.table, lens, (1, 0), page_size=16, n_sel=4, n_first=3,
                               n_recent=2)
