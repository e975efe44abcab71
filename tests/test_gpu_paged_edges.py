"""Edges of the paged-cache operators on the GPU: calls that the interface allows and
that test_gpu_paged.py does not make.  Plain implementations and tolerances as there.
"""
import numpy as np
import pytest
import torch

import paged_ref as ref
from long_context_sparse_rtp_b200 import (PagedCache, RtpError, rtp_layer_decode_paged,
                                          rtp_paged_attn_decode, rtp_paged_block_select,
                                          rtp_paged_plan)
from test_gpu_paged import (D, DEV, I32, RAGGED, Made, _gpu, check_plan, check_select, ints,  # noqa: F401
                            random_bounds, tables)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- a batch without tokens
@pytest.mark.parametrize("B", [1, 1024, 1025, 2500])
@pytest.mark.parametrize("release", [False, True])
def test_plan_without_tokens(B, release):
    """max_tokens = 0: nothing is taken, released pages go back, requests that want tokens are
    refused."""
    g = np.random.default_rng(B)
    lens = g.integers(0, 60, B).tolist()
    rel = (g.random(B) < 0.5).astype(int).tolist() if release else None
    for in_place in (False, True):
        check_plan(lens, [0] * B, ps=16, width=5, free=7, cap=12000, max_tokens=0, release=rel,
                   in_place=in_place)
    check_plan(lens, (g.integers(0, 2, B)).tolist(), ps=16, width=5, free=7, cap=12000, max_tokens=0,
               release=rel)


def test_plan_without_tokens_pads_its_spans():
    B = 2000
    spans = ints([[9, 9, 9, 9]] * 5)
    r = rtp_paged_plan(ints([3] * B), ints([0] * B), ints([[1]] * B), ints([0]), ints([0]), page_size=16,
                       max_tokens=0, out=dict(spans=spans))
    assert r["spans"].tolist() == [[-1, 0, 0, 0]] * 5


# ------------------------------------------------------------------- pages always kept
@pytest.mark.parametrize("width", [40, 200, 700, 4096, 17000])
@pytest.mark.parametrize("share", [0.3, 1.0])
def test_select_keeps_forced_pages_before_infinite_scores(width, share):
    """More pages of scale inf than the list holds: the first and the last ones stay in it."""
    lens = [16 * width, 16 * width - 37, 16 * 30]
    table, n_pages = tables(lens, 16, width, seed=width)
    b, s = random_bounds(n_pages, 2, 3)
    g = torch.Generator(device=DEV).manual_seed(7)
    s[torch.rand(s.shape, generator=g, device=DEV) < share] = float("inf")
    q = torch.randn(3, 1, 4, D, generator=g, device=DEV, dtype=torch.bfloat16)
    for n_sel, n_first, n_recent in [(1, 0, 1), (1, 1, 0), (4, 1, 1), (9, 0, 9), (20, 7, 5),
                                     (width // 2, 3, 5)]:
        check_select(q, b, s, table, lens, (1, 1), 16, n_sel, n_first, n_recent)
        sel, _ = rtp_paged_block_select(q, b, s, table, ints(lens), (1, 1), page_size=16,
                                        n_sel=n_sel, n_first=n_first, n_recent=n_recent)
        for i, n in enumerate(lens):
            nb = ref.up(n, 16)
            forced = set(range(n_first)) | set(range(nb - n_recent, nb))
            for row in sel[i].tolist():
                assert {p for p in forced if 0 <= p < nb} <= set(row)


def test_select_keeps_forced_pages_before_scores_that_overflow():
    lens = [16 * 50]
    table, n_pages = tables(lens, 16, 50, seed=3)
    b, s = random_bounds(n_pages, 1, 4)
    b[:, :, 1] = 127  # every page's product overflows
    s[:] = 3e38
    q = torch.full((1, 1, 2, D), 3e38, device=DEV, dtype=torch.bfloat16)
    check_select(q, b, s, table, lens, (1,), 16, 3, 1, 2)
    sel, _ = rtp_paged_block_select(q, b, s, table, ints(lens), (1,), page_size=16, n_sel=3,
                                    n_first=1, n_recent=2)
    assert sel.flatten().tolist() == [0, 48, 49]


# ------------------------------------------------------------------- signs of 8-bit scales
K_SCALES = [-0.02, 0.0, 0.013, -0.0, 1e-44, -1e-39, 1.2e-38, -3.0]


@pytest.mark.parametrize("H", [8, 64, 128])
@pytest.mark.parametrize("lens", [RAGGED, [20000, 3, 1037]])
def test_attn_k_scales_of_any_sign(H, lens):
    """value = scale * stored for negative, zero and tiny scales too: masked keys stay masked,
    the running maximum is that of the scores."""
    roles = (1, 0, 1, 1, 0, 1, 1, 1)
    m = Made(lens, 16, H, roles, "e4m3", seed=H)
    new = torch.tensor(K_SCALES, device=DEV)
    m.k = [k / m.k_scale.double()[:, None] * new.double()[:, None] for k in m.k]
    m.k_scale = new
    m.check(*m.attn(window=37, n_sink=5), 37, 5)


def test_attn_k_scale_not_a_number():
    """A scale of NaN or infinity reaches its own head's outputs and no others."""
    m = Made([40, 0, 5], 16, 4, (1, 1, 1, 1), "e4m3", seed=1)
    m.k_scale[1], m.k_scale[2] = float("nan"), float("inf")
    o, lse = m.attn()
    for b in (0, 2):
        assert bool(o[b, 0, 1:3].isnan().all()) and bool(lse[b, 1:3].isnan().all())
        assert bool(o[b, 0, [0, 3]].isfinite().all())
    assert bool((o[1] == 0).all()) and bool((lse[1] == float("-inf")).all())


# ------------------------------------------------------------------- captured, another stream
def test_capture_on_another_stream_keeps_memory_in_use():
    """Inside a capture too, what a call on another stream used or returned and the caller
    dropped is not handed out again while the other stream may be using it."""
    m = Made([700, 3], 16, 8, (1, 0), seed=5)
    kw = dict(window=40, n_sink=2)
    want = m.attn(**kw)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        o, lse = m.attn(stream=side, **kw)
        first = o.data_ptr()
        main.wait_stream(side)
        copy = o.clone()  # main reads it; side does not wait for that
        del o, lse
        o2, lse2 = m.attn(stream=side, **kw)
        second = o2.data_ptr()
        main.wait_stream(side)
        q = m.q.clone()
        used = q.data_ptr()
        side.wait_stream(main)
        o3, lse3 = rtp_paged_attn_decode(q, m.k_pages, m.v_pages, m.table, m.seq_lens, m.roles,
                                         stream=side, **kw)
        del q
        junk = torch.full_like(m.q, float("nan"))  # main does not wait for side
        reused = junk.data_ptr() == used
        main.wait_stream(side)
    assert first != second and not reused
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for x in (copy, o2, o3):
            assert torch.equal(x, want[0])
        assert torch.equal(lse2, want[1]) and torch.equal(lse3, want[1])


# ------------------------------------------------------------------- refused steps
def state(c):
    return [x.clone() for x in (c.seq_lens, c.free_count, c.free_pages, c.block_table)]


def unchanged(c, was):
    return all(torch.equal(x, y) for x, y in zip(state(c), was))


def half_full(dtype=torch.bfloat16, **kw):
    c = PagedCache(40, 16, (1, 0), batch=3, max_len=200, device=DEV, dtype=dtype, **kw)
    k = torch.randn(37, 2, D, device=DEV, dtype=torch.bfloat16)
    c.append(k, k, ints([20, 0, 17]))
    return c, state(c)


@pytest.mark.parametrize("bounds", [True, False])
def test_refused_append_changes_nothing(bounds):
    """Rows that the write would refuse are refused before the plan takes their pages."""
    c, was = half_full(bounds=bounds)
    k = torch.randn(5, 2, D, device=DEV, dtype=torch.bfloat16)
    wide = torch.randn(5, 2 * D + 4, device=DEV, dtype=torch.bfloat16)
    odd = torch.randn(5 * 2 * D + 4, device=DEV, dtype=torch.bfloat16)[4:].view(5, 2, D)
    value = [(k, k[:4]), (k, k.float()), (k.float(), k), (k, k[:, :1]), (k[:, :1], k[:, :1]),
             (k, k.cpu()), (k, k[:, 0]), (k, k.transpose(1, 2).contiguous().transpose(1, 2)),
             (k, k.flip(0).transpose(0, 1)), (k[..., :64], k[..., :64])]
    refused = [(k, wide[:, :2 * D].view(5, 2, D)), (wide[:, :2 * D].view(5, 2, D), k), (odd, k), (k, odd),
               (k[:1].expand(5, 2, D), k)]
    release = torch.tensor([1, 0, 1], dtype=torch.uint8, device=DEV)
    for error, pairs in ((ValueError, value), (RtpError, refused)):
        for x, y in pairs:
            with pytest.raises(error):
                c.append(x, y, ints([2, 2, 1]), release=release)
            assert unchanged(c, was)
    assert c.append(k, k, ints([2, 2, 1]))["admitted"].tolist() == [1, 1, 1]


def test_refused_append_to_a_cache_with_bad_scales_changes_nothing():
    k = torch.randn(5, 2, D, device=DEV, dtype=torch.bfloat16)
    for dtype, scale in ((torch.bfloat16, torch.ones(2, device=DEV)), (torch.float16, None),
                         (torch.float8_e4m3fn, torch.ones(3, device=DEV))):
        c = PagedCache(40, 16, (1, 0), batch=3, max_len=200, device=DEV, dtype=dtype, k_scale=scale)
        was = state(c)
        with pytest.raises(ValueError):
            c.append(k, k, ints([2, 2, 1]))
        assert unchanged(c, was)


def test_refused_step_changes_nothing():
    """A step whose attention or selection would be refused is refused before its tokens are
    taken."""
    q = torch.randn(3, 1, 8, D, device=DEV, dtype=torch.bfloat16)
    k = torch.randn(3, 1, 2, D, device=DEV, dtype=torch.bfloat16)
    ok = dict(q=q, k=k, v=k, window=9, n_sel=4)
    c, was = half_full()
    for kw in (dict(q=q.float()), dict(q=q[:2]), dict(q=q[:, 0]), dict(q=q[:, :, :7]), dict(q=q.cpu()),
               dict(k=k[:2]), dict(k=k[:, 0]), dict(v=k.float()), dict(v=k[:, :, :1]),
               dict(k=k.expand(3, 2, 2, D), v=k.expand(3, 2, 2, D)), dict(k=k[:2], v=k[:2]),
               dict(window=None), dict(n_sel=0), dict(o=q[:2]), dict(lse=torch.zeros(3, 8, device=DEV)),
               dict(window=0), dict(n_sink=-1), dict(n_sel=1), dict(n_first=9), dict(n_recent=-1),
               dict(scale=0.0), dict(scale=float("nan"))):
        a = dict(ok, **kw)
        args = [a.pop(x) for x in ("q", "k", "v")]
        with pytest.raises((ValueError, RtpError)):
            rtp_layer_decode_paged(*args, c, ints([1, 0, 1]), **a)
        assert unchanged(c, was), kw
    bare, was2 = half_full(bounds=False)
    with pytest.raises(ValueError):
        rtp_layer_decode_paged(q, k, k, bare, ints([1, 0, 1]), window=9, n_sel=4)
    assert unchanged(bare, was2)
    a = dict(ok)
    r = rtp_layer_decode_paged(*[a.pop(x) for x in ("q", "k", "v")], c, ints([1, 0, 1]), **a)
    assert r["plan"]["admitted"].tolist() == [1] * 3 and c.seq_lens.tolist() == [21, 0, 18]


# ------------------------------------------------------------------- other requests
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_other_requests_change_only_the_rounding(kv):
    """A request alone and beside others (another split, another running maximum): both within
    the bound of P's rounding.  Other values beside it, of the same lengths: the same bits."""
    lens = [517, 9000, 3, 517, 0, 40, 2500] + [77] * 40
    m = Made(lens, 16, 8, (1, 0), kv, seed=21)
    kw = dict(window=100, n_sink=3)
    o, lse = m.attn(**kw)
    m.check(o, lse, 100, 3)
    u16 = 2.0 ** -11 if kv == "e4m3" else 2.0 ** -8
    for b in (0, 1, 2, 6):
        a, la = rtp_paged_attn_decode(m.q[b:b + 1], m.k_pages, m.v_pages, m.table[b:b + 1],
                                      m.seq_lens[b:b + 1], m.roles, k_scale=m.k_scale,
                                      v_scale=m.v_scale, **kw)
        for g in range(2):
            keys = ref.keys_of(lens[b], m.roles[g], 16, 100, 3)
            h = slice(4 * g, 4 * g + 4)
            eo, el, mag, sqk = ref.attend(m.q[b, 0, h], m.k[b][keys, g], m.v[b][keys, g], D ** -0.5)
            e = (128 * 2.0 ** -24 + 2.0 ** -22) * sqk * D ** -0.5
            nn = len(keys) * 2.0 ** -24
            # two results, each within test_gpu_paged.py's bound of the exact value
            tol = 2 * (2.0 ** -8 * eo.abs() + (u16 + 2 * e + 2.0 ** -20 + nn) * mag)
            assert bool(((a[0, 0, h].double() - o[b, 0, h].double()).abs() <= tol).all())
            lt = 2 * (e + nn + 2.0 ** -20 * (1 + float(el.abs().max())))
            assert float((la[0, h] - lse[b, h]).abs().max()) <= lt
    for b in (0, 6):  # the others' pages and queries change, this request's do not
        keep = m.table[b, :ref.up(lens[b], 16)].long()
        kp, vp, q = m.k_pages.clone(), m.v_pages.clone(), -m.q
        mine = torch.zeros(kp.shape[0], dtype=torch.bool, device=DEV)
        mine[keep] = True
        for pages in (kp, vp):
            bytes_ = pages.view(torch.uint8)
            bytes_[~mine] = bytes_[~mine].flip(0)
        q[b] = m.q[b]
        o2, lse2 = rtp_paged_attn_decode(q, kp, vp, m.table, m.seq_lens, m.roles, k_scale=m.k_scale,
                                         v_scale=m.v_scale, **kw)
        assert torch.equal(o2[b], o[b]) and torch.equal(lse2[b], lse[b])


# ------------------------------------------------------------------- long loops
@pytest.mark.parametrize("kv,n", [("bf16", 1300011), ("e4m3", 2000011)])
@pytest.mark.parametrize("H", [8, 16])
@pytest.mark.parametrize("listed", [False, True])
def test_attn_runs_of_more_than_64_tiles(kv, n, H, listed):
    """Runs long enough to look their pages up three times (32 tiles each).  Keys of zero: the
    sums count the keys, exactly.  128 keys that one query each singles out: its value comes
    back exactly, from the places around every look-up and elsewhere."""
    ps, dtype = 64, torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    g = torch.Generator(device=DEV).manual_seed(n % 1000 + H)
    nb = ref.up(n, ps)
    table = torch.randperm(nb, generator=g, device=DEV).to(I32)[None]
    kp = torch.zeros(nb, ps, 1, D, device=DEV).to(dtype)
    vp = torch.randint(-15, 16, (nb, ps, 1, D), generator=g, device=DEV, dtype=torch.int8).to(dtype)
    lens = ints([n])
    kw = {}
    if listed:
        kw = dict(sel=torch.arange(nb, device=DEV, dtype=I32)[None, None].contiguous(),
                  sel_count=ints([[nb]]))
    q = torch.zeros(1, 1, H, D, device=DEV, dtype=torch.bfloat16)

    def attn():
        return rtp_paged_attn_decode(q, kp, vp, table, lens, (1,), **kw)

    o, lse = attn()
    # P = 1 for every key: l is a whole number below 2^24 and exact, its logarithm and the
    # product with ln 2 are each rounded; sixteen keys more or less would be 8e-6
    assert float((lse.double() - np.log(n)).abs().max()) <= 2.0 ** -22 * (1 + np.log2(n))
    ctas = 296 if kv == "bf16" else 444
    chunk = ref.up(ref.up(n, 64) + 5, ctas)  # tiles a CTA takes of the line
    assert chunk > 64
    offs = [0, 1, 15, 16, 17, 30, 31, 32, 33, 47, 48, 49, 62, 63, 64, 65]
    starts = torch.randint(1, ctas - 20, (7,), generator=g, device=DEV).tolist()
    tiles = [c * chunk - 5 + x for c in starts for x in offs]
    assert max(tiles) < n // 64
    pos = [t * 64 + int(torch.randint(0, 64, (1,), generator=g, device=DEV)) for t in tiles]
    pos += [0, 63, 64, n - 1, n - 12] + torch.randint(0, n, (128 - len(pos) - 5,), generator=g,
                                                     device=DEV).tolist()
    pos = torch.tensor(pos, device=DEV)
    page, row = table[0].long()[pos // ps], pos % ps
    kp[page, row, 0, torch.arange(128, device=DEV)] = torch.tensor(64.0, device=DEV).to(dtype)
    # a score of 64 * 64 * scale = 362 against 0: the others' weights are below 2^-149
    for d0 in range(0, 128, H):
        q.zero_()
        q[0, 0, torch.arange(H, device=DEV), torch.arange(d0, d0 + H, device=DEV)] = 64.0
        o, lse = attn()
        assert torch.equal(o[0, 0].float(), vp[page, row, 0][d0:d0 + H].float())


@pytest.mark.parametrize("B,width,H,roles", [
    (48, 257, 2, (1,)), (48, 512, 16, (1,)), (24, 1000, 8, (1, 1, 0, 1, 1)), (96, 1000, 1, (1,)),
    (192, 2048, 1, (1,)), (96, 2051, 2, (1,)), (192, 3000, 1, (1,)), (3, 300, 16, (1,)),
    (3, 5000, 32, (1, 1)), (40, 2500, 32, (1, 1)), (2, 20000, 12, (1,))])
def test_select_many_rows_and_rounds(B, width, H, roles):
    """Rows that fill the GPU score several rounds of pages a CTA, in one kernel and in two; more
    than eight query heads per kv head in both."""
    if H % len(roles):
        H = len(roles)
    lens = [16 * width] + [16 * (1 + (width * (37 * i % 101)) // 101) - i % 16 for i in range(1, B)]
    table, n_pages = tables(lens, 16, width, seed=B + width)
    b, s = random_bounds(n_pages, sum(roles), H)
    g = torch.Generator(device=DEV).manual_seed(B)
    q = torch.randn(B, 1, H, D, generator=g, device=DEV, dtype=torch.bfloat16)
    check_select(q, b, s, table, lens, roles, 16, min(90, width // 2), 1, 2)


# ------------------------------------------------------------------- precision
@pytest.mark.parametrize("H,roles", [(4, (1, 1)), (32, (1, 0))])
def test_attn_bf16_probabilities_with_their_remainder(H, roles):
    """bf16 pages: P cut off to bf16 leaves a remainder of 2^-7 P at most, which is rounded to
    bf16 (2^-8 of it): off by 2^-15 of P, far below what one bf16 number (2^-8) would leave in
    outputs near zero."""
    lens = [17, 40, 120, 300, 16 * 1700]
    m = Made(lens, 16, H, roles, seed=H)
    m.q *= 0.25
    o, _ = m.attn(window=60, n_sink=3)
    for b, n in enumerate(lens[:4]):
        for g, role in enumerate(roles):
            h = slice(g * m.G, (g + 1) * m.G)
            idx = torch.tensor(ref.keys_of(n, role, 16, 60, 3), device=DEV)
            eo, _, mag, sqk = ref.attend(m.q[b, 0, h], m.k[b][idx, g], m.v[b][idx, g], D ** -0.5)
            e = (128 * 2.0 ** -24 + 2.0 ** -22) * sqk * D ** -0.5
            tol = 2.0 ** -8 * eo.abs() + (2.0 ** -15 + 2 * e + 2.0 ** -20 + len(idx) * 2.0 ** -24) * mag
            err = (o[b, 0, h].double() - eo).abs()
            assert bool((err <= tol).all()), (b, g, float((err / tol).max()))


def test_attn_infinite_values_beside_probabilities_that_bf16_holds():
    """P = 1, 1 / 2, 0.3 and so on: each sign of infinity in V comes back as it is."""
    m = Made([1, 2, 17], 16, 2, (1, 1), seed=1)
    m.q[0], m.q[1] = 0, 0
    for b in range(3):
        page = int(m.table[b, 0])
        m.v_pages[page, 0, :, 3], m.v_pages[page, 0, :, 4] = float("inf"), float("-inf")
    o, lse = m.attn()
    assert bool((o[..., 3] == float("inf")).all()) and bool((o[..., 4] == float("-inf")).all())
    rest = [d for d in range(D) if d not in (3, 4)]
    assert bool(o[..., rest].isfinite().all()) and bool(lse.isfinite().all())


def test_attn_small_probabilities_beside_8_bit_pages():
    """Peaked rows: P below 2^-22 of the largest is subnormal in fp16, off by 2^-33 of the
    largest at most, which outputs next to zero show (a V of zero beside the largest P)."""
    m = Made([60, 300, 5], 16, 16, (1, 1, 1, 1), "e4m3", seed=5)
    m.q *= 20
    page = m.v_pages.view(torch.uint8)
    for b in range(3):
        for g in range(4):
            best = int((m.q[b, 0, 4 * g].double() @ m.k[b][:, g].T).argmax())
            page[int(m.table[b, best // 16]), best % 16, g] = 0
            m.v[b][best, g] = 0
    o, _ = m.attn()
    for b, n in enumerate(m.lens):
        for g in range(4):
            h = slice(4 * g, 4 * g + 4)
            eo, _, mag, sqk = ref.attend(m.q[b, 0, h], m.k[b][:, g], m.v[b][:, g], D ** -0.5)
            e = (128 * 2.0 ** -24 + 2.0 ** -22) * sqk * D ** -0.5
            tol = 2.0 ** -8 * eo.abs() + (2.0 ** -11 + 2 * e + 2.0 ** -20 + n * 2.0 ** -24) * mag + \
                n * 2.0 ** -33 * float(m.v[b][:, g].abs().max())
            assert bool(((o[b, 0, h].double() - eo).abs() <= tol).all()), (b, g)
