"""The paged-cache operators as a serving program calls them, beside their plain forms.

  plan     block tables, slot map and page spans of a step, from request lengths
  write    new K/V rows into pages by a slot map
  append   the same by page spans, with the touched pages' bounds refreshed
  attn     one token per request over its pages (retrieval heads: every key, local heads: sinks and window)
  sparse   pages chosen per kv head by a cheap integer score, then attention over them

``run`` computes the plain form (elementary torch operations, 32 bits) unless ``own`` is set, which makes the
library's calls instead.
"""
import random

import torch

own = False

DEV = "cuda"
D = 128
#: pages a request's table holds beyond its present need
SPARE = 3


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's bookkeeping for 64 running requests: latency alone counts
        dict(name="plan_step_b64", op="plan", B=64, page=64, lo=1, hi=8192, new_lo=1, new_hi=1),
        # a burst of prompts beside running requests, small pages: 200 K tokens get their slots
        dict(name="plan_prompts_b301", op="plan", B=301, page=16, lo=0, hi=4000, new_lo=1, new_hi=1400),
        # the decode step's own token of 64 requests, bounds of 64 part-filled pages refreshed
        dict(name="append_step_b64", op="append", B=64, page=64, lo=0, hi=8191, new_lo=1, new_hi=1, Hkv=4,
             roles="1100", kv="bf16"),
        # five prompts, 128 K tokens in all, into fresh and part-filled pages
        dict(name="append_prompts_128k", op="append", B=5, page=64, lo=0, hi=1000, new_lo=9001, new_hi=43427,
             Hkv=4, roles="1000", kv="bf16"),
        # a chunk of prompts into an 8-bit cache by a slot map of their own
        dict(name="write_e4m3_20k", op="write", B=7, page=16, lo=0, hi=333, new_lo=2001, new_hi=3717, Hkv=8,
             roles="11111111", kv="e4m3"),
        # one user, a short context: latency alone counts
        dict(name="attn_b1_517", op="attn", B=1, page=16, lo=517, hi=517, H=8, Hkv=2, roles="11", kv="bf16",
             window=0, n_sink=0),
        # a full decode batch of ragged requests, one row of it unused, every head over every key
        dict(name="attn_b64_8k", op="attn", B=64, page=64, lo=0, hi=8192, H=32, Hkv=4, roles="1111", kv="bf16",
             window=0, n_sink=0),
        # the benchmark's decode batch in pages: one retrieval kv head of four, window 4096 + 4 sinks
        dict(name="attn_b8_128k_mixed", op="attn", B=8, page=64, lo=120011, hi=131072, H=32, Hkv=4, roles="1000",
             kv="bf16", window=4096, n_sink=4),
        # the same lengths in an 8-bit cache, every head over every key
        dict(name="attn_b8_128k_e4m3", op="attn", B=8, page=128, lo=120011, hi=131072, H=32, Hkv=4, roles="1111",
             kv="e4m3", window=0, n_sink=0),
        # the decode batch with 64 of up to 2048 pages kept on the retrieval head
        dict(name="sparse_b8_128k", op="sparse", B=8, page=64, lo=120011, hi=131072, H=32, Hkv=4, roles="1000",
             kv="bf16", window=4096, n_sink=4, n_sel=64),
        # ragged requests, small 8-bit pages, every kv head selecting
        dict(name="sparse_b24_32k_e4m3", op="sparse", B=24, page=16, lo=700, hi=32768, H=16, Hkv=4, roles="1111",
             kv="e4m3", window=0, n_sink=0, n_sel=128),
        # one request of a million tokens
        dict(name="sparse_b1_1m", op="sparse", B=1, page=64, lo=1048003, hi=1048003, H=32, Hkv=4, roles="1111",
             kv="bf16", window=0, n_sink=0, n_sel=256),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over their logarithm."""
    return min(hi, max(lo, int(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["plan", "append", "write", "attn", "attn", "sparse", "sparse"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 400)
        new_hi = rng.choice([1, _log(rng, 2, 180_000 // B + 2)])
        return dict(op=op, B=B, page=page, lo=0, hi=_log(rng, 1, 8192), new_lo=rng.choice([0, 1]), new_hi=new_hi)
    G, Hkv = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    roles = "".join(rng.choice("01") for _ in range(Hkv))
    kv = rng.choice(["bf16", "e4m3"])
    if op in ("append", "write"):
        B = _log(rng, 1, 96)
        new_hi = rng.choice([1, _log(rng, 2, 400_000 // (B * Hkv) + 2)])
        return dict(op=op, B=B, page=page, lo=0, hi=_log(rng, 1, 4096), new_lo=1, new_hi=new_hi, Hkv=Hkv,
                    roles=roles if op == "append" else "1" * Hkv, kv=kv)
    B = _log(rng, 1, 96)
    hi = _log(rng, 16, max(17, 2_000_000 // (B * Hkv)))
    if op == "sparse":
        roles = "1" + roles[1:]
    case = dict(op=op, B=B, page=page, lo=_log(rng, 1, hi), hi=hi, H=G * Hkv, Hkv=Hkv, roles=roles, kv=kv,
                window=_log(rng, 1, 4096), n_sink=rng.choice([0, 1, 4, 33]))
    if op == "sparse":
        case["n_sel"] = _log(rng, 4, 256)
    return case


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], from the case alone: the last is hi, the others by the golden section."""
    out = [lo + int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]
    out[-1] = hi
    return out


def _lens(c):
    return _spread(c["B"], c["lo"], c["hi"])


def _news(c):
    return _spread(c["B"], c["new_lo"], c["new_hi"])


def _up(a, b):
    return -(-a // b)


def _spans_cap(T, B, page):
    return min(T, T // page + 2 * B)


# ---------------------------------------------------------------------------------------- prepare
def _tables(c, need, gen):
    """Page ids in random order: block tables for `need` pages of each request (-1 behind them), and the pages left."""
    width = max(need) + SPARE
    n_pages = sum(need) + c["B"] * SPARE + 5
    ids = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    used = torch.arange(width, device=DEV)[None, :] < torch.tensor(need, device=DEV)[:, None]
    table = torch.full((c["B"], width), -1, dtype=torch.int32, device=DEV)
    table[used] = ids[:sum(need)]
    return table, ids[sum(need):].contiguous(), n_pages


def _stored(x, kv, scale):
    """Rows as the pages hold them: [..., Hkv, 128] in bf16, or x / scale in e4m3."""
    if kv == "bf16":
        return x.to(torch.bfloat16)
    return (x.float() / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _fill(c, n_pages, gen):
    """K and V pages: keys drift from page to page, as the keys of neighbouring tokens do."""
    shape = (n_pages, c["page"], c["Hkv"], D)
    sk = torch.full((c["Hkv"],), 0.0131, device=DEV) if c["kv"] == "e4m3" else None
    sv = torch.full((c["Hkv"],), 0.0117, device=DEV) if c["kv"] == "e4m3" else None
    k = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    k += torch.randn((n_pages, 1, c["Hkv"], D), generator=gen, device=DEV, dtype=torch.bfloat16) * 0.6
    v = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    if c["kv"] == "e4m3":
        return _stored(k, "e4m3", sk), _stored(v, "e4m3", sv), sk, sv
    return k, v, None, None


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    lens, ps = _lens(c), c["page"]
    s = dict(c=c, page=ps, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    if c["op"] in ("plan", "append", "write"):
        news = _news(c)
        need = [_up(n, ps) for n in lens]
        total = [_up(n + m, ps) for n, m in zip(lens, news)]
        s["n_new"] = torch.tensor(news, dtype=torch.int32, device=DEV)
        s["T"] = sum(news)
        extra = sum(total) - sum(need)
        table, spare, n_pages = _tables(c, [max(a, b) for a, b in zip(need, total)], gen)
        if c["op"] == "plan":
            # the tables hold the present pages; the pages to come lie on the free stack
            keep = torch.arange(table.shape[1], device=DEV)[None, :] < torch.tensor(need, device=DEV)[:, None]
            coming = table[(table >= 0) & ~keep]
            table[~keep] = -1
            s["free_pages"] = torch.cat([spare, coming]).contiguous()
            s["free_count"] = torch.tensor([len(spare) + extra], dtype=torch.int32, device=DEV)
            s["max_tokens"] = _up(s["T"], 64) * 64  # a captured step pads its batch
            s["table"] = table
            return s
        # the rows to write, and where they go (what rtp_paged_plan gives for these lengths)
        rows = torch.repeat_interleave(torch.arange(c["B"], device=DEV), s["n_new"].long())
        start = torch.cumsum(s["n_new"].long(), 0) - s["n_new"].long()
        pos = torch.arange(s["T"], device=DEV) - start[rows] + s["seq_lens"].long()[rows]
        s["slot_map"] = (table[rows, pos // ps].long() * ps + pos % ps).to(torch.int32)
        first, last = [n // ps for n in lens], total
        spans = [(b, p) for b in range(c["B"]) for p in range(first[b], last[b])]
        b_of, p_of = (torch.tensor([x[i] for x in spans], device=DEV) for i in (0, 1))
        old, new = s["seq_lens"].long()[b_of], (s["seq_lens"] + s["n_new"]).long()[b_of]
        n_rows = torch.clamp(new - p_of * ps, max=ps)
        fresh = torch.clamp(old - p_of * ps, min=0)
        token = start[b_of] + p_of * ps + fresh - old
        cap = _spans_cap(s["T"], c["B"], ps)
        s["spans"] = torch.tensor([-1, 0, 0, 0], dtype=torch.int32, device=DEV).repeat(cap, 1)
        s["spans"][:len(spans)] = torch.stack([table[b_of, p_of].long(), n_rows, fresh, token], 1).to(torch.int32)
        s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"] = _fill(c, n_pages, gen)
        # k and v are slices of one projection's output, as a layer has them
        qkv = torch.randn((s["T"], 2, c["Hkv"], D), generator=gen, device=DEV, dtype=torch.bfloat16)
        s["k"], s["v"] = qkv[:, 0], qkv[:, 1]
        if c["op"] == "append":
            s["bounds"], s["bound_scale"] = _bounds(_retrieval(s["k_pages"], c).float())
        return s
    table, _, n_pages = _tables(c, [_up(n, ps) for n in lens], gen)
    s["table"] = table
    s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"] = _fill(c, n_pages, gen)
    s["q"] = torch.randn((c["B"], 1, c["H"], D), generator=gen, device=DEV, dtype=torch.bfloat16)
    if c["op"] == "sparse":
        s["bounds"], s["bound_scale"] = _all_bounds(s["k_pages"], c)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _roles(c):
    return [int(x) for x in c["roles"]]


def _kv_heads(c, role):
    return torch.tensor([g for g, r in enumerate(_roles(c)) if r == role], dtype=torch.long, device=DEV)


def _retrieval(pages, c):
    return pages if "0" not in c["roles"] else pages[:, :, _kv_heads(c, 1)]


def _quantised_bounds(lo, hi):
    """Per-page bounds in 8 bits: lo rounded down, hi rounded up, in steps of the largest magnitude / 127."""
    a = torch.maximum(lo.abs(), hi.abs()).amax(-1)
    s = a / 127.0
    safe = torch.where(s > 0, s, torch.ones_like(s))[..., None]
    hi8 = torch.ceil(hi / safe).clamp(-127, 127)
    lo8 = torch.floor(lo / safe).clamp(-127, 127)
    q = torch.stack([lo8, hi8], -2) * (s > 0)[..., None, None]
    return q.to(torch.int8), s


def _bounds(k, valid=None):
    """k [n, page, heads, 128] in 32 bits -> (bounds [n, heads, 2, 128] int8, scale [n, heads])."""
    lo = hi = k
    if valid is not None:
        lo, hi = k.masked_fill(~valid, float("inf")), k.masked_fill(~valid, float("-inf"))
    return _quantised_bounds(lo.amin(1), hi.amax(1))


def _all_bounds(pages, c):
    lo, hi = (_retrieval(p, c) for p in (pages, pages))
    if c["kv"] == "bf16":
        return _quantised_bounds(lo.amin(1).float(), hi.amax(1).float())
    return _bounds(lo.float())


def _plan(s):
    ps, B = s["page"], s["c"]["B"]
    old, new, free = s["seq_lens"].long(), s["n_new"].long(), s["free_count"].long()
    width = s["table"].shape[1]
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(new, 0)])
    have = (old + ps - 1) // ps
    want = (old + new + ps - 1) // ps
    fits = (want <= width) & (cu[1:] <= s["max_tokens"])
    need = torch.where(fits, want - have, torch.zeros_like(want))
    upto = torch.cumsum(need, 0)
    ok = fits & ((need == 0) | (upto <= free))
    take = torch.where(ok, need, torch.zeros_like(need))
    off = upto - need  # a request that is refused leaves no gap: all that need pages behind it are refused too
    col = torch.arange(width, device=DEV)[None, :]
    fresh = (col >= have[:, None]) & (col < (have + take)[:, None])
    popped = (free - 1 - off)[:, None] - (col - have[:, None])
    table = s["table"]
    table[fresh] = s["free_pages"][popped[fresh]]
    after = old + torch.where(ok, new, torch.zeros_like(new))
    t = torch.arange(s["max_tokens"], device=DEV)
    row = torch.searchsorted(cu[1:], t, right=True)
    live = row < B
    row = row.clamp(max=B - 1)
    pos = t - cu[row] + old[row]
    live &= ok[row]
    page = table[row, (pos // ps).clamp(0, width - 1)].long()
    slot = torch.where(live, page * ps + pos % ps, torch.full_like(pos, -1))
    first = old // ps
    n_span = torch.where(ok & (new > 0), want - first, torch.zeros_like(want))
    ends = torch.cumsum(n_span, 0)
    i = torch.arange(_spans_cap(s["max_tokens"], B, ps), device=DEV)
    b = torch.searchsorted(ends, i, right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    p = first[b] + i - (ends - n_span)[b]
    rows = torch.clamp(after[b] - p * ps, max=ps)
    had = torch.clamp(old[b] - p * ps, min=0)
    spans = torch.stack([table[b, p.clamp(0, width - 1)].long(), rows, had, cu[b] + p * ps + had - old[b]], 1)
    spans = torch.where(live[:, None], spans, torch.tensor([-1, 0, 0, 0], device=DEV))
    i32 = torch.int32
    return dict(seq_lens=after.to(i32), cu_new=cu.to(i32), slot_map=slot.to(i32), spans=spans.to(i32),
                free_count=(free - take.sum()).to(i32), admitted=ok.to(i32), block_table=table)


def _write(s):
    c, ps = s["c"], s["page"]
    slot = s["slot_map"].long()
    for pages, x, scale in ((s["k_pages"], s["k"], s["k_scale"]), (s["v_pages"], s["v"], s["v_scale"])):
        pages[slot // ps, slot % ps] = _stored(x, c["kv"], scale)
    return [s["k_pages"], s["v_pages"]]


def _append(s):
    c = s["c"]
    _write(s)
    spans = s["spans"][s["spans"][:, 0] >= 0].long()
    k = _retrieval(s["k_pages"], c)[spans[:, 0]].float()
    valid = torch.arange(s["page"], device=DEV)[None, :] < spans[:, 1:2]
    q, scale = _bounds(k, valid[:, :, None, None])
    s["bounds"][spans[:, 0]] = q
    s["bound_scale"][spans[:, 0]] = scale
    return [s["k_pages"], s["v_pages"], s["bounds"], s["bound_scale"]]


def _attend(q, k, v, keep, scale):
    """q [B, g, G, 128], k / v [B, n, g, 128], keep [B, n] or [B, n, g]: (o, lse), zeros and -inf where nothing is kept."""
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * scale
    keep = (keep[:, :, None] if keep.dim() == 2 else keep).permute(0, 2, 1)[:, :, None, :]
    x = x.masked_fill(~keep, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p / torch.where(z > 0, z, torch.ones_like(z)), v.permute(0, 2, 1, 3))
    return o, (m + torch.log(z)).squeeze(-1)


def _rows(pages, table, pos, heads, scale, ps):
    """The stored rows of positions pos [B, n] (or [B, n, heads]) as 32-bit values [B, n, heads, 128]."""
    at = table.long().clamp(min=0)
    if pos.dim() == 2:
        page = torch.gather(at, 1, pos // ps)[:, :, None]
        pos = pos[:, :, None]
    else:
        page = torch.gather(at, 1, (pos // ps).flatten(1)).view(pos.shape)
    x = pages[page, pos % ps, heads].float()
    return x if scale is None else x * scale[heads][:, None]


def _attention(s, sel=None, count=None):
    c, ps, table = s["c"], s["page"], s["table"]
    B, H, Hkv = c["B"], c["H"], c["Hkv"]
    G, lens = H // Hkv, s["seq_lens"].long()
    q = s["q"].view(B, Hkv, G, D).float()
    o = torch.zeros((B, Hkv, G, D), device=DEV)
    lse = torch.full((B, Hkv, G), float("-inf"), device=DEV)
    scale = D ** -0.5
    ret, loc = _kv_heads(c, 1), _kv_heads(c, 0)
    if len(ret):
        if sel is None:
            pos = torch.arange(table.shape[1] * ps, device=DEV).expand(B, -1)
            keep = pos < lens[:, None]
        else:
            page = sel.long().clamp(min=0)[..., None] * ps + torch.arange(ps, device=DEV)
            live = (torch.arange(sel.shape[2], device=DEV) < count.long()[..., None])[..., None]
            keep = (live & (page < lens[:, None, None, None])).flatten(2).permute(0, 2, 1)
            pos = page.flatten(2).permute(0, 2, 1)
        k = _rows(s["k_pages"], table, pos, ret, s["k_scale"], ps)
        v = _rows(s["v_pages"], table, pos, ret, s["v_scale"], ps)
        o[:, ret], lse[:, ret] = _attend(q[:, ret], k, v, keep, scale)
    if len(loc):
        w, n_sink = c["window"], c["n_sink"]
        low = lens[:, None] - w
        pos = torch.cat([torch.arange(n_sink, device=DEV).expand(B, -1), low + torch.arange(w, device=DEV)], 1)
        sink = torch.arange(n_sink + w, device=DEV)[None, :] < n_sink
        keep = (pos >= 0) & (pos < lens[:, None]) & (sink | (pos >= n_sink))
        pos = pos.clamp(min=0).clamp(max=table.shape[1] * ps - 1)
        k = _rows(s["k_pages"], table, pos, loc, s["k_scale"], ps)
        v = _rows(s["v_pages"], table, pos, loc, s["v_scale"], ps)
        o[:, loc], lse[:, loc] = _attend(q[:, loc], k, v, keep, scale)
    return o.view(B, 1, H, D).to(torch.bfloat16), lse.view(B, H, 1)


#: pages that a selection always keeps: the first (attention sinks) and the last (the newest tokens)
FIRST, RECENT = 1, 1


def _select(s):
    c, ps, lens = s["c"], s["page"], s["seq_lens"].long()
    B, G, ret = c["B"], c["H"] // c["Hkv"], _kv_heads(c, 1)
    n_sel, table = c["n_sel"], s["table"].long().clamp(min=0)
    q = s["q"].view(B, c["Hkv"], G, D)[:, ret].float()
    sq = q.abs().amax(-1) / 127.0
    q8 = torch.round(q / torch.where(sq > 0, sq, torch.ones_like(sq))[..., None]) * (sq > 0)[..., None]
    both = torch.cat([q8.clamp(max=0.0), q8.clamp(min=0.0)], -1)  # against lo, against hi
    b8 = s["bounds"][table].flatten(3).permute(0, 2, 3, 1).float()
    dot = torch.matmul(both, b8)  # whole numbers under 2^24: exact
    sp = s["bound_scale"][table].permute(0, 2, 1)
    score = (dot * (sq[..., None] * sp[:, :, None, :])).amax(2)
    n = ((lens + ps - 1) // ps)[:, None, None]
    p = torch.arange(table.shape[1], device=DEV)
    score = score.masked_fill((p < FIRST) | (p >= n - RECENT), float("inf")).masked_fill(p >= n, float("-inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n_sel]
    count = torch.clamp(n[..., 0], max=n_sel).expand(B, len(ret))
    live = torch.arange(order.shape[-1], device=DEV) < count[..., None]
    last = table.shape[1]
    order = torch.sort(order.masked_fill(~live, last), dim=-1).values
    sel = torch.full((B, len(ret), n_sel), -1, dtype=torch.int32, device=DEV)
    sel[..., :order.shape[-1]] = order.masked_fill(order == last, -1).to(torch.int32)
    return sel, count.to(torch.int32)


# -------------------------------------------------------------------------------------------- run
def run(state):
    s = state
    c, op = s["c"], s["c"]["op"]
    if own:
        return _own(s)
    if op == "plan":
        return _plan(s)
    if op == "write":
        return _write(s)
    if op == "append":
        return _append(s)
    if op == "attn":
        return list(_attention(s))
    sel, count = _select(s)
    o, lse = _attention(s, sel, count)
    return [o, lse, sel, count]


def _own(s):
    import long_context_sparse_rtp_b200 as rtp
    c, op = s["c"], s["c"]["op"]
    if op == "plan":
        out = rtp.rtp_paged_plan(s["seq_lens"], s["n_new"], s["table"], s["free_pages"], s["free_count"],
                                 page_size=s["page"], max_tokens=s["max_tokens"])
        return dict(out, block_table=s["table"])
    if op == "write":
        rtp.rtp_paged_kv_write(s["k"], s["v"], s["slot_map"], s["k_pages"], s["v_pages"],
                               k_scale=s["k_scale"], v_scale=s["v_scale"])
        return [s["k_pages"], s["v_pages"]]
    if op == "append":
        rtp.rtp_paged_kv_append(s["k"], s["v"], s["spans"], s["k_pages"], s["v_pages"], _roles(c),
                                s["bounds"], s["bound_scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return [s["k_pages"], s["v_pages"], s["bounds"], s["bound_scale"]]
    local = dict(window=c["window"], n_sink=c["n_sink"]) if "0" in c["roles"] else {}
    if op == "attn":
        return list(rtp.rtp_paged_attn_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seq_lens"],
                                              _roles(c), k_scale=s["k_scale"], v_scale=s["v_scale"], **local))
    sel, count = rtp.rtp_paged_block_select(s["q"], s["bounds"], s["bound_scale"], s["table"], s["seq_lens"],
                                            _roles(c), page_size=s["page"], n_sel=c["n_sel"], n_first=FIRST,
                                            n_recent=RECENT)
    o, lse = rtp.rtp_paged_attn_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seq_lens"], _roles(c),
                                       sel=sel, sel_count=count, k_scale=s["k_scale"], v_scale=s["v_scale"],
                                       **local)
    return [o, lse, sel, count]


# ------------------------------------------------------------------------------------------- work
def _row_bytes(c):
    return D * (2 if c["kv"] == "bf16" else 1)


def work(case):
    c = dict(case)
    lens, ps, B = _lens(c), c["page"], c["B"]
    if c["op"] == "plan":
        news = _news(c)
        pages = sum(_up(n + m, ps) - _up(n, ps) for n, m in zip(lens, news))
        spans = sum(_up(n + m, ps) - n // ps for n, m in zip(lens, news) if m)
        return {"bytes": 4 * 2 * B + 8 * pages + 4 * sum(news) + 16 * spans + 12 * B, "flops": 0}
    if c["op"] in ("write", "append"):
        news = _news(c)
        T = sum(news)
        total = T * (4 + 2 * c["Hkv"] * (2 * D + _row_bytes(c)))
        if c["op"] == "append":
            n_ret = c["roles"].count("1")
            spans = sum(_up(n + m, ps) - n // ps for n, m in zip(lens, news))
            total += 16 * spans - 4 * T + n_ret * (spans * (2 * D + 4) + sum(n % ps for n in lens) * _row_bytes(c))
        return {"bytes": total, "flops": 0}
    n_ret = c["roles"].count("1")
    n_loc, G = c["Hkv"] - n_ret, c["H"] // c["Hkv"]
    local = [min(n, c["window"]) + min(c["n_sink"], max(0, n - c["window"])) for n in lens]
    full, score = lens, 0
    if c["op"] == "sparse":
        pages = [_up(n, ps) for n in lens]
        score = n_ret * sum(pages)
        full = [n if p <= c["n_sel"] else (c["n_sel"] - 1) * ps + n - (p - 1) * ps for n, p in zip(lens, pages)]
    keys = n_ret * sum(full) + n_loc * sum(local)
    return {"bytes": keys * 2 * _row_bytes(c) + score * (2 * D + 4) + B * c["H"] * (4 * D + 4)
            + 4 * B + 4 * sum(_up(n, ps) for n in lens),
            "flops": keys * G * 4 * D + score * G * 4 * D}


# ------------------------------------------------------------------------------------------ exact
def _e4m3_64(x):
    """The nearest e4m3 value of x in 64 bits, ties to even, the largest at 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    step = torch.pow(torch.full_like(e, 2.0), e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    c, ps = s["c"], s["page"]
    if c["op"] == "plan":
        return None  # whole numbers only
    if c["op"] in ("write", "append"):
        out = []
        for name in ("k", "v"):
            pages = s[name + "_pages"].double()
            x = s[name].double()
            if c["kv"] == "e4m3":
                x = _e4m3_64(x / s[name + "_scale"].double()[:, None])
            flat = pages.view(-1, c["Hkv"], D)
            flat.index_copy_(0, s["slot_map"].long(), x)
            out.append(pages)
        if c["op"] == "write":
            return out
        scale = s["bound_scale"].double()
        heads = [g for g, r in enumerate(_roles(c)) if r]
        live = s["spans"][s["spans"][:, 0] >= 0]
        for at in range(0, ps):  # pages by how many rows they hold
            pick = live[live[:, 1] == at + 1, 0].long()
            if len(pick) and heads:
                scale[pick] = out[0][pick, :at + 1][:, :, heads].abs().amax(dim=(1, 3)) / 127.0
        return out + [None, scale]
    H, Hkv = c["H"], c["Hkv"]
    G, o, lse = H // Hkv, [], []
    chosen = [None, None]
    if c["op"] == "sparse":
        # the selection is a rule on whole numbers and their 32-bit scales: the keys follow it
        chosen = _select(s)
    for b, n in enumerate(_lens(c)):
        ob, lb = [], []
        for g, role in enumerate(_roles(c)):
            pos = torch.arange(n, device=DEV)
            if not role:
                pos = pos[(pos < c["n_sink"]) | (pos >= n - c["window"])]
            elif c["op"] == "sparse":
                r = sum(_roles(c)[:g])
                mine = torch.isin(pos // ps, chosen[0][b, r, :int(chosen[1][b, r])].long())
                pos = pos[mine]
            if not len(pos):
                ob.append(torch.zeros(G, D, dtype=torch.float64, device=DEV))
                lb.append(torch.full((G,), float("-inf"), dtype=torch.float64, device=DEV))
                continue
            page = s["table"][b].long()[pos // ps]
            k, v = s["k_pages"][page, pos % ps, g].double(), s["v_pages"][page, pos % ps, g].double()
            if c["kv"] == "e4m3":
                k, v = k * s["k_scale"][g].double(), v * s["v_scale"][g].double()
            x = s["q"][b, 0, g * G:(g + 1) * G].double() @ k.T / D ** 0.5
            lb.append(torch.logsumexp(x, -1))
            ob.append(torch.softmax(x, -1) @ v)
        o.append(torch.cat(ob))
        lse.append(torch.cat(lb))
    out = [torch.stack(o)[:, None], torch.stack(lse)[..., None]]
    return out + [None, None] if c["op"] == "sparse" else out


if __name__ == "__main__":
    for case in listed() + [dict(draw(random.Random(i)), name="drawn") for i in range(4)]:
        w = work(case)
        print("%-22s %10.3f MB %10.3f GFLOP" % (case["name"], w["bytes"] / 1e6, w["flops"] / 1e9))
