"""Plain implementations of the paged-cache operators, for the tests: whole
numbers as they are, values in 64 bits, one request at a time."""
import numpy as np
import torch

D = 128


def up(a, b):
    return -(-a // b)


def plan(seq_lens, n_new, table, free_pages, free_count, *, page_size, max_tokens, n_spans,
         row_tokens=0, release=None):
    """rtp_paged_plan on numpy copies; returns the dict plus block_table and free_pages."""
    ps, B, width = page_size, len(seq_lens), table.shape[1]
    table, stack = table.copy(), list(free_pages[:free_count])
    cap = len(free_pages)
    lens = [max(0, int(x)) for x in seq_lens]
    for b in range(B):
        if release is not None and release[b]:
            for p in table[b, :min(width, up(lens[b], ps))]:
                if len(stack) < cap:
                    stack.append(int(p))
            lens[b] = 0
    pool = np.array(free_pages)
    pool[:len(stack)] = stack
    top, asked, taken = len(stack), 0, 0
    cu, slots, spans, admitted, after = [0], np.full(max_tokens, -1), [], [], []
    for b in range(B):
        n, old = max(0, int(n_new[b])), lens[b]
        start = b * row_tokens if row_tokens else cu[-1]
        cu.append((b + 1) * row_tokens if row_tokens else cu[-1] + n)
        want, have = up(old + n, ps), up(old, ps)
        ok = want <= width and start + n <= max_tokens and not (row_tokens and n > row_tokens)
        need = want - have if ok else 0
        asked += need
        ok = ok and (need == 0 or asked <= top)
        admitted.append(int(ok))
        after.append(old + (n if ok else 0))
        if not ok:
            continue
        for j in range(need):
            table[b, have + j] = stack[top - 1 - (asked - need) - j]
        taken += need
        for i in range(n):
            x = old + i
            slots[start + i] = table[b, x // ps] * ps + x % ps
        if n:
            for c in range(old // ps, want):
                fresh = max(0, old - c * ps)
                spans.append([table[b, c], min(ps, old + n - c * ps), fresh,
                              start + c * ps + fresh - old])
    spans = (spans + [[-1, 0, 0, 0]] * n_spans)[:n_spans]
    return dict(seq_lens=np.array(after), cu_new=np.minimum(cu, 2 ** 31 - 1),  # int32, saturating
                 slot_map=slots,
                spans=np.array(spans).reshape(n_spans, 4), free_count=np.array([top - taken]),
                admitted=np.array(admitted), block_table=table, free_pages=pool)


def e4m3(x):
    """The nearest e4m3 value of x (fp64), ties to even, saturating."""
    x = np.asarray(x, dtype=np.float64)
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -20))), -6)
    step = 2.0 ** (e - 3)
    return np.clip(np.rint(x / step) * step, -448, 448)


def bounds(rows):
    """rows [n, 128] of one page and head (stored values) -> (lo8, hi8, scale) in fp32 steps."""
    f = np.float32
    r = np.asarray(rows, dtype=f)
    zero = np.zeros(D, dtype=np.int64)
    if not np.isfinite(r).all():
        return zero, zero, f(np.inf)
    lo, hi = r.min(0), r.max(0)
    s = np.maximum(np.abs(lo), np.abs(hi)).max() * (f(1) / f(127))
    if not s > 0:
        return zero, zero, f(0)
    return (np.maximum(np.floor(lo / s), -127).astype(np.int64),
            np.minimum(np.ceil(hi / s), 127).astype(np.int64), s)


def select(q, lo8, hi8, scale, n_sel, n_first, n_recent):
    """q [G, 128], bounds [nb, 128] and scale [nb] of a row's pages (scale < 0: no such
    page) -> ascending page indices.  The first n_first and the last n_recent pages come
    before every other, whatever they or the others score."""
    f = np.float32
    nb = len(scale)
    if nb <= n_sel:
        return list(range(nb))
    best = np.full(nb, -np.inf, dtype=f)
    for x in np.asarray(q, dtype=f):
        s = np.abs(x).max() * (f(1) / f(127)) if np.isfinite(x).all() else f(0)
        q8 = np.rint(x / s).astype(np.int64) if s > 0 else np.zeros(D, dtype=np.int64)
        I = np.maximum(q8 * lo8, q8 * hi8).sum(1)
        with np.errstate(over="ignore"):
            t = np.minimum(s * np.where(np.isfinite(scale), scale, f(1)).astype(f),
                           np.finfo(f).max)
            best = np.maximum(best, I.astype(f) * t)
    best[scale == np.inf] = np.inf
    best[scale < 0] = -np.inf
    order = sorted(range(nb), key=lambda p: (n_first <= p < nb - n_recent, -best[p], p))
    return sorted(order[:n_sel])


def keys_of(length, role, page_size, window=None, n_sink=0, pages=None):
    """The positions a head attends to."""
    if role == 0:
        return [j for j in range(length) if j < n_sink or j >= length - window]
    if pages is None:
        return list(range(length))
    return [j for p in pages for j in range(p * page_size, min(length, (p + 1) * page_size))]


def attend(q, k, v, scale):
    """q [G, 128], k, v [n, 128] in 64 bits -> (o, lse, sum p |v|, largest sum |q k|)."""
    q, k, v = (x.double() for x in (q, k, v))
    if k.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, torch.full((q.shape[0],), float("-inf"), dtype=torch.float64), z, 0.0
    x = q @ k.T * scale
    p = torch.softmax(x, -1)
    return p @ v, torch.logsumexp(x, -1), p @ v.abs(), float((q.abs() @ k.abs().T).max())
