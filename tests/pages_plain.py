"""Plain implementations of the page bookkeeping, of moved pages and rows, and of the
check of drafted tokens: one sequence after the other on the CPU, in whole numbers."""
import numpy as np


def up(n, ps):
    return -(-n // ps)


def reserve(refs, table, kv_len, new_len, ps):
    """Returns (refs, table, got_len, copy_src, copy_dst, bad); inputs are left alone.
    ``bad``: whether a length or an id was out of range."""
    refs, table = list(map(int, refs)), [list(map(int, r)) for r in table]
    held, free = list(refs), [p for p, r in enumerate(refs) if r == 0]
    old = list(refs)
    at, full, bad = 0, False, False
    got, src, dst = [], [], []
    for s, (a, b) in enumerate(zip(map(int, kv_len), map(int, new_len))):
        ok = 0 <= a <= b <= len(table[s]) * ps
        page = -1
        if ok and b > a and a % ps:
            page = table[s][a // ps]
            ok = 0 <= page < len(refs)
        if not ok:
            bad = True
            got.append(a), src.append(-1), dst.append(-1)
            continue
        shared = page >= 0 and old[page] > 1
        cow = shared and held[page] > 1
        held[page] -= cow
        need = up(b, ps) - up(a, ps) + cow
        full = full or (need > 0 and at + need > len(free))
        if full and (need > 0 or shared):
            got.append(a), src.append(-1), dst.append(-1)
            continue
        pages = free[at:at + need]
        at += need
        for p in pages:
            refs[p] = 1
        got.append(b), src.append(page if cow else -1), dst.append(pages[0] if cow else -1)
        if cow:
            refs[page] -= 1
            table[s][a // ps] = pages[0]
        table[s][up(a, ps):up(b, ps)] = pages[cow:]
    return refs, table, got, src, dst, bad


def fork(refs, table, kv_len, new_len, ps, parent=None, out=None):
    """Returns (refs, out_table); ``out`` is what out_table held before."""
    refs, table = list(map(int, refs)), [list(map(int, r)) for r in table]
    for row, a in zip(table, kv_len):
        for p in row[:up(int(a), ps)]:
            refs[p] -= 1
    out = table if parent is None else [list(map(int, r)) for r in out]
    for d, b in enumerate(map(int, new_len)):
        n = up(b, ps)
        if parent is not None and n:
            out[d][:n] = table[int(parent[d])][:n]
        for p in out[d][:n]:
            refs[p] += 1
    return refs, out


def copy_pages(x, src, dst):
    """x [n_pages, ...] after the copies; an entry with -1, or of a page onto itself, is none."""
    y = x.copy()
    for a, b in zip(src, dst):
        if a >= 0 and b >= 0 and a != b:
            y[b] = x[a]
    return y


def compact(x, keep, cu, table, ps, start=None, out_table=None):
    """x [n_pages, Hkv, ps, ...] after the rows moved, from a copy."""
    y = x.copy()
    out = table if out_table is None else out_table
    for s in range(len(cu) - 1):
        to = (0 if start is None else start[s]) + np.arange(cu[s + 1] - cu[s])
        for h in range(x.shape[1]):
            k = np.asarray((keep[h] if np.ndim(keep) == 2 else keep)[cu[s]:cu[s + 1]], dtype=int)
            y[np.asarray(out[s])[to // ps], h, to % ps] = x[np.asarray(table[s])[k // ps], h, k % ps]
    return y


def units(p):
    """Probabilities as whole multiples of 2^-60, the nearest; what is outside [0, 2) as 0."""
    p = np.asarray(p, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        p = np.where((p >= 0) & (p < 2), p, 0.0)
    return np.rint(np.ldexp(p, 60)).astype(np.int64)


def draw(w, u):
    """Smallest t with w_0 + .. + w_t > u * sum(w), in whole numbers; the last token for zeros."""
    w = w.astype(np.uint64)
    total = int(w.sum(dtype=np.uint64))
    if total == 0:
        return len(w) - 1
    num, den = float(u).as_integer_ratio()
    return int(np.searchsorted(np.cumsum(w, dtype=np.uint64), np.uint64(num * total // den), "right"))


def verify(target, drafted, cu, max_draft, u_accept, u_sample, draft=None):
    """target [total + n_seq, V], draft [total, V] float64; returns (tokens, n_accepted)."""
    n_seq, V = len(cu) - 1, target.shape[1]
    tokens = np.full((n_seq, max_draft + 1), -1, dtype=np.int32)
    accepted = np.zeros(n_seq, dtype=np.int32)
    for s in range(n_seq):
        n, w = cu[s + 1] - cu[s], None
        for i in range(n):
            d, x = cu[s] + i, int(drafted[cu[s] + i])
            known = 0 <= x < V
            q = 1.0 if draft is None else draft[d][x] if known else 0.0
            # (Both factors have at most 24 bits: the product is exact in 64.)
            if known and float(u_accept[d]) * q < target[d + s][x]:
                tokens[s, i] = x
                accepted[s] += 1
                continue
            p = units(target[d + s])
            if draft is None:
                w = p.copy()
                if known:
                    w[x] = 0
            else:
                w = np.maximum(p - units(draft[d]), 0)
            if not w.any():
                w = p
            break
        if w is None:
            w = units(target[cu[s + 1] + s])
        tokens[s, accepted[s]] = draw(w, min(max(float(u_sample[s]), 0.0), 1 - 2.0 ** -24))
    return tokens, accepted
