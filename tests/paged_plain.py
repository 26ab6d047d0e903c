"""Plain 64-bit paged-cache operators (numpy, on the CPU): the row formats from
their definitions, and the attention of a chunk of new tokens with the block
loop written out."""
import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_table():
    c = np.arange(256)
    ex, f = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(ex == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (ex - 7.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


E4M3 = _e4m3_table()
_POS = E4M3[:127]  # codes 0 .. 0x7e, ascending


def nearest_even(x, grid):
    """Index into the ascending ``grid`` of the value nearest to x >= 0, ties to
    the even index, values past the end to the last."""
    i = np.clip(np.searchsorted(grid, x, side="right") - 1, 0, len(grid) - 2)
    lo, hi = grid[i], grid[i + 1]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (i % 2 == 1))
    return i + up


def row_scale(x, top):
    """(byte, 2^e, bad) per row of x [..., 128] (float64)."""
    bad = ~np.isfinite(x).all(-1)
    a = np.where(bad[..., None], 0.0, np.abs(x)).max(-1)
    frac, ex = np.frexp(a / top)  # exact: top is 7/4 or 21/16 times a power of two ...
    e = np.where(frac == 0.5, ex - 1, ex)
    # ... but the quotient may have rounded: settle it by exact products.
    e = np.where(a > top * np.exp2(e.astype(float)), e + 1, e)
    e = np.where(a <= top * np.exp2(e - 1.0), e - 1, e)
    e = np.where(a > 0, np.clip(e, -110, 120), 0)
    return np.where(bad, 255, e + 127).astype(np.uint8), np.exp2(e.astype(float)), bad


def encode(fmt, x):
    """Rows x [..., 128] (float64) as dict(codes, scale, bs)."""
    if fmt == "e4m3":
        byte, s, bad = row_scale(x, 448.0)
        y = np.where(bad[..., None], 0.0, x) / s[..., None]
        c = nearest_even(np.abs(y), _POS).astype(np.uint8) | (np.signbit(y).astype(np.uint8) << 7)
        return dict(codes=np.where(bad[..., None], 0, c).astype(np.uint8), scale=byte)
    byte, s, bad = row_scale(x, 2688.0)
    y = (np.where(bad[..., None], 0.0, x) / s[..., None]).reshape(*x.shape[:-1], 8, 16)
    top = np.abs(y).max(-1)
    bs = np.searchsorted(6 * _POS, top, side="left")  # the first with 6 b >= top
    b = _POS[bs][..., None]
    # Nearest to y / b: compare y with b times the values (products exact).
    c = np.zeros(y.shape, dtype=np.uint8)
    a = np.abs(y)
    for k in range(7):
        mid = (E2M1[k] + E2M1[k + 1]) / 2 * b
        c += ((a >= mid) if k % 2 else (a > mid)).astype(np.uint8)
    c = np.where(b > 0, c, 0).astype(np.uint8) | (np.signbit(y).astype(np.uint8) << 3)
    c = np.where(bad[..., None, None], 0, c).reshape(x.shape)
    bs = np.where(bad[..., None], 0, bs).astype(np.uint8)
    return dict(codes=(c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8), scale=byte, bs=bs)


def decode(fmt, codes, scale, bs=None):
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(float) - 127))[..., None]
    if fmt == "e4m3":
        return E4M3[codes] * s
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 128)
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    return v * np.repeat(E4M3[bs], 16, -1) * s


def attend(q, k, v, n, kv, G, lam, causal, scale, bps, force=None):
    """One sequence: q [n, Hkv, G, 128], k and v [kv, Hkv, 128], float64.

    Returns dict(o, lse, absv, dots, skip, margin): o [n, Hkv, G, 128], lse [n,
    Hkv, G], absv = sum of p |v| (the scale of rounding errors in o), dots =
    scale * the largest sum |q_d k_d| of a visible key, skip / margin [Hkv, n_t,
    n_splits, bps] (NaN margin: not traversed).  ``force`` takes the skip
    decisions instead of the rule."""
    Hkv, tt = q.shape[1], 128 // G
    n_t, n_splits = -(-n // tt), force.shape[2] if force is not None else None
    nb_all = -(-kv // 128)
    n_splits = n_splits or max(1, -(-nb_all // max(bps, 1)))
    ln_lam = math.log(lam) if lam > 0 else -math.inf
    out = dict(o=np.zeros((n, Hkv, G, 128)), lse=np.full((n, Hkv, G), -math.inf),
               absv=np.zeros((n, Hkv, G, 128)), dots=np.zeros((n, Hkv, G)),
               skip=np.zeros((Hkv, n_t, n_splits, max(bps, 1)), dtype=bool),
               margin=np.full((Hkv, n_t, n_splits, max(bps, 1)), np.nan))
    for h in range(Hkv):
        for t in range(n_t):
            i0, i1 = t * tt, min(n, (t + 1) * tt)
            pos = kv - n + np.arange(i0, i1)
            limit = np.maximum(pos + 1, 0) if causal else np.full(i1 - i0, kv)
            blocks = -(-int(limit.max()) // 128)
            qt = q[i0:i1, h].reshape(-1, 128)  # rows (token, head)
            lim = np.repeat(limit, G)
            s = scale * (qt @ k[:, h].T)
            seen = np.arange(kv)[None, :] < lim[:, None]
            s = np.where(seen, s, -math.inf)
            dots = scale * (np.abs(qt) @ np.abs(k[:, h]).T)
            kept = np.zeros_like(seen)
            for sp in range(n_splits):
                m = np.full(len(qt), -math.inf)
                for p in range(bps):
                    j = sp * bps + p
                    if j >= blocks:
                        break
                    cols = slice(j * 128, min(kv, (j + 1) * 128))
                    top = s[:, cols].max(-1)
                    m = np.maximum(m, top)
                    with np.errstate(invalid="ignore"):
                        d = np.where(top == -math.inf, -math.inf, top - m)
                    out["margin"][h, t, sp, p] = d.max()
                    skip = bool((d < ln_lam).all() or (top == -math.inf).all())
                    if force is not None:
                        skip = bool(force[h, t, sp, p])
                    out["skip"][h, t, sp, p] = skip
                    if not skip:
                        kept[:, cols] = seen[:, cols]
            x = np.where(kept, s, -math.inf)
            top = x.max(-1) if kv else np.full(len(qt), -math.inf)
            ref = np.where(np.isfinite(top), top, 0.0)
            e = np.exp(x - ref[:, None])
            l = e.sum(-1)
            with np.errstate(divide="ignore", invalid="ignore"):
                p = np.where(l[:, None] > 0, e / l[:, None], 0.0)
                lse = ref + np.log(l)
            vh = v[:, h]
            shape = (i1 - i0, G, 128)
            out["o"][i0:i1, h] = (p @ vh).reshape(shape)
            out["absv"][i0:i1, h] = (p @ np.abs(vh)).reshape(shape)
            out["lse"][i0:i1, h] = lse.reshape(shape[:2])
            out["dots"][i0:i1, h] = np.where(seen, dots, 0.0).max(-1, initial=0.0).reshape(shape[:2])
    return out
