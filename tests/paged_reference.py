"""The paged-cache operators restated in 64 bits with numpy, one element at a time in
meaning and without the package, for the tests: e4m3 codes, rotation, append, attention
with score rules, and the error bounds the tests hold the kernels to."""
import math

import numpy as np

E4M3_MAX = 448.0


def e4m3_values():
    """float64 [256]: the value of every code (NaN at 0x7F and 0xFF)."""
    out = np.empty(256)
    for c in range(256):
        sign = -1.0 if c & 0x80 else 1.0
        e, m = (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            out[c] = math.nan
        elif e == 0:
            out[c] = sign * m * 2.0 ** -9
        else:
            out[c] = sign * (1 + m / 8) * 2.0 ** (e - 7)
    return out


VALUES = e4m3_values()


def to_e4m3(x):
    """Codes (uint8) nearest to x, ties to the even code, at most 448 in magnitude, NaN to 0x7F."""
    x = np.asarray(x, np.float64)
    mag = np.minimum(np.abs(x), E4M3_MAX)
    grid = VALUES[:127]                                   # 0 .. 448 ascending
    hi = np.clip(np.searchsorted(grid, mag, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = mag - grid[lo], grid[hi] - mag
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    pick = pick | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), pick).astype(np.uint8)


def scale_for(amax):
    """Smallest power of two s in 2^-60 .. 2^60 with amax <= 448 s."""
    s = 2.0 ** -60
    while amax > E4M3_MAX * s and s < 2.0 ** 60:
        s *= 2
    return s


def rotate(x, pos, freq, interleaved, mscale=1.0):
    """x [tokens, heads, hd] rotated by pos [tokens]; freq [rot / 2] radians per position."""
    x = np.array(x, np.float64)
    r = len(freq)
    ang = np.asarray(pos, np.float64)[:, None] * freq
    c, s = np.cos(ang)[:, None] * mscale, np.sin(ang)[:, None] * mscale
    if interleaved:
        a, b = x[..., 0:2 * r:2].copy(), x[..., 1:2 * r:2].copy()
        x[..., 0:2 * r:2], x[..., 1:2 * r:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :r].copy(), x[..., r:2 * r].copy()
        x[..., :r], x[..., r:2 * r] = a * c - b * s, b * c + a * s
    return x


def frequencies(rot, base, scaling=0, factor=1.0, low=0.0, high=0.0, trained=0):
    if scaling == 2:
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == 1:
        f = f / factor
    if scaling == 3:
        keep = np.clip((trained * f / (2 * math.pi) - low) / (high - low), 0, 1)
        f = keep * f + (1 - keep) * f / factor
    return f


def append(pool, scale, rows, table, positions, counts):
    """Write rows [tokens, n_kv, hd] (float64, in sequence order) into pool [n_pages, page, n_kv, hd]:
    float64 values for a 16-bit cache (scale None), codes with scale [n_pages, n_kv] for e4m3.
    Returns the mask of the elements written or rescaled [n_pages, page]."""
    page = pool.shape[1]
    cap = table.shape[1] * page
    touched = np.zeros(pool.shape[:2], bool)
    at = 0
    for s, n in enumerate(counts):
        first = int(positions[s]) + 1 - n
        by_page = {}
        for i in range(n):
            j = first + i
            if 0 <= j < cap:
                by_page.setdefault(j // page, []).append((j % page, at + i))
        at += n
        for p, items in by_page.items():
            pid = int(table[s, p])
            if not 0 <= pid < pool.shape[0]:
                continue
            offs, toks = [o for o, _ in items], [t for _, t in items]
            touched[pid, offs] = True
            if scale is None:
                pool[pid, offs] = rows[toks]
                continue
            for h in range(pool.shape[2]):
                x = rows[toks, h]
                fin = np.abs(x[np.isfinite(x)])
                new = scale_for(fin.max() if fin.size else 0.0)
                if offs[0] > 0:
                    old = float(scale[pid, h])
                    new = max(new, old)
                    if new > old:
                        pool[pid, :offs[0], h] = to_e4m3(VALUES[pool[pid, :offs[0], h]] * (old / new))
                        touched[pid, :offs[0]] = True
                scale[pid, h] = new
                pool[pid, offs, h] = to_e4m3(x / new)
    return touched


def attend(q, k_rows, v_rows, positions, scale, softcap=0.0, slopes=None, window=0, starts=None,
           eps_pair=2.0 ** -22):
    """q [n_seq, n_q, n_head, hd]; k_rows, v_rows: per sequence float64 [nkv, n_kv, hd] with NaN
    rows where a page is not there (never seen). Returns (out, bound): the result and how far
    the kernel's may be off, element by element.

    The bound: a score is a sum of hd products of q (carried to eps_pair) and exact cache values in
    32-bit accumulation, hd / 16 steps of 16 products each rounded to 2^-23 of at most the sum of
    magnitudes A; then a few 32-bit roundings of the score itself (2^-22 of it, for rows that
    weigh), and 2^-22 of the cap. An error d of every score moves each weight by at most
    e^2d - 1 of itself, and a weighted mean by that times the largest |v|; the weights' own
    rounding (eps_pair, and 2^-21 for the exponential) and the sums' (2^-20, tiles and splits)
    count likewise."""
    n_seq, n_q, n_head, hd = q.shape
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for s in range(n_seq):
        k, v = k_rows[s], v_rows[s]
        nkv, n_kv = k.shape[0], k.shape[1]
        g = n_head // n_kv
        there = ~np.isnan(k).any(axis=(1, 2)) if nkv else np.zeros(0, bool)
        for t in range(n_q):
            pos = nkv - n_q + t
            lo = max(starts[s] if starts is not None else 0, pos - window + 1 if window else 0, 0)
            if pos < lo:
                continue
            rows = np.arange(lo, pos + 1)
            rows = rows[there[lo:pos + 1]]
            if not rows.size:
                continue
            for h in range(n_head):
                x = np.asarray(q[s, t, h], np.float64)
                kk, vv = k[rows, h // g], v[rows, h // g]
                sc = kk @ x * scale
                mag = (np.abs(kk) @ np.abs(x)).max() * abs(scale)
                if softcap:
                    sc = softcap * np.tanh(sc / softcap)
                if slopes is not None:
                    sc = sc - float(slopes[h]) * (pos - rows)
                p = np.exp(sc - sc.max())
                out[s, t, h] = p @ vv / p.sum()
                seen = np.abs(sc[sc > sc.max() - 25]).max()
                d = mag * (eps_pair + (hd / 16 + 4) * 2.0 ** -23) + 2.0 ** -22 * (seen + softcap)
                w = np.abs(vv).max()
                bound[s, t, h] = w * (math.expm1(2 * d) + eps_pair + 2.0 ** -21 + 2.0 ** -20) + 1e-30
    return out, bound
