"""Trees over a paged cache and the page bookkeeping restated in 64 bits with numpy and plain loops,
without the package, for the tests; and how far the attention kernel may be off, from its inputs."""
import math

import numpy as np

import paged_reference as ref


def rules(parents):
    """(list of each node's visible nodes, depths, wrong) of one tree; a parent outside it counts as none, a
    circle ends where it closes."""
    n, sees, depths, wrong = len(parents), [], [], False
    for t in range(n):
        row, p = [t], int(parents[t])
        while True:
            if p >= n:
                wrong, p = True, -1
            if p < 0:
                break
            if p in row:
                wrong = True
                break
            row.append(p)
            p = int(parents[p])
        sees.append(row)
        depths.append(len(row) - 1)
    return sees, depths, wrong


def words(sees, n_words):
    out = np.zeros((len(sees), n_words), np.uint32)
    for t, row in enumerate(sees):
        for j in row:
            out[t, j // 32] |= np.uint32(1 << (j % 32))
    return out.view(np.int32)


# What one rounding to 16 bits may be off by, and q and the weights in `parts` such roundings of what is left
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def parts_of(kv, src):
    """(parts of q, of a weight; type of the parts)."""
    t = "bf16" if kv == "bf16" else "f16"
    two = src == "f32" or (src == "f16" and kv == "bf16")
    return (2 if two else 1), (2 if two else 1), t


def attend(q, sees, depths, k_rows, v_rows, scale, kv, src, softcap=0.0, slopes=None, window=0, starts=None,
           vmax=None):
    """q: per sequence [n, n_head, hd]; sees, depths: per sequence as from `rules`; k_rows, v_rows: per sequence
    float64 [nkv, n_kv, hd], NaN where a page is not there. Returns per sequence (out, bound).

    The bound. A score is q (in parts, off by at most HALF^parts of itself, 0 for one part of a type that holds it;
    16-bit queries over e4m3 caches in e4m3 parts that hold all their bits, but for what lies below 2^-17 of the row's
    largest: e4m3's smallest step is 2^-9, the row's largest is brought to 2^7 or more, half a step is lost) times exact cache values, summed in 32 bits in steps of 16 products: a step is off by at
    most 2^-21 of the sum of magnitudes A (17 terms cut at 2^-25 of the largest, the sum at 2^-23), and there are
    parts * hd / 16; then a few 32-bit roundings of the score (2^-21 of it) and of the cap. An error d of every
    score moves each weight by a factor within e^(+-2d). A weight is off by HALF^parts of itself and 2^-21 (the
    exponential), or, near the 16-bit types' smallest, by 2^-31 of the row's largest (product with V's
    page scale). The sum of p v is off by 2^-21 of the sum of magnitudes a step of 16 rows and part. The
    result is rounded to its type."""
    out, bound = [], []
    pq, pp, t16 = parts_of(kv, src)
    exact_q = src == t16 or (src == "bf16" and t16 == "f16")
    eps_q = 2.0 ** -38 if exact_q else HALF[t16] ** pq
    if src == "f16" and t16 == "bf16":
        eps_q = HALF[t16] ** 2
    eps_p = HALF[t16] ** pp
    for s in range(len(q)):
        n, n_head, hd = q[s].shape
        k, v = k_rows[s], v_rows[s]
        nkv, n_kv = k.shape[0], k.shape[1]
        g, base = n_head // n_kv, nkv - n
        there = ~np.isnan(k).all(axis=(1, 2)) if nkv else np.zeros(0, bool)
        o, b = np.zeros(q[s].shape), np.zeros(q[s].shape)
        place = np.array([j if j < base else base + depths[s][j - base] for j in range(nkv)])
        for t in range(n):
            x = base + depths[s][t]
            rows = [j for j in range(max(base, 0)) if there[j]]
            rows += [base + y for y in sorted(sees[s][t]) if y < n and base + y >= 0 and there[base + y]]
            rows = np.array(rows, int)
            if starts is not None:
                rows = rows[rows >= starts[s]]
            if window:
                rows = rows[x - place[rows] < window]
            if not rows.size:
                continue
            for h in range(n_head):
                qv = np.asarray(q[s][t, h], np.float64)
                kk, vv = k[rows, h // g], v[rows, h // g]
                sc = kk @ qv * scale
                mag = (np.abs(kk) @ np.abs(qv)).max() * abs(scale)
                lost = 2.0 ** -17 * np.abs(qv).max() * np.abs(kk).sum(-1).max() * abs(scale) if kv == "e4m3" and src != "f32" else 0.0
                if softcap:
                    sc = softcap * np.tanh(sc / softcap)
                if slopes is not None:
                    sc = sc - float(slopes[h]) * (x - place[rows])
                p = np.exp(sc - sc.max())
                total = p.sum()
                o[t, h] = p @ vv / total
                seen = np.abs(sc[sc > sc.max() - 25]).max()
                d = lost + mag * (eps_q + max(pq, 3) * hd / 16 * 2.0 ** -21) + 2.0 ** -21 * (seen + softcap)
                mean = p @ np.abs(vv) / total
                steps = pp * (-(-nkv // 16) + 8)
                b[t, h] = (mean * (math.expm1(2 * d) + eps_p + 2.0 ** -21 + steps * 2.0 ** -21) * 1.01 +
                           rows.size * 2.0 ** -31 * (vmax[s] if vmax is not None else np.abs(vv).max()) / total +
                           HALF[src] * np.abs(o[t, h]) * 1.01 + 2.0 ** -24 * (src == "f16") + 1e-30)
        out.append(o)
        bound.append(b)
    return out, bound


def keep(pool, scale, table, base, path, n):
    """keep_rows on one sequence, in place: values (scale None) or codes with scales [n_pages, n_kv]."""
    page = pool.shape[1]
    at = [(int(table[(base + p) // page]), (base + p) % page) for p in path[:n]]
    if scale is None:
        rows = np.array([pool[pid, o] for pid, o in at])
    else:
        rows = np.array([ref.VALUES[pool[pid, o]] * scale[pid][:, None] for pid, o in at])
    return ref.append(pool, scale, rows, np.asarray(table)[None], [base + n - 1], [n])


def resize(refs, table, page, have, want):
    """In place; returns the error bits (no page 16, shared page 32, bad page 4)."""
    err, up = 0, lambda x: -(-int(x) // page)
    for s in range(len(have)):
        for e in range(up(want[s]), up(have[s])):
            p = table[s, e]
            if p != -1:
                if 0 <= p < len(refs) and refs[p] > 0:
                    refs[p] -= 1
                else:
                    err |= 4
            table[s, e] = -1
    for s in range(len(have)):
        if want[s] < have[s] and want[s] % page:
            p = table[s, up(want[s]) - 1]
            if 0 <= p < len(refs) and refs[p] > 1:
                err |= 32
    free = iter(np.flatnonzero(refs == 0).tolist())
    for s in range(len(have)):
        for e in range(up(have[s]), up(want[s])):
            p = next(free, -1)
            table[s, e] = p
            if p < 0:
                err |= 16
            else:
                refs[p] = 1
    return err


def fork(refs, table, page, src, dst, rows):
    """In place; returns (copies, error bits)."""
    n_seq, cap = table.shape[0], table.shape[1] * page
    copies, err = np.zeros((len(src), 4), np.int32), 0
    free = iter(np.flatnonzero(refs == 0).tolist())
    ok = [0 <= f < n_seq and 0 <= t < n_seq and f != t and 0 <= r <= cap for f, t, r in zip(src, dst, rows)]
    sources, ends = ([int(x) for x, y in zip(a, ok) if y] for a in (src, dst))
    for i, (f, t, r) in enumerate(zip(src, dst, rows)):
        copies[i] = (-1, -1, 0, 0)
        if not ok[i] or t in sources or ends.count(t) > 1:
            err |= 8
            continue
        for e in range(r // page):
            p = table[f, e]
            if 0 <= p < len(refs):
                refs[p] += 1
                table[t, e] = p
            else:
                table[t, e] = -1
                err |= 4
        if r % page:
            p, frm = next(free, -1), table[f, r // page]
            table[t, r // page] = p
            if p < 0:
                err |= 16
            else:
                refs[p] = 1
            if not 0 <= frm < len(refs):
                err |= 4
            elif p >= 0:
                copies[i] = (frm, p, r % page, 0)
    return copies, err
