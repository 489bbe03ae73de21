"""Cases of the paged-cache operators: appending rotated keys and values to a
paged cache (``rope_append``) and decode attention over that cache
(``paged_decode_attention``), held in 8 bits with a scale per page and KV head
or in 16 bits, with plain scores or with scores that are capped, biased by
distance and windowed.

``own`` false: the operators in elementary torch operations. ``own`` true: the
package's entry points. Both read the same prepared tensors.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
          "e4m3": torch.float8_e4m3fn}
ESIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0


def _append(name, n_seq, n_new_lo, n_new_hi, n_head, n_kv, hd, page, kv, src, rot, layout, past):
    return {"name": name, "op": "append", "n_seq": n_seq, "new_lo": n_new_lo, "new_hi": n_new_hi,
            "n_head": n_head, "n_kv": n_kv, "hd": hd, "page": page, "kv": kv, "src": src,
            "rot": rot, "layout": layout, "past": past, "scaling": "none", "fused": False}


def _attend(name, op, n_seq, ctx_lo, ctx_hi, n_q, n_head, n_kv, hd, page, kv, order="rows",
            softcap=0.0, slopes=False, window=0, starts=False):
    return {"name": name, "op": op, "n_seq": n_seq, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "n_q": n_q,
            "n_head": n_head, "n_kv": n_kv, "hd": hd, "page": page, "kv": kv, "order": order,
            "softcap": softcap, "slopes": slopes, "window": window, "starts": starts}


def listed():
    return [
        # one decode step of one sequence of the 7b-like layer: latency alone
        _append("append_step_1", 1, 1, 1, 28, 4, 128, 64, "e4m3", "bf16", 128, "half", 8000),
        # one decode step of a batch; rows still 16-bit; q, k and v are parts of one projection
        dict(_append("append_step_64", 64, 1, 1, 32, 8, 128, 16, "f16", "f16", 128, "half", 4001),
             fused=True),
        # prompts of a batch into the 8-bit cache, ragged
        _append("append_prompts", 6, 200, 2600, 28, 4, 128, 64, "e4m3", "bf16", 128, "half", 37),
        # a long prompt, large heads of which a quarter is rotated, float32 projections
        dict(_append("append_long_part", 1, 8399, 8399, 16, 2, 256, 32, "bf16", "f32", 64,
                     "interleaved", 0), scaling="bands"),
        # the smallest call: a short context
        _attend("attend8_tiny", "attend8", 1, 512, 512, 1, 8, 2, 128, 16, "e4m3"),
        # the 7b-like layer at its full context
        _attend("attend8_7b", "attend8", 1, 8192, 8192, 1, 28, 4, 128, 64, "e4m3"),
        # a ragged batch, up to 32768 rows: bandwidth
        _attend("attend8_ragged", "attend8", 32, 1, 32768, 1, 32, 8, 128, 64, "e4m3"),
        # one very long sequence; pages ordered by head, as a cache laid out for one head's reads
        _attend("attend8_131072", "attend8", 1, 131072, 131072, 1, 64, 8, 128, 128, "e4m3",
                order="heads"),
        # four draft rows a sequence checked at once, head_dim 256
        _attend("attend8_draft", "attend8", 4, 2100, 8400, 4, 16, 2, 256, 32, "e4m3"),
        # capped scores and a sliding window over a 16-bit cache, head_dim 256
        _attend("scored_cap_window", "scored", 8, 300, 8400, 1, 16, 8, 256, 32, "bf16",
                softcap=50.0, window=4096),
        # distance bias, left-padded batch, 16-bit cache
        _attend("scored_distance", "scored", 48, 129, 4097, 1, 32, 8, 128, 16, "f16", slopes=True,
                starts=True),
        # every rule at once, a few query rows, small heads, 8-bit cache
        _attend("scored_all_rows", "scored", 5, 77, 2049, 3, 24, 8, 64, 48, "e4m3", softcap=30.0,
                slopes=True, window=1000, starts=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hd = rng.choice([64, 128, 128, 256])
    n_kv = rng.choice([1, 2, 4, 8])
    group = rng.randint(1, 8)
    page = rng.choice([16, 32, 48, 64, 128, 256])
    kv = rng.choice(["e4m3", "e4m3", "f16", "bf16"])
    op = rng.choice(["append", "attend8", "scored"])
    if op == "append":
        n_seq = _log(rng, 1, 64)
        most = max(1, 6000 // n_seq)
        a, b = _log(rng, 1, most), _log(rng, 1, most)
        c = _append("", n_seq, min(a, b), max(a, b), n_kv * group, n_kv, hd, page, kv,
                    rng.choice(["f32", "f16", "bf16"]), rng.choice([hd, hd, hd // 2, hd // 4]),
                    rng.choice(["half", "interleaved"]), _log(rng, 1, 9000))
        c["scaling"] = rng.choice(["none", "linear", "base", "bands"])
        c["fused"] = rng.random() < 0.5
    else:
        n_seq = _log(rng, 1, 48)
        most = min(131072, max(64, 250000000 // (n_seq * n_kv * hd)))
        a, b = _log(rng, 1, most), _log(rng, 1, most)
        c = _attend("", op, n_seq, min(a, b), max(a, b), rng.choice([1, 1, 1, 2, 3, 5, 8]),
                    n_kv * group, n_kv, hd, page, "e4m3" if op == "attend8" else kv,
                    rng.choice(["rows", "heads"]))
        if op == "scored":
            c["softcap"] = rng.choice([0.0, 20.0, 30.0, 50.0])
            c["slopes"] = rng.random() < 0.5
            c["window"] = rng.choice([0, _log(rng, 1, 8192)])
            c["starts"] = rng.random() < 0.4
            if not (c["softcap"] or c["slopes"] or c["window"] or c["starts"]):
                c["softcap"] = 30.0
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Lengths: the same for every seed, spread over the case's range.
# ---------------------------------------------------------------------------
def _spread(n, lo, hi):
    return [hi if n == 1 else lo + int(round((hi - lo) * ((i * 0.6180339887498949 + 0.05) % 1.0)))
            for i in range(n)]


def _new_counts(c):
    return _spread(c["n_seq"], c["new_lo"], c["new_hi"])


def _contexts(c):
    return _spread(c["n_seq"], c["ctx_lo"], c["ctx_hi"])


def _starts(c, ctx):
    return [(i * 7919) % max(1, n // 3 + 1) for i, n in enumerate(ctx)] if c["starts"] else [0] * len(ctx)


def _rows(c):
    """Rows attended per (sequence, query row), and rows read per sequence."""
    ctx = _contexts(c)
    per, read = [], 0
    for n, st in zip(ctx, _starts(c, ctx)):
        first = n
        for t in range(c["n_q"]):
            pos = n - c["n_q"] + t
            lo = max(st, pos - c["window"] + 1 if c["window"] else 0, 0)
            per.append(max(0, pos + 1 - lo))
            if pos >= lo:
                first = min(first, lo)
        read += n - first
    return per, read


def work(case):
    c = case
    if c["op"] == "append":
        t = sum(_new_counts(c))
        src, dst = ESIZE[c["src"]], ESIZE[c["kv"]]
        q = t * c["n_head"] * c["hd"]
        kv = 2 * t * c["n_kv"] * c["hd"]
        return {"bytes": q * (src + 4) + kv * (src + dst), "flops": 3 * t * c["rot"] * (c["n_head"] + c["n_kv"])}
    per, read = _rows(c)
    es = ESIZE[c["kv"]]
    pages = -(-read // c["page"])
    kv = read * c["n_kv"] * c["hd"] * 2 * es + (8 * pages * c["n_kv"] if es == 1 else 0) + 4 * pages
    io = 2 * c["n_seq"] * c["n_q"] * c["n_head"] * c["hd"] * 4
    return {"bytes": kv + io, "flops": 4 * sum(per) * c["n_head"] * c["hd"]}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
BASE, TRAINED, FACTOR, LOW, HIGH = 10000.0, 8192, 4.0, 1.0, 4.0


def _inv_freq(c):
    """Radians per position of each rotated pair, in 64 bits."""
    rot = c["rot"]
    base = BASE * FACTOR ** (rot / (rot - 2)) if c["scaling"] == "base" else BASE
    f = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    if c["scaling"] == "linear":
        f = f / FACTOR
    elif c["scaling"] == "bands":
        turns = TRAINED * f / (2 * math.pi)
        keep = ((turns - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / FACTOR
    return f


def _scale_for(amax):
    """Smallest power of two s with amax <= 448 s, kept in 2^-60 .. 2^60."""
    m, e = torch.frexp(amax.double())
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-60, 60)
    e = torch.where(amax > 0, e, torch.full_like(e, -60))
    return torch.ldexp(torch.ones_like(amax, dtype=torch.float32), e)


def _to_e4m3(x):
    return x.float().clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _pool(c, n_pages, gen, dev):
    """A filled pool [n_pages, page, n_kv, hd] and its scales: some channels larger than
    others, as keys have them, and pages of different size."""
    shape = (n_pages, c["page"], c["n_kv"], c["hd"])
    heads = c.get("order") == "heads"
    store = (n_pages, c["n_kv"], c["page"], c["hd"]) if heads else shape
    pool = torch.empty(store, dtype=DTYPES[c["kv"]], device=dev)
    if heads:
        pool = pool.transpose(1, 2)
    gain = torch.exp(0.7 * torch.randn(c["n_kv"], c["hd"], generator=gen, device=dev))
    scale = torch.ones(n_pages, c["n_kv"], device=dev) if c["kv"] == "e4m3" else None
    step = max(1, (1 << 27) // (c["page"] * c["n_kv"] * c["hd"]))
    for i in range(0, n_pages, step):
        x = torch.randn((min(step, n_pages - i),) + shape[1:], generator=gen, device=dev)
        x *= gain * torch.exp(0.5 * torch.randn(x.shape[0], 1, 1, 1, generator=gen, device=dev))
        if scale is not None:
            s = _scale_for(x.abs().amax(dim=(1, 3)))
            scale[i:i + step] = s
            pool[i:i + step].view(torch.uint8).copy_(_to_e4m3(x / s[:, None, :, None]).view(torch.uint8))
        else:
            pool[i:i + step].copy_(x)
    return pool, scale


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    new = _new_counts(c) if c["op"] == "append" else None
    ctx = [c["past"] + (i * 13) % 29 * (c["past"] > 0) + n for i, n in enumerate(new)] if new else _contexts(c)
    max_pages = -(-max(ctx) // c["page"])
    used = [-(-n // c["page"]) for n in ctx]
    n_pages = sum(used) + 3
    ids = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((c["n_seq"], max_pages), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = ids[at:at + n]
        at += n
    st = {"case": c, "table": table,
          "positions": torch.tensor([n - 1 for n in ctx], dtype=torch.int32, device=dev)}
    st["k"], st["k_scale"] = _pool(c, n_pages, gen, dev)
    st["v"], st["v_scale"] = _pool(c, n_pages, gen, dev)
    if c["op"] == "append":
        t, dt = sum(new), DTYPES[c["src"]]
        width = (c["n_head"] + 2 * c["n_kv"]) * c["hd"]
        a, b = c["n_head"], c["n_head"] + c["n_kv"]
        if c["fused"]:
            x = torch.randn(t, width, generator=gen, device=dev).to(dt).view(t, -1, c["hd"])
            st["q"], st["k_new"], st["v_new"] = x[:, :a], x[:, a:b], x[:, b:]
        else:
            st["q"] = torch.randn(t, a, c["hd"], generator=gen, device=dev).to(dt)
            st["k_new"] = torch.randn(t, c["n_kv"], c["hd"], generator=gen, device=dev).to(dt)
            st["v_new"] = torch.randn(t, c["n_kv"], c["hd"], generator=gen, device=dev).to(dt)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        st["inv_freq"] = _inv_freq(c).to(dev)
        st["q_out"] = torch.empty(t, a, c["hd"], device=dev)
        st["one_each"] = all(n == 1 for n in new)
    else:
        st["q"] = torch.randn(c["n_seq"], c["n_q"], c["n_head"], c["hd"], generator=gen, device=dev)
        st["out"] = torch.empty_like(st["q"])
        st["scale"] = 1.0 / math.sqrt(c["hd"])
        st["starts"] = torch.tensor(_starts(c, ctx), dtype=torch.int32, device=dev) if c["starts"] else None
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["n_head"] + 1, device=dev) / c["n_head"]) \
            if c["slopes"] else None
    if own:
        import decode_attention_gqa_gb300 as attn
        st["attn"] = attn
        st["cache"] = attn.PagedCache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        if c["op"] == "append":
            how = {"none": attn.ATTN_ROPE_PLAIN, "linear": attn.ATTN_ROPE_LINEAR,
                   "base": attn.ATTN_ROPE_BASE, "bands": attn.ATTN_ROPE_BANDS}[c["scaling"]]
            st["rope"] = attn.Rope(c["rot"], base=BASE, scaling=how, factor=FACTOR, low_turns=LOW,
                                   high_turns=HIGH, trained_len=TRAINED,
                                   interleaved=c["layout"] == "interleaved", device=dev)
    return st


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(state):
    s = state
    c = s["case"]
    if c["op"] == "append":
        if own:
            s["attn"].rope_append(s["cache"], s["table"], s["positions"], s["k_new"], s["v_new"],
                                  q=s["q"], q_out=s["q_out"], rope=s["rope"],
                                  cu_tokens=None if s["one_each"] else s["cu"])
            out = {"q": s["q_out"], "k": s["k"], "v": s["v"]}
        else:
            out = _append_plain(s, c)
        if c["kv"] == "e4m3":
            out["k_scale"], out["v_scale"] = s["k_scale"], s["v_scale"]
        return out
    if own:
        return s["attn"].paged_decode_attention(
            s["cache"], s["table"], s["positions"], s["q"], scale=s["scale"], out=s["out"],
            softcap=c["softcap"], slopes=s["slopes"], window=c["window"], starts=s["starts"])
    return _attend_plain(s, c)


def _rotate(x, cos, sin, rot, layout):
    x = x.double()
    r, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    return torch.cat((r, rest), dim=-1)


def _append_plain(s, c):
    t, page = s["q"].shape[0], c["page"]
    cu, table = s["cu"].long(), s["table"]
    i = torch.arange(t, device=table.device)
    seq = torch.searchsorted(cu, i, right=True) - 1
    pos = s["positions"].long()[seq] + 1 - cu[seq + 1] + i
    pid, off = table[seq, pos // page].long(), pos % page
    ang = pos.double()[:, None] * s["inv_freq"]
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["rot"], c["layout"]))
    k = _rotate(s["k_new"], cos, sin, c["rot"], c["layout"])
    _store(s["k"], s["k_scale"], k, pid, off, c)
    _store(s["v"], s["v_scale"], s["v_new"].double(), pid, off, c)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _store(pool, scale, x, pid, off, c):
    if scale is None:
        pool[pid, off] = x.to(pool.dtype)
        return
    codes = pool.view(torch.uint8)
    n, page = pool.shape[0], c["page"]
    amax = torch.zeros(n, c["n_kv"], dtype=torch.float64, device=x.device)
    amax.scatter_reduce_(0, pid[:, None].expand(-1, c["n_kv"]), x.abs().amax(-1), "amax")
    first = torch.full((n,), page, dtype=torch.int64, device=x.device)
    first.scatter_reduce_(0, pid, off, "amin")
    touched = torch.unique(pid)
    first = first[touched]
    old = scale[touched]
    new = torch.maximum(_scale_for(amax[touched]), torch.where(first[:, None] > 0, old, torch.zeros_like(old)))
    before = codes[touched]                          # rows kept from earlier calls, at the new scale
    kept = _to_e4m3(before.view(torch.float8_e4m3fn).float() * (old / new)[:, None, :, None]).view(torch.uint8)
    row = torch.arange(page, device=x.device)
    codes[touched] = torch.where((row < first[:, None])[:, :, None, None], kept, before)
    scale[touched] = new
    codes[pid, off] = _to_e4m3(x / scale[pid][:, :, None].double()).view(torch.uint8)


def _attend_plain(s, c):
    nq, h, kvh, hd = c["n_q"], c["n_head"], c["n_kv"], c["hd"]
    g = h // kvh
    table = s["table"].long()
    n_seq, rows = table.shape[0], table.shape[1] * c["page"]

    def dense(pool, scale):
        ids = table.clamp(min=0)
        if scale is None:
            x = pool[ids].float()
        else:
            x = pool.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
            x *= scale[ids][:, :, None, :, None]
        return x.reshape(n_seq, rows, kvh, hd).transpose(1, 2)

    q = s["q"].view(n_seq, nq, kvh, g, hd).permute(0, 2, 1, 3, 4).reshape(n_seq, kvh, nq * g, hd)
    score = torch.matmul(q * s["scale"], dense(s["k"], s["k_scale"]).transpose(2, 3))
    score = score.view(n_seq, kvh, nq, g, rows)
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    last = s["positions"].long()[:, None] - nq + 1 + torch.arange(nq, device=q.device)   # [n_seq, nq]
    j = torch.arange(rows, device=q.device)
    dist = last[:, :, None] - j                                                           # [n_seq, nq, rows]
    if s["slopes"] is not None:
        score = score - s["slopes"].view(kvh, 1, g, 1) * dist[:, None, :, None, :]
    ok = dist >= 0
    if c["window"]:
        ok &= dist < c["window"]
    if s["starts"] is not None:
        ok &= j >= s["starts"].long()[:, None, None]
    score = score.masked_fill(~ok[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = (p / torch.where(total > 0, total, torch.ones_like(total))).view(n_seq, kvh, nq * g, rows)
    del score
    o = torch.matmul(p, dense(s["v"], s["v_scale"]))
    return o.view(n_seq, kvh, nq, g, hd).permute(0, 2, 1, 3, 4).reshape(n_seq, nq, h, hd)


# ---------------------------------------------------------------------------
# The definitions in 64 bits, one sequence at a time.
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    return _append_exact(s, c) if c["op"] == "append" else _attend_exact(s, c)


def _append_exact(s, c):
    page, hd, rot = c["page"], c["hd"], c["rot"]
    e4m3 = c["kv"] == "e4m3"
    f = s["inv_freq"]
    out = {"q": torch.empty_like(s["q_out"], dtype=torch.float64)}
    res = {}
    for name in ("k", "v"):
        pool = s[name].double().contiguous()
        res[name] = (pool, s[name + "_scale"].double() if e4m3 else None)

    def turned(x, pos):
        x = x.double().clone()
        z = torch.polar(torch.ones(len(pos), rot // 2, dtype=torch.float64, device=x.device),
                        torch.outer(pos.double(), f))[:, None]
        if c["layout"] == "half":
            w = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
            x[..., :rot // 2], x[..., rot // 2:rot] = w.real, w.imag
        else:
            w = torch.view_as_complex(x[..., :rot].reshape(x.shape[0], x.shape[1], rot // 2, 2).contiguous()) * z
            x[..., :rot] = torch.view_as_real(w).flatten(-2)
        return x

    cu, end, table = s["cu"].tolist(), s["positions"].tolist(), s["table"].tolist()
    for i in range(c["n_seq"]):
        a, b = cu[i], cu[i + 1]
        first = end[i] + 1 - (b - a)
        pos = torch.arange(first, end[i] + 1, device=f.device)
        out["q"][a:b] = turned(s["q"][a:b], pos)
        for name in ("k", "v"):
            x = turned(s["k_new"][a:b], pos) if name == "k" else s["v_new"][a:b].double()
            pool, scale = res[name]
            for p in range(first // page, end[i] // page + 1):
                r0, r1 = max(first, p * page), min(end[i] + 1, (p + 1) * page)
                rows, pid, at = x[r0 - first:r1 - first], table[i][p], r0 - p * page
                if not e4m3:
                    pool[pid, at:at + r1 - r0] = rows
                    continue
                need = torch.exp2(torch.ceil(torch.log2((rows.abs().amax((0, 2)) / E4M3_MAX).clamp(min=2.0 ** -60))))
                new = torch.maximum(need, scale[pid]) if at else need
                pool[pid, :at] *= (scale[pid] / new)[None, :, None]
                pool[pid, at:at + r1 - r0] = rows / new[None, :, None]
                scale[pid] = new
    out["k"], out["v"] = res["k"][0], res["v"][0]
    if e4m3:
        out["k_scale"], out["v_scale"] = res["k"][1], res["v"][1]
    return out


def _attend_exact(s, c):
    nq, kvh, hd = c["n_q"], c["n_kv"], c["hd"]
    g = c["n_head"] // kvh
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for i, p in enumerate(s["positions"].tolist()):
        n = p + 1
        ids = s["table"][i, :-(-n // c["page"])].long()
        kv = []
        for name in ("k", "v"):
            x = (s[name].view(torch.uint8)[ids].view(torch.float8_e4m3fn) if c["kv"] == "e4m3" else s[name][ids]).double()
            if c["kv"] == "e4m3":
                x = x * s[name + "_scale"][ids].double()[:, None, :, None]
            kv.append(x.reshape(-1, kvh, hd)[:n])
        start = int(s["starts"][i]) if s["starts"] is not None else 0
        for t in range(nq):
            last = p - nq + 1 + t
            lo = max(start, last - c["window"] + 1 if c["window"] else 0, 0)
            if last < lo:
                continue
            x = torch.einsum("kgd,nkd->kgn", s["q"][i, t].double().view(kvh, g, hd), kv[0][lo:last + 1]) * s["scale"]
            if c["softcap"]:
                x = torch.tanh(x / c["softcap"]) * c["softcap"]
            if s["slopes"] is not None:
                back = torch.arange(last - lo, -1, -1, device=x.device, dtype=torch.float64)
                x = x - s["slopes"].double().view(kvh, g, 1) * back
            out[i, t] = torch.einsum("kgn,nkd->kgd", torch.softmax(x, -1), kv[1][lo:last + 1]).reshape(-1, hd)
    return out
