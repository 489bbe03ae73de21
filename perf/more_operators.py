"""Cases of the operators that decode with drafted trees over a paged cache, and of the paging below it:
appending a tree's tokens (``tree_rules`` and ``rope_append`` with depths), attention of its nodes
(``tree_decode_attention``), keeping the rows of the accepted path (``keep_rows``), forking sequences
(``PageBook.fork`` and ``copy_pages``) and growing, shrinking and freeing them (``PageBook.resize``).

``own`` false: the operators in elementary torch operations. ``own`` true: the package's entry points. Both
read the same prepared tensors.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
          "e4m3": torch.float8_e4m3fn}
ESIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0
BASE = 10000.0


def _attend(name, n_seq, ctx_lo, ctx_hi, n_lo, n_hi, n_head, n_kv, hd, page, kv, src, softcap=0.0, slopes=False,
            window=0, starts=False):
    return {"name": name, "op": "attend", "n_seq": n_seq, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "n_lo": n_lo,
            "n_hi": n_hi, "n_head": n_head, "n_kv": n_kv, "hd": hd, "page": page, "kv": kv, "src": src,
            "softcap": softcap, "slopes": slopes, "window": window, "starts": starts}


def _append(name, n_seq, n_lo, n_hi, n_head, n_kv, hd, page, kv, src, past, interleaved=False, fused=False):
    return {"name": name, "op": "append", "n_seq": n_seq, "n_lo": n_lo, "n_hi": n_hi, "n_head": n_head, "n_kv": n_kv,
            "hd": hd, "page": page, "kv": kv, "src": src, "past": past, "interleaved": interleaved, "fused": fused}


def _keep(name, n_seq, n_nodes, keep_lo, keep_hi, n_kv, hd, page, kv, past):
    return {"name": name, "op": "keep", "n_seq": n_seq, "n_nodes": n_nodes, "keep_lo": keep_lo, "keep_hi": keep_hi,
            "n_kv": n_kv, "hd": hd, "page": page, "kv": kv, "past": past}


def _fork(name, n_src, children, rows_lo, rows_hi, n_kv, hd, page, kv, spare):
    return {"name": name, "op": "fork", "n_src": n_src, "children": children, "rows_lo": rows_lo, "rows_hi": rows_hi,
            "n_kv": n_kv, "hd": hd, "page": page, "kv": kv, "spare": spare}


def _resize(name, n_seq, max_pages, rows_hi, step, page, spare):
    return {"name": name, "op": "resize", "n_seq": n_seq, "max_pages": max_pages, "rows_hi": rows_hi, "step": step,
            "page": page, "spare": spare}


def listed():
    return [
        # the smallest call: a short context and a small tree, float32 queries
        _attend("tree_tiny", 1, 512, 512, 8, 8, 8, 2, 128, 16, "e4m3", "f32"),
        # the 7b-like layer at its full context, one sequence, a tree of 64 nodes
        _attend("tree_7b", 1, 8192, 8192, 64, 64, 28, 4, 128, 64, "e4m3", "bf16"),
        # a ragged batch up to 32768 rows, trees of different size
        _attend("tree_ragged", 32, 17, 32768, 5, 16, 32, 8, 128, 64, "e4m3", "bf16"),
        # large heads, capped scores, a window by position, a 16-bit cache
        _attend("tree_cap_window", 4, 2100, 8400, 33, 60, 16, 2, 256, 32, "bf16", "bf16", softcap=50.0, window=4096),
        # one decode step of one sequence of the 7b-like layer: latency
        _append("tree_append_1", 1, 64, 64, 28, 4, 128, 64, "e4m3", "bf16", 8000),
        # a batch, trees of different size, q, k and v parts of one projection
        _append("tree_append_48", 48, 7, 26, 32, 8, 128, 16, "f16", "f16", 4001, fused=True),
        # the accepted path of one sequence
        _keep("keep_1", 1, 64, 5, 5, 4, 128, 64, "e4m3", 8000),
        # the accepted paths of a batch, large heads
        _keep("keep_64", 64, 40, 1, 12, 8, 256, 32, "bf16", 1003),
        # a beam step of one sequence: four children
        _fork("fork_4", 1, 4, 1000, 1000, 4, 128, 64, "e4m3", 100),
        # a beam step of a batch: 16 prompts with four children each
        _fork("fork_64", 16, 4, 900, 4097, 8, 128, 128, "f16", 1000),
        # a decode step of a batch: a tree more for each sequence
        _resize("resize_64", 64, 64, 4001, 40, 64, 3000),
        # a thousand sequences that grow, shrink, begin and end over a large pool
        _resize("resize_1000", 1000, 512, 8192, 0, 16, 100000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hd = rng.choice([64, 128, 128, 256])
    n_kv = rng.choice([1, 2, 4, 8])
    group = rng.randint(1, 8)
    page = rng.choice([16, 32, 48, 64, 128, 256])
    kv = rng.choice(["e4m3", "e4m3", "f16", "bf16"])
    op = rng.choice(["attend", "attend", "append", "keep", "fork", "resize"])
    if op == "attend":
        n_seq, n = _log(rng, 1, 48), _log(rng, 1, 128)
        most = min(131072, 250000000 // (n_seq * n_kv * hd), 20000000000 // (n_seq * n * n_kv * group * hd))
        most = max(most, n + 1)
        a, b = _log(rng, n, most), _log(rng, n, most)
        rules = rng.random() < 0.4
        c = _attend("", n_seq, min(a, b), max(a, b), _log(rng, 1, n), n, n_kv * group, n_kv, hd, page, kv,
                    rng.choice(["f32", "f16", "bf16"]),
                    softcap=rng.choice([0.0, 30.0, 50.0]) if rules else 0.0, slopes=rules and rng.random() < 0.5,
                    window=rng.choice([0, _log(rng, 4, 8192)]) if rules else 0, starts=rng.random() < 0.3)
    elif op == "append":
        a, b = _log(rng, 1, 128), _log(rng, 1, 128)
        c = _append("", _log(rng, 1, 64), min(a, b), max(a, b), n_kv * group, n_kv, hd, page, kv,
                    rng.choice(["f32", "f16", "bf16"]), _log(rng, 1, 9000), rng.random() < 0.5, rng.random() < 0.5)
    elif op == "keep":
        n = _log(rng, 1, 128)
        a, b = _log(rng, 1, n), _log(rng, 1, n)
        c = _keep("", _log(rng, 1, 64), n, min(a, b), max(a, b), n_kv, hd, page, kv, _log(rng, 1, 2000))
    elif op == "fork":
        n_src = _log(rng, 1, 16)
        a, b = _log(rng, 1, 4097), _log(rng, 1, 4097)
        c = _fork("", n_src, rng.randint(1, 6), min(a, b), max(a, b), n_kv, hd, page, kv, _log(rng, 100, 2000))
    else:
        page = rng.choice([16, 32, 64, 128])
        n_seq, pages = _log(rng, 1, 1000), _log(rng, 4, 500)
        c = _resize("", n_seq, pages, _log(rng, page, pages * page), rng.choice([0, _log(rng, 1, 3 * page)]), page,
                    _log(rng, 100, 100000))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Lengths: the same for every seed, spread over the case's range.
# ---------------------------------------------------------------------------
def _spread(n, lo, hi, shift=0.05):
    return [hi if n == 1 else lo + int(round((hi - lo) * ((i * 0.6180339887498949 + shift) % 1.0)))
            for i in range(n)]


def _nodes(c):
    return _spread(c["n_seq"], c["n_lo"], c["n_hi"], 0.4)


def _contexts(c):
    return [max(x, n) for x, n in zip(_spread(c["n_seq"], c["ctx_lo"], c["ctx_hi"]), _nodes(c))]


def _starts(c, ctx):
    nodes = _nodes(c)
    return [(i * 7919) % max(1, (x - nodes[i]) // 3 + 1) for i, x in enumerate(ctx)] if c["starts"] else [0] * len(ctx)


def _sizes(c):
    """Rows that each sequence of a resize case has in its two states."""
    n, top = c["n_seq"], min(c["rows_hi"], c["max_pages"] * c["page"])
    a = _spread(n, 0 if n > 1 and not c["step"] else 1, top)
    if c["step"]:
        b = [min(x + 1 + (i * 31) % c["step"], c["max_pages"] * c["page"]) for i, x in enumerate(a)]
    else:
        b = _spread(n, 0, top, 0.55) if n > 1 else [top // 2]
        b = [0 if i % 11 == 3 else y for i, y in enumerate(b)]
    return a, b


def _up(x, y):
    return -(-x // y)


def work(case):
    c = case
    if c["op"] == "attend":
        ctx, es = _contexts(c), ESIZE[c["kv"]]
        rows = pairs = 0
        for x, n, st in zip(ctx, _nodes(c), _starts(c, ctx)):
            seen = min(x - n - st, c["window"] - 1) if c["window"] else x - n - st
            rows += max(seen, 0) + n
            pairs += n * (max(seen, 0) + 1)
        t = sum(_nodes(c))
        kv = rows * c["n_kv"] * (c["hd"] * 2 * es + (8.0 / c["page"] if es == 1 else 0))
        io = 2 * t * c["n_head"] * c["hd"] * ESIZE[c["src"]] + t * _up(c["n_hi"], 32) * 4
        return {"bytes": kv + io, "flops": 4 * pairs * c["n_head"] * c["hd"]}
    if c["op"] == "append":
        t = sum(_nodes(c))
        src, dst = ESIZE[c["src"]], ESIZE[c["kv"]]
        return {"bytes": t * c["n_head"] * c["hd"] * (src + 4) + 2 * t * c["n_kv"] * c["hd"] * (src + dst) +
                t * (8 + 4 * _up(c["n_hi"], 32)), "flops": 3 * t * c["hd"] * (c["n_head"] + c["n_kv"])}
    if c["op"] == "keep":
        t = sum(_spread(c["n_seq"], c["keep_lo"], c["keep_hi"]))
        return {"bytes": 4 * t * c["n_kv"] * c["hd"] * ESIZE[c["kv"]], "flops": 0}
    if c["op"] == "fork":
        rows = _spread(c["n_src"], c["rows_lo"], c["rows_hi"])
        moved = sum(x % c["page"] for x in rows) * c["children"]
        entries = sum(_up(x, c["page"]) for x in rows) * c["children"]
        return {"bytes": 4 * moved * c["n_kv"] * c["hd"] * ESIZE[c["kv"]] + 16 * entries, "flops": 0}
    a, b = _sizes(c)
    moved = sum(abs(_up(x, c["page"]) - _up(y, c["page"])) for x, y in zip(a, b))
    held = sum(max(_up(x, c["page"]), _up(y, c["page"])) for x, y in zip(a, b))
    return {"bytes": 4 * (held + c["spare"]) + 8 * moved + 8 * c["n_seq"], "flops": 0}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _scale_for(amax):
    """Smallest power of two s with amax <= 448 s, kept in 2^-60 .. 2^60."""
    m, e = torch.frexp(amax.double())
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-60, 60)
    e = torch.where(amax > 0, e, torch.full_like(e, -60))
    return torch.ldexp(torch.ones_like(amax, dtype=torch.float32), e)


def _to_e4m3(x):
    return x.float().clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _pool(c, n_pages, gen, dev):
    """A filled pool [n_pages, page, n_kv, hd] and its scales: some channels larger than others, as keys
    have them, and pages of different size."""
    pool = torch.empty(n_pages, c["page"], c["n_kv"], c["hd"], dtype=DTYPES[c["kv"]], device=dev)
    gain = torch.exp(0.7 * torch.randn(c["n_kv"], c["hd"], generator=gen, device=dev))
    scale = torch.ones(n_pages, c["n_kv"], device=dev) if c["kv"] == "e4m3" else None
    step = max(1, (1 << 27) // (c["page"] * c["n_kv"] * c["hd"]))
    for i in range(0, n_pages, step):
        x = torch.randn((min(step, n_pages - i),) + pool.shape[1:], generator=gen, device=dev)
        x *= gain * torch.exp(0.5 * torch.randn(x.shape[0], 1, 1, 1, generator=gen, device=dev))
        if scale is not None:
            s = _scale_for(x.abs().amax(dim=(1, 3)))
            scale[i:i + step] = s
            pool[i:i + step].view(torch.uint8).copy_(_to_e4m3(x / s[:, None, :, None]).view(torch.uint8))
        else:
            pool[i:i + step].copy_(x)
    return pool, scale


def _parents(nodes, rng):
    """A drafted tree per sequence: each node hangs on one of the eight before it, or on the context."""
    return [-1 if t == 0 else rng.randint(max(-1, t - 8), t - 1) for n in nodes for t in range(n)]


def _int(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _pages(c, used, n_pages, max_pages, gen, dev):
    """A table [n_seq, max_pages] of pages in random order, -1 where a sequence has none."""
    ids = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(used), max_pages), -1, dtype=torch.int32, device=dev)
    n = torch.tensor(used, device=dev)
    have = torch.arange(max_pages, device=dev) < n[:, None]
    table[have] = ids[:sum(used)]
    return table


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    st = {"case": c}
    if own:
        import decode_attention_gqa_gb300 as attn
        st["attn"] = attn
    if c["op"] in ("attend", "append"):
        nodes = _nodes(c)
        ctx = _contexts(c) if c["op"] == "attend" else [c["past"] + (i * 13) % 29 + n for i, n in enumerate(nodes)]
        used = [_up(x, c["page"]) for x in ctx]
        n_pages = sum(used) + 3
        st["table"] = _pages(c, used, n_pages, max(used), gen, dev)
        st["positions"] = _int([x - 1 for x in ctx], dev)
        cu = [0]
        for n in nodes:
            cu.append(cu[-1] + n)
        st["cu"], st["most"], st["parents"] = _int(cu, dev), max(nodes), _int(_parents(nodes, rng), dev)
        t = cu[-1]
    if c["op"] == "attend":
        st["k"], st["k_scale"] = _pool(c, n_pages, gen, dev)
        st["v"], st["v_scale"] = _pool(c, n_pages, gen, dev)
        st["mask"], st["depths"] = _rules_plain(st)
        st["q"] = torch.randn(t, c["n_head"], c["hd"], generator=gen, device=dev).to(DTYPES[c["src"]])
        st["out"] = torch.empty_like(st["q"])
        st["scale"] = 1.0 / math.sqrt(c["hd"])
        st["starts"] = _int(_starts(c, ctx), dev) if c["starts"] else None
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["n_head"] + 1, device=dev) / c["n_head"]) \
            if c["slopes"] else None
    elif c["op"] == "append":
        st["k"], st["k_scale"] = _pool(c, n_pages, gen, dev)
        st["v"], st["v_scale"] = _pool(c, n_pages, gen, dev)
        dt, h, kvh, hd = DTYPES[c["src"]], c["n_head"], c["n_kv"], c["hd"]
        if c["fused"]:
            x = torch.randn(t, (h + 2 * kvh) * hd, generator=gen, device=dev).to(dt).view(t, -1, hd)
            st["q"], st["k_new"], st["v_new"] = x[:, :h], x[:, h:h + kvh], x[:, h + kvh:]
        else:
            st["q"] = torch.randn(t, h, hd, generator=gen, device=dev).to(dt)
            st["k_new"] = torch.randn(t, kvh, hd, generator=gen, device=dev).to(dt)
            st["v_new"] = torch.randn(t, kvh, hd, generator=gen, device=dev).to(dt)
        st["inv_freq"] = torch.tensor([BASE ** (-2.0 * i / hd) for i in range(hd // 2)], dtype=torch.float64, device=dev)
        st["q_out"] = torch.empty(t, h, hd, device=dev)
        if own:
            st["rope"] = attn.Rope(hd, base=BASE, interleaved=c["interleaved"], device=dev)
    elif c["op"] == "keep":
        keep = _spread(c["n_seq"], c["keep_lo"], c["keep_hi"])
        past = [c["past"] + (i * 13) % 29 for i in range(c["n_seq"])]
        used = [_up(x + c["n_nodes"], c["page"]) for x in past]
        n_pages = sum(used) + 3
        st["table"] = _pages(c, used, n_pages, max(used), gen, dev)
        st["k"], st["k_scale"] = _pool(c, n_pages, gen, dev)
        st["v"], st["v_scale"] = _pool(c, n_pages, gen, dev)
        most = max(keep)
        st["base"], st["kept"] = _int(past, dev), _int(keep, dev)
        st["path"] = _int([sorted(rng.sample(range(c["n_nodes"]), n)) + [-1] * (most - n) for n in keep], dev)
    elif c["op"] == "fork":
        rows = _spread(c["n_src"], c["rows_lo"], c["rows_hi"])
        n, m = c["n_src"], c["children"]
        used = [_up(x, c["page"]) for x in rows]
        n_pages = sum(used) + n * m + c["spare"]
        max_pages = max(used) + 1
        table = torch.full((n * (m + 1), max_pages), -1, dtype=torch.int32, device=dev)
        table[:n] = _pages(c, used, n_pages, max_pages, gen, dev)
        refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        refs.index_add_(0, table[:n][table[:n] >= 0].long(), torch.ones(sum(used), dtype=torch.int32, device=dev))
        st.update(refs=refs, table=table)
        st["src"] = _int([i for i in range(n) for _ in range(m)], dev)
        st["dst"] = _int([n + i for i in range(n * m)], dev)
        st["rows"] = _int([rows[i] for i in range(n) for _ in range(m)], dev)
        # the beams of the step before, which this one replaces
        st["have"] = torch.cat((_int(rows, dev), st["rows"]))
        st["want"] = torch.cat((_int(rows, dev), torch.zeros_like(st["rows"])))
        _fork_plain(st, c)
        st["k"], st["k_scale"] = _pool(c, n_pages, gen, dev)
        st["v"], st["v_scale"] = _pool(c, n_pages, gen, dev)
    else:
        a, b = _sizes(c)
        used = [_up(x, c["page"]) for x in a]
        grown = sum(max(_up(x, c["page"]), _up(y, c["page"])) for x, y in zip(a, b))
        n_pages = grown + c["spare"]
        st["table"] = _pages(c, used, n_pages, c["max_pages"], gen, dev)
        st["refs"] = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        held = st["table"][st["table"] >= 0].long()
        st["refs"][held] = 1
        st["sizes"], st["at"] = (_int(a, dev), _int(b, dev)), 0
    if own:
        if "k" in st:
            st["cache"] = attn.PagedCache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        if "refs" in st:
            st["book"] = attn.PageBook(st["refs"], st["table"], c["page"])
    return st


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def _cache_of(s, out):
    out["k"], out["v"] = s["k"], s["v"]
    if s["k_scale"] is not None:
        out["k_scale"], out["v_scale"] = s["k_scale"], s["v_scale"]
    return out


def run(state):
    s = state
    c = s["case"]
    if c["op"] == "attend":
        if own:
            return s["attn"].tree_decode_attention(
                s["cache"], s["table"], s["positions"], s["q"], mask=s["mask"], depths=s["depths"], cu_tokens=s["cu"],
                max_nodes=s["most"], scale=s["scale"], out=s["out"], softcap=c["softcap"], slopes=s["slopes"],
                window=c["window"], starts=s["starts"])
        return _attend_plain(s, c)
    if c["op"] == "append":
        if own:
            mask, depths = s["attn"].tree_rules(s["parents"], cu_tokens=s["cu"], max_nodes=s["most"])
            s["attn"].rope_append(s["cache"], s["table"], s["positions"], s["k_new"], s["v_new"], q=s["q"],
                                  q_out=s["q_out"], rope=s["rope"], cu_tokens=s["cu"], depths=depths)
        else:
            mask, depths = _rules_plain(s)
            _append_plain(s, c, depths)
        return _cache_of(s, {"mask": mask, "depths": depths, "q": s["q_out"]})
    if c["op"] == "keep":
        if own:
            s["attn"].keep_rows(s["cache"], s["table"], s["base"], s["path"], s["kept"])
        else:
            _keep_plain(s, c)
        return _cache_of(s, {})
    if c["op"] == "fork":
        if own:
            s["book"].resize(s["have"], s["want"])
            copies = s["book"].fork(s["src"], s["dst"], s["rows"])
            s["attn"].copy_pages(s["cache"], copies)
        else:
            _resize_plain(s, c, s["have"], s["want"])
            copies = _fork_plain(s, c)
            _copy_plain(s, c, copies)
        return _cache_of(s, {"table": s["table"], "refs": s["refs"], "copies": copies})
    have, want = s["sizes"][s["at"]], s["sizes"][1 - s["at"]]
    s["at"] = 1 - s["at"]
    if own:
        s["book"].resize(have, want)
    else:
        _resize_plain(s, c, have, want)
    return {"table": s["table"], "refs": s["refs"]}


def _where(s):
    """Sequence of each token, its place in it, and the row it has in the cache."""
    cu = s["cu"].long()
    i = torch.arange(s["parents"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu, i, right=True) - 1
    at = i - cu[seq]
    return seq, at, s["positions"].long()[seq] + 1 - cu[seq + 1] + i


def _rules_plain(s):
    """The rows of the tree that each node sees (itself and its ancestors) as bits, and its depth."""
    parents, cu, most = s["parents"].long(), s["cu"].long(), s["most"]
    t = parents.shape[0]
    i = torch.arange(t, device=cu.device)
    first = cu[torch.searchsorted(cu, i, right=True) - 1]
    # up: ancestors 2^k levels above, as an index of all tokens; t stands for none
    up = torch.cat((torch.where(parents < 0, t, first + parents), torch.tensor([t], device=cu.device)))
    words = _up(most, 32)
    seen = torch.zeros(t + 1, words * 32, dtype=torch.bool, device=cu.device)
    seen[i, i - first] = True
    depth = torch.zeros(t + 1, dtype=torch.int64, device=cu.device)
    depth[:t] = (parents >= 0).long()
    k = 1
    while k < most:
        seen = seen | seen[up]
        depth = depth + depth[up]
        up = up[up]
        k *= 2
    bits = seen[:t].view(t, words, 32).long() << torch.arange(32, device=cu.device)
    word = bits.sum(-1)
    return torch.where(word >= 1 << 31, word - (1 << 32), word).int(), depth[:t].int()


def _rotate(x, cos, sin, interleaved):
    x = x.double()
    half = x.shape[-1] // 2
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)


def _append_plain(s, c, depths):
    seq, at, row = _where(s)
    pid, off = s["table"][seq, row // c["page"]].long(), row % c["page"]
    ang = (row - at + depths).double()[:, None] * s["inv_freq"]
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["interleaved"]))
    _store(s["k"], s["k_scale"], _rotate(s["k_new"], cos, sin, c["interleaved"]), pid, off, c)
    _store(s["v"], s["v_scale"], s["v_new"].double(), pid, off, c)


def _store(pool, scale, x, pid, off, c):
    """Rows x [tokens, n_kv, hd] into places (pid, off) of the pool; a page's rows before the first of
    them keep their values."""
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
    before = codes[touched]
    kept = _to_e4m3(before.view(torch.float8_e4m3fn).float() * (old / new)[:, None, :, None]).view(torch.uint8)
    row = torch.arange(page, device=x.device)
    codes[touched] = torch.where((row < first[:, None])[:, :, None, None], kept, before)
    scale[touched] = new
    codes[pid, off] = _to_e4m3(x / scale[pid][:, :, None].double()).view(torch.uint8)


def _keep_plain(s, c):
    most = s["path"].shape[1]
    i = torch.arange(most, device=s["path"].device)
    live = i < s["kept"][:, None]
    seq = torch.arange(c["n_seq"], device=i.device)[:, None].expand(-1, most)[live]
    old = (s["base"][:, None].long() + s["path"])[live]
    new = (s["base"][:, None].long() + i)[live]
    page = c["page"]
    frm, at = s["table"][seq, old // page].long(), old % page
    to, off = s["table"][seq, new // page].long(), new % page
    for name in ("k", "v"):
        pool, scale = s[name], s[name + "_scale"]
        if scale is None:
            x = pool[frm, at].double()
        else:
            x = pool.view(torch.uint8)[frm, at].view(torch.float8_e4m3fn).double() * scale[frm][:, :, None]
        _store(pool, scale, x, to, off, c)


def _take_free(refs, n):
    """The lowest-numbered pages that nothing holds, for requests numbered from 1 in `n`; -1 past the last."""
    free = (refs == 0).cumsum(0)
    page = torch.searchsorted(free, n)
    return torch.where(page < refs.shape[0], page, -1)


def _resize_plain(s, c, have, want):
    refs, table = s["refs"], s["table"]
    i = torch.arange(table.shape[1], device=table.device)
    a = ((have.long() + c["page"] - 1) // c["page"])[:, None]
    b = ((want.long() + c["page"] - 1) // c["page"])[:, None]
    gone = (i >= b) & (i < a) & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).flatten().long(), -gone.flatten().int())
    new = (i >= a) & (i < b)
    page = _take_free(refs, new.flatten().cumsum(0)).view(new.shape)
    got = new & (page >= 0)
    refs.index_add_(0, page.clamp(min=0).flatten(), got.flatten().int())
    table.copy_(torch.where(new, page.int(), torch.where((i >= b) & (i < a), -1, table)))


def _fork_plain(s, c):
    refs, table, src, dst, rows = s["refs"], s["table"], s["src"].long(), s["dst"].long(), s["rows"].long()
    i = torch.arange(table.shape[1], device=table.device)
    full, rest = rows // c["page"], rows % c["page"]
    shared = i < full[:, None]
    refs.index_add_(0, table[src].clamp(min=0).flatten().long(), shared.flatten().int())
    part = rest > 0
    page = _take_free(refs, part.cumsum(0))
    got = part & (page >= 0)
    refs.index_add_(0, page.clamp(min=0), got.int())
    last = torch.gather(table[src], 1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    table[dst] = torch.where(shared, table[src], torch.where((i == full[:, None]) & part[:, None],
                                                             page[:, None].int(), table[dst]))
    none = torch.full_like(rows, -1)
    return torch.stack((torch.where(got, last, none), torch.where(got, page, none), torch.where(got, rest, 0),
                        torch.zeros_like(rows)), 1).int()


def _copy_plain(s, c, copies):
    frm, to, rows = copies[:, 0].long(), copies[:, 1].long(), copies[:, 2]
    n = s["k"].shape[0]
    # what nothing is copied to is written back as it is
    source = torch.arange(n + 1, device=frm.device)
    upto = torch.zeros(n + 1, dtype=torch.int32, device=frm.device)
    source[torch.where(to < 0, n, to)] = torch.where(to < 0, n, frm)
    upto[torch.where(to < 0, n, to)] = torch.where(to < 0, 0, rows)
    at = torch.where(to < 0, 0, to)
    src, m = source[at], upto[at]
    row = torch.arange(c["page"], device=frm.device)
    for name in ("k", "v"):
        pool = s[name].view(torch.uint8) if c["kv"] == "e4m3" else s[name]
        pool[at] = torch.where((row < m[:, None])[:, :, None, None], pool[src], pool[at])
        if s[name + "_scale"] is not None:
            s[name + "_scale"][at] = s[name + "_scale"][src]


def _attend_plain(s, c):
    h, kvh, hd, most = c["n_head"], c["n_kv"], c["hd"], s["most"]
    g = h // kvh
    table = s["table"].long()
    n_seq, rows = table.shape[0], table.shape[1] * c["page"]
    seq, at, row = _where(s)

    def dense(pool, scale):
        ids = table.clamp(min=0)
        if scale is None:
            x = pool[ids].float()
        else:
            x = pool.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
            x *= scale[ids][:, :, None, :, None]
        return x.reshape(n_seq, rows, kvh, hd).transpose(1, 2)

    q = torch.zeros(n_seq, most, h, hd, device=table.device)
    q[seq, at] = s["q"].float()
    q = q.view(n_seq, most, kvh, g, hd).permute(0, 2, 1, 3, 4).reshape(n_seq, kvh, most * g, hd)
    score = torch.matmul(q * s["scale"], dense(s["k"], s["k_scale"]).transpose(2, 3))
    score = score.view(n_seq, kvh, most, g, rows)
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    j = torch.arange(rows, device=q.device)
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    base = s["positions"].long() + 1 - n
    node = j - base[:, None]                                               # [n_seq, rows]: below 0 for the context
    drafted = (node >= 0) & (node < n[:, None])
    depth = torch.zeros(n_seq, most, dtype=torch.int64, device=q.device)
    depth[seq, at] = s["depths"].long()
    mask = torch.zeros(n_seq, most, s["mask"].shape[1], dtype=torch.int32, device=q.device)
    mask[seq, at] = s["mask"]
    bits = (mask[..., None] >> torch.arange(32, device=q.device)) & 1
    sees = torch.gather(bits.flatten(2), 2, node.clamp(0, most - 1)[:, None].expand(-1, most, -1)) > 0
    ok = (node < 0)[:, None] | (drafted[:, None] & sees)                   # [n_seq, most, rows]
    place = torch.where(node < 0, j, base[:, None] + torch.gather(depth, 1, node.clamp(0, most - 1)))
    dist = (base[:, None] + depth)[:, :, None] - place[:, None]
    if s["slopes"] is not None:
        score = score - s["slopes"].view(kvh, 1, g, 1) * dist[:, None, :, None, :]
    if c["window"]:
        ok &= dist < c["window"]
    if s["starts"] is not None:
        ok &= j >= s["starts"].long()[:, None, None]
    score = score.masked_fill(~ok[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    del score
    total = p.sum(-1, keepdim=True)
    p = (p / torch.where(total > 0, total, torch.ones_like(total))).view(n_seq, kvh, most * g, rows)
    o = torch.matmul(p, dense(s["v"], s["v_scale"]))
    o = o.view(n_seq, kvh, most, g, hd).permute(0, 2, 1, 3, 4).reshape(n_seq, most, h, hd)
    return o[seq, at].to(s["q"].dtype)


# ---------------------------------------------------------------------------
# The definitions in 64 bits, one sequence at a time.
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "attend":
        return _attend_exact(s, c)
    if c["op"] == "append":
        return _append_exact(s, c)
    if c["op"] == "keep":
        return _keep_exact(s, c)
    if c["op"] == "fork":
        return _fork_exact(s, c)
    return None                      # numbers of pages alone


def _ancestors(parents):
    """Each node's path from itself up to the context."""
    out = []
    for t, p in enumerate(parents):
        out.append([t] + (out[p] if p >= 0 else []))
    return out


def _attend_exact(s, c):
    kvh, hd = c["n_kv"], c["hd"]
    g = c["n_head"] // kvh
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    cu, parents = s["cu"].tolist(), s["parents"].tolist()
    for i, p in enumerate(s["positions"].tolist()):
        a, n = cu[i], cu[i + 1] - cu[i]
        base = p + 1 - n
        paths = _ancestors(parents[a:a + n])
        ids = s["table"][i, :_up(p + 1, c["page"])].long()
        kv = []
        for name in ("k", "v"):
            x = (s[name].view(torch.uint8)[ids].view(torch.float8_e4m3fn) if c["kv"] == "e4m3" else s[name][ids]).double()
            if c["kv"] == "e4m3":
                x = x * s[name + "_scale"][ids].double()[:, None, :, None]
            kv.append(x.reshape(-1, kvh, hd)[:p + 1])
        start = int(s["starts"][i]) if s["starts"] is not None else 0
        place = torch.tensor(list(range(base)) + [base + len(x) - 1 for x in paths], device=out.device)
        sees = torch.zeros(n, p + 1, dtype=torch.bool, device=out.device)
        sees[:, start:base] = True
        for t, path in enumerate(paths):
            sees[t, [base + x for x in path]] = True
        sees[:, :start] = False
        dist = place[base:, None] - place
        if c["window"]:
            sees &= dist < c["window"]
        x = torch.einsum("tkgd,nkd->tkgn", s["q"][a:a + n].double().view(n, kvh, g, hd), kv[0]) * s["scale"]
        if c["softcap"]:
            x = torch.tanh(x / c["softcap"]) * c["softcap"]
        if s["slopes"] is not None:
            x = x - s["slopes"].double().view(1, kvh, g, 1) * dist[:, None, None]
        x = torch.where(sees[:, None, None], x, -math.inf)
        out[a:a + n] = torch.einsum("tkgn,nkd->tkgd", torch.softmax(x, -1), kv[1]).reshape(n, -1, hd)
    return out


def _put(pool, scale, ids, first, rows):
    """Rows [n, n_kv, hd] to cache rows first .. of the sequence with pages `ids`, in values; scales as an append
    leaves them."""
    page = pool.shape[1]
    for p in range(first // page, (first + len(rows) - 1) // page + 1):
        r0, r1 = max(first, p * page), min(first + len(rows), (p + 1) * page)
        x, pid, at = rows[r0 - first:r1 - first], ids[p], r0 - p * page
        if scale is None:
            pool[pid, at:at + r1 - r0] = x
            continue
        need = torch.exp2(torch.ceil(torch.log2((x.abs().amax((0, 2)) / E4M3_MAX).clamp(min=2.0 ** -60))))
        new = torch.maximum(need, scale[pid]) if at else need
        pool[pid, :at] *= (scale[pid] / new)[None, :, None]
        pool[pid, at:at + r1 - r0] = x / new[None, :, None]
        scale[pid] = new


def _pools(s):
    out = {}
    for name in ("k", "v"):
        x = s[name].view(torch.uint8).view(torch.float8_e4m3fn) if s[name + "_scale"] is not None else s[name]
        out[name] = (x.double(), None if s[name + "_scale"] is None else s[name + "_scale"].double())
    return out


def _append_exact(s, c):
    pools = _pools(s)
    cu, parents, table = s["cu"].tolist(), s["parents"].tolist(), s["table"].tolist()
    q_out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    half = c["hd"] // 2

    def turned(x, place):
        z = torch.polar(torch.ones(len(place), half, dtype=torch.float64, device=x.device),
                        torch.outer(torch.tensor(place, dtype=torch.float64, device=x.device), s["inv_freq"]))[:, None]
        x = x.double()
        if c["interleaved"]:
            return torch.view_as_real(torch.view_as_complex(x.reshape(x.shape[0], x.shape[1], half, 2).contiguous()) * z).flatten(-2)
        w = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * z
        return torch.cat((w.real, w.imag), -1)

    for i, last in enumerate(s["positions"].tolist()):
        a, b = cu[i], cu[i + 1]
        base = last + 1 - (b - a)
        place = [base + len(x) - 1 for x in _ancestors(parents[a:b])]
        q_out[a:b] = turned(s["q"][a:b], place)
        _put(*pools["k"], table[i], base, turned(s["k_new"][a:b], place))
        _put(*pools["v"], table[i], base, s["v_new"][a:b].double())
    out = {"mask": None, "depths": None, "q": q_out, "k": pools["k"][0], "v": pools["v"][0]}
    if c["kv"] == "e4m3":
        out["k_scale"], out["v_scale"] = pools["k"][1], pools["v"][1]
    return out


def _keep_exact(s, c):
    pools = _pools(s)
    table, page = s["table"].tolist(), c["page"]
    for i, n in enumerate(s["kept"].tolist()):
        base, path = int(s["base"][i]), s["path"][i, :n].tolist()
        for name in ("k", "v"):
            pool, scale = pools[name]
            rows = []
            for p in path:
                pid, at = table[i][(base + p) // page], (base + p) % page
                rows.append(pool[pid, at] * (1.0 if scale is None else scale[pid][:, None]))
            _put(pool, scale, table[i], base, torch.stack(rows))
    out = {"k": pools["k"][0], "v": pools["v"][0]}
    if c["kv"] == "e4m3":
        out["k_scale"], out["v_scale"] = pools["k"][1], pools["v"][1]
    return out


def _fork_exact(s, c):
    pools, page = _pools(s), c["page"]
    table, refs = s["table"].tolist(), s["refs"].tolist()
    src, dst, rows = s["src"].tolist(), s["dst"].tolist(), s["rows"].tolist()
    for d, r in zip(dst, rows):
        for p in table[d][:_up(r, page)]:
            refs[p] -= 1
    for f, d, r in zip(src, dst, rows):
        if r % page:
            frm, to = table[f][r // page], refs.index(0)
            refs[to] = 1
            for pool, scale in pools.values():
                pool[to, :r % page] = pool[frm, :r % page]
                if scale is not None:
                    scale[to] = scale[frm]
    out = {"table": None, "refs": None, "copies": None, "k": pools["k"][0], "v": pools["v"][0]}
    if c["kv"] == "e4m3":
        out["k_scale"], out["v_scale"] = pools["k"][1], pools["v"][1]
    return out
