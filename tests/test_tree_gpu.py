"""GPU: drafted trees over a paged cache against the 64-bit restatement in tree_reference.py: rules from
parents, the append at a tree's depths, attention of its nodes (held to the element-wise bound that the reference
derives from the inputs), the rows that are kept, and all of them together as a step of decoding uses them."""
import math

import numpy as np
import pytest

import paged_reference as ref
import tree_reference as tree
from test_paged_gpu import Pool, check, pkg, tt        # noqa: F401  (pkg is the fixture)

pytestmark = pytest.mark.gpu


def dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def make_parents(rng, n, wide=8):
    """Each node hangs on one of the `wide` before it, or on the sequence."""
    return np.array([-1 if t == 0 else rng.integers(max(-1, t - wide), t) for t in range(n)], np.int32).reshape(-1)


def flat(xs, dt=np.int32):
    return np.concatenate([np.asarray(x, dt).reshape(-1) for x in xs] or [np.zeros(0, dt)]).astype(dt)


def setup(seed, nodes, n_words, wide=8):
    rng = np.random.default_rng(seed)
    parents = [make_parents(rng, n, wide) for n in nodes]
    sees, depths = [], []
    for p in parents:
        a, b, _ = tree.rules(p)
        sees.append(a)
        depths.append(b)
    mask = np.concatenate([tree.words(s, n_words) for s in sees] + [np.zeros((0, n_words), np.int32)])
    return parents, sees, depths, mask


def vmax_of(pool, v):
    """What a weight's smallest step may multiply, for each sequence: the largest |v|, for 8 bits 448 of the largest
    page scale."""
    if pool.kv != "e4m3":
        return [max(np.nanmax(np.abs(x), initial=0.0), 1e-30) for x in v]
    return [448.0 * pool.scale[1].max()] * len(v)


def tree_check(pkg, pool, nodes, n_head, src="f32", seed=1, splits=(0,), pad=0, chain=False, masks=None, extra_words=0,
               ctx=None, positions=None, q=None, wide=8, most=None, what="", **rules):
    import torch
    rng = np.random.default_rng(seed)
    hd = pool.host[0].shape[3]
    most = most or max(max(nodes), 1)
    n_words = -(-most // 32) + extra_words
    t = sum(nodes)
    parents, sees, depths, mask = setup(seed, nodes, n_words, wide)
    if masks is not None:                                     # any bits
        sees = masks
        mask = np.concatenate([tree.words(s, n_words) for s in sees])
    if chain:
        sees = [[list(range(i + 1)) for i in range(n)] for n in nodes]
        depths = [list(range(n)) for n in nodes]
    if q is None:
        q = rng.standard_normal((t + pad, n_head, hd)).astype(np.float32)
    dq = tt(q).to(dtype(src))
    q = dq.double().cpu().numpy()
    host, dev = dict(rules), dict(rules)
    if rules.get("slopes") is not None:
        host["slopes"] = np.asarray(rules["slopes"], np.float32)
        dev["slopes"] = tt(host["slopes"])
    if rules.get("starts") is not None:
        dev["starts"] = tt(np.asarray(rules["starts"], np.int32))
    pos = np.asarray(positions if positions is not None else [c - 1 for c in pool.ctx], np.int32)
    cu = np.cumsum([0] + list(nodes)).astype(np.int32)
    k, v = pool.rows(0, ctx), pool.rows(1, ctx)
    want, bound = tree.attend([q[cu[s]:cu[s + 1]] for s in range(len(nodes))], sees, depths, k, v, hd ** -0.5, pool.kv,
                              src, vmax=vmax_of(pool, v), **host)
    out = None
    for P in splits:
        out = torch.full((t + pad, n_head, hd), -7.0, device="cuda", dtype=dq.dtype)
        m = np.concatenate([mask, np.full((pad, n_words), -1, np.int32)])
        d = np.concatenate([flat(depths), np.full(pad, 5, np.int32)])
        pkg.tree_decode_attention(pool.cache(pkg), tt(pool.table), tt(pos), dq, mask=None if chain else tt(m),
                                  depths=None if chain else tt(d), cu_tokens=tt(cu), max_nodes=most, out=out,
                                  n_splits=P, **dev)
        if t:
            check(out[:t], np.concatenate(want), np.concatenate(bound), "%s P=%d" % (what, P))
        assert bool((out[t:] == -7.0).all())
    return out


# ---------------------------------------------------------------------------
# Rules from parents.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("nodes,most", [((1,), 1), ((5, 1, 0, 31, 32, 33), 33), ((64, 65, 100), 128), ((257, 1024), 1024),
                                        ((3,) * 700, 7)])
def test_rules_from_parents(pkg, nodes, most):
    n_words = -(-most // 32)
    parents, sees, depths, mask = setup(sum(nodes), nodes, n_words)
    cu = tt(np.cumsum([0] + list(nodes)).astype(np.int32))
    pad = 3
    import torch
    m = torch.full((sum(nodes) + pad, n_words), 9, dtype=torch.int32, device="cuda")
    d = torch.full((sum(nodes) + pad,), 9, dtype=torch.int32, device="cuda")
    pkg.tree_rules(tt(np.concatenate([flat(parents), np.full(pad, 77, np.int32)])), cu_tokens=cu, max_nodes=most, mask=m,
                   depths=d)
    t = sum(nodes)
    np.testing.assert_array_equal(m[:t].cpu().numpy(), mask)
    np.testing.assert_array_equal(d[:t].cpu().numpy(), flat(depths))
    assert bool((m[t:] == 9).all()) and bool((d[t:] == 9).all())
    if len(set(nodes)) == 1:
        m2, d2 = pkg.tree_rules(tt(np.stack(parents)), max_nodes=most)
        assert torch.equal(m2, m[:t]) and torch.equal(d2, d[:t])
    assert pkg.attn_read_device_error() == 0


def test_parents_in_any_order_and_wrong_ones(pkg):
    good = [3, 0, 3, -5, 1]
    m, d = pkg.tree_rules(tt(np.int32([good])))
    sees, depths, wrong = tree.rules(good)
    assert not wrong
    np.testing.assert_array_equal(m.cpu().numpy(), tree.words(sees, 1))
    assert d.tolist() == depths and pkg.attn_read_device_error() == 0
    for bad in ([0, 5, -1, 1, 2], [1, 2, 0, 3, -1], [2 ** 31 - 1, -2 ** 31, 0, 0, 0]):
        m, d = pkg.tree_rules(tt(np.int32([bad])))
        sees, depths, wrong = tree.rules(bad)
        assert wrong
        np.testing.assert_array_equal(m.cpu().numpy(), tree.words(sees, 1))
        assert d.tolist() == depths and pkg.attn_read_device_error() == pkg.ATTN_DEVERR_BAD_REQUEST
    # more nodes than max_nodes: left alone
    import torch
    m, d = torch.full((5, 1), 7, dtype=torch.int32, device="cuda"), torch.full((5,), 7, dtype=torch.int32, device="cuda")
    pkg.tree_rules(tt(np.int32(good)), cu_tokens=tt(np.int32([0, 5])), max_nodes=4, mask=m, depths=d)
    assert bool((m == 7).all()) and pkg.attn_read_device_error() == pkg.ATTN_DEVERR_BAD_REQUEST


# ---------------------------------------------------------------------------
# Attention.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group,page", [(1, 16), (5, 48), (8, 64)])
def test_attention_of_trees(pkg, kv, hd, src, group, page):
    ctx = (1, 2, 16, 17, 40, 64, 65, 127, 128, 129, 260)
    nodes = (1, 2, 7, 1, 33, 16, 20, 5, 12, 40, 9)
    pool = Pool(hd + group, kv, 2, hd, page, ctx)
    tree_check(pkg, pool, nodes, 2 * group, src, splits=(0, 1, 5), what="%s %d %s" % (kv, hd, src))
    assert pkg.attn_read_device_error() == 0


@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("hd,n,group,ctx", [(128, 64, 7, 700), (64, 130, 3, 515), (256, 33, 8, 400), (128, 1, 1, 2000),
                                            (128, 300, 1, 333), (64, 1, 64, 900), (256, 129, 2, 1111), (128, 1024, 1, 1100)])
def test_trees_of_many_sizes(pkg, kv, hd, n, group, ctx):
    pool = Pool(n, kv, 1, hd, 64, (ctx,))
    src = {"e4m3": "f32", "f16": "bf16", "bf16": "f32"}[kv]
    tree_check(pkg, pool, (n,), group, src, splits=(0, 3), what="%s %d" % (kv, hd))


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("rules", [{}, dict(softcap=30.0, window=300), dict(slopes=[0.01, 0.5, 0.1, 0.02, 0.3, 1.0])])
def test_weights_carry_more_bits_than_a_result_of_the_caches_type(pkg, monkeypatch, kv, hd, rules):
    """Queries of a 16-bit cache's type: the bound for weights in two parts."""
    monkeypatch.setattr(tree, "parts_of", lambda a, b: (1, 2, kv))
    pool = Pool(27, kv, 2, hd, 32, (2, 40, 129, 700, 1300, 260))
    tree_check(pkg, pool, (2, 7, 1, 33, 20, 5), 6, kv, splits=(0, 1, 3), **rules)


@pytest.mark.parametrize("kv,hd,src", [("e4m3", 128, "f32"), ("f16", 64, "f16"), ("bf16", 256, "bf16"), ("e4m3", 128, "bf16")])
def test_chains_and_a_padded_batch(pkg, kv, hd, src):
    pool = Pool(5, kv, 2, hd, 32, (0, 5, 70, 300, 133))
    nodes = (0, 5, 3, 60, 1)
    tree_check(pkg, pool, nodes, 6, src, chain=True, pad=5)
    tree_check(pkg, pool, nodes, 6, src, pad=5, most=200, extra_words=2)
    tree_check(pkg, pool, nodes, 6, src, pad=0, most=1024)


def test_a_chain_is_paged_decode_attention(pkg):
    pool = Pool(6, "e4m3", 2, 128, 64, (300, 77, 128))
    rng = np.random.default_rng(3)
    q = tt(rng.standard_normal((3, 6, 8, 128)).astype(np.float32))
    table, pos = tt(pool.table), tt(np.int32([299, 76, 127]))
    a = pkg.tree_decode_attention(pool.cache(pkg), table, pos, q)
    b = pkg.paged_decode_attention(pool.cache(pkg), table, pos, q)
    assert a.shape == q.shape and float((a - b).abs().max()) < 1e-5 * float(b.abs().max())


RULES = [dict(softcap=20.0), dict(window=50), dict(window=3), dict(slopes=True), dict(starts=True),
         dict(softcap=5.0, slopes=True, window=100, starts=True)]


@pytest.mark.parametrize("kv,hd,src", [("e4m3", 128, "f32"), ("f16", 64, "f32"), ("bf16", 256, "f32"), ("f16", 128, "f16"),
                                       ("bf16", 128, "bf16"), ("e4m3", 256, "f32")])
@pytest.mark.parametrize("rules", RULES)
@pytest.mark.parametrize("group", [3, 8])
def test_score_rules(pkg, kv, hd, src, rules, group):
    ctx, nodes = (20, 40, 130, 300, 260), (20, 7, 33, 50, 12)
    pool = Pool(8, kv, 2, hd, 32, ctx)
    r = dict(rules)
    if r.pop("slopes", None):
        r["slopes"] = 2.0 ** (-8.0 * np.arange(1, 2 * group + 1) / (2 * group))
    if r.pop("starts", None):
        r["starts"] = [3, -5, 129, 17, 256]                     # 129: the last node alone sees itself
    tree_check(pkg, pool, nodes, 2 * group, src, splits=(0, 3), **r)
    tree_check(pkg, pool, nodes, 2 * group, src, chain=True, **r)


@pytest.mark.parametrize("kv,hd", [("e4m3", 128), ("f16", 64), ("bf16", 256)])
def test_windows_and_nodes_deeper_than_the_capacity(pkg, kv, hd):
    """A node's position may lie past the cache's last row, so a window longer than the cache can mask some of it."""
    import torch
    pool = Pool(24, kv, 1, hd, 16, (64, 50))                      # 64 rows of capacity
    depths = [[0, 70, 1023, 7], [5, 900, 33]]
    sees = [[[0], [0, 1], [0, 1, 2], [3, 0]], [[0], [1, 0], [0, 2]]]
    mask = np.concatenate([tree.words(s, 32) for s in sees])
    cu = np.int32([0, 4, 7])
    q = tt(np.random.default_rng(3).standard_normal((7, 4, hd)).astype(np.float32))
    qh = q.double().cpu().numpy()
    k, v = pool.rows(0), pool.rows(1)
    for window in (64, 65, 66, 90, 1000, 1064, 1083, 1084, 1087, 1088, 2 ** 31 - 1):
        want, bound = tree.attend([qh[:4], qh[4:]], sees, depths, k, v, hd ** -0.5, kv, "f32", vmax=vmax_of(pool, v),
                                  window=window)
        for P in (1, 2):
            out = pkg.tree_decode_attention(pool.cache(pkg), tt(pool.table), tt(np.int32([63, 49])), q, mask=tt(mask),
                                            depths=tt(flat(depths)), cu_tokens=tt(cu), max_nodes=1024, window=window, n_splits=P)
            check(out, np.concatenate(want), np.concatenate(bound), "window %d" % window)


@pytest.mark.parametrize("kv,hd", [("e4m3", 128), ("f16", 64), ("bf16", 256)])
def test_starts_before_the_first_row_mask_nothing(pkg, kv, hd):
    """Down to the smallest 32-bit number, as one may write where there is no start."""
    import torch
    ctx, nodes = (700, 300, 40, 515), (20, 33, 12, 7)
    pool = Pool(23, kv, 2, hd, 32, ctx)
    parents, sees, depths, mask = setup(4, nodes, 2)
    rng = np.random.default_rng(2)
    q = tt(rng.standard_normal((sum(nodes), 6, hd)).astype(np.float32))
    a = [pool.cache(pkg), tt(pool.table), tt(np.int32(ctx) - 1), q]
    cu = tt(np.cumsum((0,) + nodes).astype(np.int32))
    for kw in (dict(mask=tt(mask), depths=tt(flat(depths))), {}):
        kw.update(cu_tokens=cu, max_nodes=33, n_splits=3)
        plain = pkg.tree_decode_attention(*a, **kw)
        for starts in ([-1] * 4, [-2 ** 31] * 4, [-2 ** 31 + 1, -2 ** 31 + 600, -2 ** 30, 0]):
            assert torch.equal(pkg.tree_decode_attention(*a, starts=tt(np.int32(starts)), **kw), plain)


@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
def test_masks_of_any_bits_and_rows_that_see_nothing(pkg, kv, src):
    """Masks that are no tree's; with starts past the context some rows see nothing: 0."""
    rng = np.random.default_rng(4)
    ctx, nodes = (150, 64, 9, 130), (40, 33, 9, 1)
    masks = [[sorted(rng.choice(n, rng.integers(0, n + 1), replace=False).tolist()) for _ in range(n)] for n in nodes]
    masks[0][3] = masks[1][0] = masks[2][8] = masks[3][0] = []
    masks[0][5] = [0]                                             # not itself
    pool = Pool(12, kv, 2, 128, 16, ctx)
    tree_check(pkg, pool, nodes, 8, src, masks=masks)
    out = tree_check(pkg, pool, nodes, 8, src, masks=masks, starts=[110, 31, 0, 130])
    cu = np.cumsum((0,) + nodes)
    for t in (3, cu[1], cu[2] + 8, cu[3]):
        assert bool((out[t] == 0).all())


@pytest.mark.parametrize("src", ["f32", "f16"])
@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_unseen_infinities_and_nan(pkg, kv, src, hd):
    """A node's row may hold anything for the nodes that do not see it, a row in front of starts or behind a
    window for those that do not; whoever sees it gets NaN or infinity there, and only in the dimensions that
    hold it."""
    import torch
    n, ctx = 20, 150
    pool = Pool(11, kv, 1, hd, 16, (ctx,))
    rng = np.random.default_rng(2)
    parents, sees, depths, mask = setup(9, (n,), 1)
    bad, front = [ctx - n + 4, ctx - n + 11], 37
    for row in bad + [front]:
        p, o = int(pool.table[0, row // 16]), row % 16
        for i in range(2):
            if row == bad[1] and i == 0:
                continue
            d = pool.dev[i].view(torch.uint8) if kv == "e4m3" else pool.dev[i]
            at = slice(None) if row != bad[1] else slice(3, 5)
            d[p, o, :, at] = 0x7F if kv == "e4m3" else math.inf if (i and row != front) else math.nan
    q = tt(rng.standard_normal((n, 4, hd)).astype(np.float32)).to(dtype(src))
    k, v = pool.rows(0), pool.rows(1)
    for row in bad + [front]:
        k[0][row], v[0][row] = 0.0, 0.0
    kw = dict(starts=[front + 1])
    want, bound = tree.attend([q.double().cpu().numpy()], sees, depths, k, v, hd ** -0.5, kv, src,
                              vmax=vmax_of(pool, v), **kw)
    for P in (0, 1, 2):
        out = pkg.tree_decode_attention(pool.cache(pkg), tt(pool.table), tt(np.int32([ctx - 1])), q, mask=tt(mask),
                                        depths=tt(flat(depths)), starts=tt(np.int32([front + 1])), n_splits=P)
        clean = [t for t in range(n) if not {4, 11} & set(sees[0][t])]
        assert len(clean) > 3
        check(out[clean], want[0][clean], bound[0][clean], kv)
        for t in range(n):
            if 4 in sees[0][t]:
                assert not bool(out[t].isfinite().any())
            elif 11 in sees[0][t]:
                assert not bool(out[t, :, 3:5].isfinite().any())
                assert bool(out[t, :, 5:].isfinite().all()) and bool(out[t, :, :3].isfinite().all())
    # a window that hides the row from all but the shallow nodes
    out = pkg.tree_decode_attention(pool.cache(pkg), tt(pool.table), tt(np.int32([ctx - 1])), q, mask=tt(mask),
                                    depths=tt(flat(depths)), window=ctx - n - front + 2)
    for t in range(n):
        if not {4, 11} & set(sees[0][t]):
            assert bool(out[t].isfinite().all()) == (depths[0][t] >= 2), (t, depths[0][t])


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_infinities_and_nan_in_v_alone(pkg, kv, src, hd):
    """K is finite, V is not in some dimensions of two nodes and of a row beside `starts`: those dimensions of the nodes
    that see them, and nothing else, with equal bits from every run. Over many tiles, as parts and as a whole."""
    import torch
    ctx, nodes, n_head, n_words = (1300, 37, 2100), (20, 9, 33), 8, 2
    pool = Pool(21, kv, 2, hd, 32, ctx)
    parents, sees, depths, mask = setup(9, nodes, n_words)
    rng = np.random.default_rng(3)
    starts = [5, 0, 900]
    put = [(0, 1280 + 4, 3, 5), (0, 1280 + 11, hd - 1, hd), (1, 28 + 2, 8, 9), (2, 2067 + 13, 0, 2), (2, 900, 30, 34)]
    k, v = pool.rows(0), pool.rows(1)
    for i, (s, row, d0, d1) in enumerate(put):
        p, o = int(pool.table[s, row // 32]), row % 32
        d = pool.dev[1].view(torch.uint8) if kv == "e4m3" else pool.dev[1]
        d[p, o, :, d0:d1] = 0x7F if kv == "e4m3" else (math.nan if i == 1 else math.inf)
        v[s][row, :, d0:d1] = 0.0
    t, cu = sum(nodes), np.cumsum((0,) + nodes)
    wild = np.zeros((t, hd), bool)                                # what cannot be finite
    for s, row, d0, d1 in put:
        y = row - (ctx[s] - nodes[s])
        who = [cu[s] + x for x in range(nodes[s]) if y < 0 or y in sees[s][x]]
        assert who
        wild[who, d0:d1] = True
    for s, row, d0, d1 in put[:4]:                                # nobody sees all of them, some see one alone
        assert not wild[cu[s]:cu[s + 1], d0].all()
    q = tt(rng.standard_normal((t, n_head, hd)).astype(np.float32)).to(dtype(src))
    qh = q.double().cpu().numpy()
    want, bound = (np.concatenate(x) for x in tree.attend(
        [qh[cu[s]:cu[s + 1]] for s in range(3)], sees, depths, k, v, hd ** -0.5, kv, src, vmax=vmax_of(pool, v), starts=starts))
    a = [pool.cache(pkg), tt(pool.table), tt(np.int32(ctx) - 1), q]
    kw = dict(mask=tt(mask), depths=tt(flat(depths)), cu_tokens=tt(cu.astype(np.int32)), max_nodes=max(nodes),
              starts=tt(np.int32(starts)))
    bits = torch.int32 if src == "f32" else torch.int16
    there = tt(wild)[:, None, :].expand(t, n_head, hd)
    pkg.attn_read_device_error()
    for P in (1, 0, 2, 7):
        first = pkg.tree_decode_attention(*a, n_splits=P, **kw)
        assert bool((first.isfinite() == ~there).all())
        check(torch.where(there, torch.zeros_like(first), first), np.where(wild[:, None], 0.0, want), bound, "P=%d" % P)
        for _ in range(10):
            assert torch.equal(pkg.tree_decode_attention(*a, n_splits=P, **kw).view(bits), first.view(bits))
    assert pkg.attn_read_device_error() == 0


@pytest.mark.parametrize("kv", ["e4m3", "f16"])
def test_pages_that_are_not_there(pkg, kv):
    pool = Pool(9, kv, 2, 128, 32, (200, 70, 40))
    pool.table[0, 2] = -1
    pool.table[1, 2] = pool.n_pages
    pool.table[2, 0] = pool.table[2, 1] = -7
    pkg.attn_read_device_error()
    tree_check(pkg, pool, (20, 9, 5), 8, splits=(0, 1, 4))
    assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_BAD_PAGE


def test_positions_and_counts_out_of_range(pkg):
    import torch
    pool = Pool(10, "f16", 1, 64, 16, (48, 48, 3, 10, 20))
    # past the capacity: clamped; below -1: no rows; fewer rows than nodes; more nodes than max_nodes
    pkg.attn_read_device_error()
    nodes, pos = (5, 4, 7, 3, 12), [50, -9, 2, 9, 19]
    cu = np.cumsum((0,) + nodes).astype(np.int32)
    parents, sees, depths, mask = setup(3, nodes, 1)
    rng = np.random.default_rng(1)
    q = tt(rng.standard_normal((31, 2, 64)).astype(np.float32))
    out = torch.full_like(q, -7.0)
    pkg.tree_decode_attention(pool.cache(pkg), tt(pool.table), tt(np.int32(pos)), q, mask=tt(mask), depths=tt(flat(depths)),
                              cu_tokens=tt(cu), max_nodes=7, out=out)
    assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_POSITION_CLAMPED | pkg.ATTN_DEVERR_BAD_REQUEST
    cut = [48, 0, 3, 10, 20]
    k, v = pool.rows(0, cut), pool.rows(1, cut)
    want, bound = tree.attend([q[cu[s]:cu[s + 1]].double().cpu().numpy() for s in range(4)], sees, depths, k, v, 0.125,
                              "f16", "f32")
    check(out[:cu[4]], np.concatenate(want[:4]), np.concatenate(bound[:4]), "")
    assert bool((out[cu[4]:] == -7.0).all())


@pytest.mark.parametrize("order", ["heads", "joint"])
@pytest.mark.parametrize("kv,hd", [("e4m3", 64), ("e4m3", 256), ("f16", 128)])
def test_other_orders_and_parts_of_an_allocation(pkg, order, kv, hd):
    pool = Pool(13, kv, 3, hd, 48, (100, 230), order=order)
    tree_check(pkg, pool, (20, 50), 6, "f32", splits=(0, 2))


def test_scales_of_any_size(pkg):
    """Page scales from 2^-60 to 2^60, 0 and negative ones."""
    pool = Pool(14, "e4m3", 1, 128, 16, (160, 160))
    rng = np.random.default_rng(5)
    sc = 2.0 ** rng.integers(-10, 3, (pool.n_pages, 1)).astype(np.float64)
    ks = np.where(rng.random((pool.n_pages, 1)) < 0.3, -0.003, 0.005)
    sc[pool.table[0, 3]] = 2.0 ** 60
    sc[pool.table[1, 2]] = 0.0
    sc[pool.table[1, 3]] = -0.7
    sc[pool.table[1, 4]] = 2.0 ** -60
    pool.scale = [ks, sc]
    pool.dscale = [tt(ks.astype(np.float32)), tt(sc.astype(np.float32))]
    pool.scale = [x.double().cpu().numpy() for x in pool.dscale]
    for src in ("f32", "bf16"):
        tree_check(pkg, pool, (20, 31), 4, src, splits=(0, 1, 3))


def test_more_sequences_than_a_launch_takes(pkg):
    rng = np.random.default_rng(7)
    ctx = rng.integers(1, 60, 300)
    nodes = [int(rng.integers(0, min(c, 9) + 1)) for c in ctx]
    pool = Pool(15, "bf16", 1, 64, 16, ctx)
    tree_check(pkg, pool, nodes, 3, "f32")


@pytest.mark.parametrize("kv,hd,src,n_kv,group", [("f16", 64, "f16", 2, 2), ("bf16", 128, "f32", 3, 4), ("e4m3", 256, "f32", 1, 1),
                                                  ("e4m3", 128, "bf16", 2, 40)])
def test_blocks_that_cross_many_sequences(pkg, kv, hd, src, n_kv, group):
    rng = np.random.default_rng(8)
    ctx = rng.integers(4, 500, 40)
    nodes = [int(rng.integers(0, 5)) if i % 7 else 0 for i in range(40)]
    pool = Pool(16, kv, n_kv, hd, 32, ctx)
    tree_check(pkg, pool, nodes, n_kv * group, src, splits=(0, 1, 2, 3, 7, 61))


def test_four_rounds_of_blocks(pkg):
    """Units just over half of the SMs: with a block an SM almost half would have none, so that each unit's tiles are shared
    by as many blocks as make four rounds."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n_kv, group = 8, 8
    units = sms // 2 // n_kv * n_kv + n_kv
    nodes = (units // n_kv) * 128 // group
    pool = Pool(26, "f16", n_kv, 64, 64, (1700, 900, 300))
    P = pkg.attn_tree_plan(pool.cache(pkg), pool.max_pages, 3, nodes + 4, nodes, pkg.ATTN_TYPE_BF16, n_kv * group)[0]
    assert P == 4 * sms // units and P * units > 3 * sms
    tree_check(pkg, pool, (nodes, 1, 3), n_kv * group, "bf16", splits=(0,))


def test_long_context(pkg):
    """A long cache: rows by a plain 64-bit form on the GPU."""
    import torch
    for kv, ctx in (("e4m3", 40007), ("bf16", 33000)):
        dt = torch.float8_e4m3fn if kv == "e4m3" else torch.bfloat16
        n_pages = -(-ctx // 64) + 1
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        pools = []
        for _ in range(2):
            x = torch.randn(n_pages, 64, 2, 128, device="cuda", generator=g)
            pools.append(x.to(dt))
        one = torch.ones(n_pages, 2, device="cuda") if kv == "e4m3" else None
        ids = torch.randperm(n_pages, device="cuda", generator=g)[:-(-ctx // 64)].int()
        n = 30
        parents, sees, depths, mask = setup(3, (n,), 1)
        q = torch.randn(n, 8, 128, device="cuda", generator=g)
        out = pkg.tree_decode_attention(pkg.PagedCache(*pools, one, one), ids[None].contiguous(),
                                        tt(np.int32([ctx - 1])), q, mask=tt(mask), depths=tt(flat(depths)))
        k, v = (p[ids.long()].double().reshape(-1, 2, 128)[:ctx] for p in pools)
        ok = torch.ones(n, ctx, dtype=torch.bool, device="cuda")
        ok[:, ctx - n:] = False
        for t in range(n):
            ok[t, [ctx - n + y for y in sees[0][t]]] = True
        s = torch.einsum("tkgd,nkd->tkgn", q.double().view(n, 2, 4, 128), k) / math.sqrt(128)
        p = torch.softmax(torch.where(ok[:, None, None], s, -math.inf), -1)
        want = torch.einsum("tkgn,nkd->tkgd", p, v).reshape(n, 8, 128)
        # 16 bits of q and weights (2^-16 of a score of magnitude up to 50, of a weight) over bf16, 22 else; averages over
        # some 10^4 rows of random sign stay far below the sum of magnitudes
        tol = 2e-5 if kv == "e4m3" else 2e-4
        assert float((out - want).norm() / want.norm()) < tol


@pytest.mark.parametrize("kv,hd", [("e4m3", 128), ("f16", 64), ("f16", 256), ("bf16", 128), ("e4m3", 256)])
@pytest.mark.parametrize("P", [1, 2, 5])
def test_long_runs_of_one_block_keep_their_bits(pkg, kv, hd, P):
    """Rows are added up on the tensor cores, which cut a sum off at 24 bits at each step (16 rows of a part): half a unit of
    2^-23 .. 2^-24 of it on average, always towards 0. Over 2048 rows these are 256 steps, in which a sum of terms of random sign
    grows as the square root: 256 * 2 / 3 * 2^-24 = 1.0e-5 of the result. Beside it 1e-6, or 5e-6 for the 16 bits of q and
    weights over bf16."""
    import torch
    n_seq, n_kv, n, ctx, page = 3, 2, 6, 30011, 64
    per = -(-ctx // page)
    rng = np.random.default_rng(3)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    dt = torch.float8_e4m3fn if kv == "e4m3" else dtype(kv)
    pools = [torch.randn(n_seq * per, page, n_kv, hd, device="cuda", generator=g).to(dt) for _ in range(2)]
    one = [torch.ones(n_seq * per, n_kv, device="cuda")] * 2 if kv == "e4m3" else []
    table = tt(rng.permutation(n_seq * per).astype(np.int32).reshape(n_seq, per))
    q = torch.randn(n_seq, n, 3 * n_kv, hd, device="cuda", generator=g)
    pos = np.int32([ctx - 1, 2000, 17000])
    out = pkg.tree_decode_attention(pkg.PagedCache(*pools, *one), table, tt(pos), q, n_splits=P)
    for s in range(n_seq):
        rows = int(pos[s]) + 1
        k, v = (p[table[s].long()].double().reshape(-1, n_kv, hd)[:rows] for p in pools)
        ok = torch.arange(rows, device="cuda")[None] <= rows - n + torch.arange(n, device="cuda")[:, None]
        sc = torch.einsum("tkgd,nkd->tkgn", q[s].double().view(n, n_kv, 3, hd), k) / math.sqrt(hd)
        p = torch.softmax(torch.where(ok[:, None, None], sc, -math.inf), -1)
        want = torch.einsum("tkgn,nkd->tkgd", p, v).reshape(n, 3 * n_kv, hd)
        off = float((out[s] - want).norm() / want.norm())
        assert off < 1.0e-5 + (5e-6 if kv == "bf16" else 1e-6), (s, off)


def test_a_block_may_take_seconds(pkg):
    """One block over 2^27 rows (1.6 s; pages that stand in the table many times): warps without a slot wait longer than a wait
    may take otherwise. Each row has its weight 2^14 times, so that the result is the one of 2^13 rows; 2^22 additions to a
    32-bit sum of weights, each off by 2^-24 at most, may leave a quarter of it."""
    import torch
    page, n_pages, hd = 1024, 8, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    k, v = (torch.randn(n_pages, page, 1, hd, device="cuda", generator=g).to(torch.float8_e4m3fn) for _ in range(2))
    one = torch.ones(n_pages, 1, device="cuda")
    table = torch.arange(2 ** 17, device="cuda", dtype=torch.int32)[None] % n_pages
    q = torch.randn(1, 1, hd, device="cuda", generator=g)
    pkg.attn_read_device_error()
    out = pkg.tree_decode_attention(pkg.PagedCache(k, v, one, one), table, tt(np.int32([2 ** 27 - 1])), q, n_splits=1)
    assert pkg.attn_read_device_error() == 0
    sc = k.double().reshape(-1, hd) @ q[0, 0].double() / math.sqrt(hd)
    want = torch.softmax(sc, 0) @ v.double().reshape(-1, hd)
    assert float((out[0, 0] - want).norm() / want.norm()) < 0.25


@pytest.mark.parametrize("kv,hd,page", [("e4m3", 128, 64), ("e4m3", 64, 48), ("f16", 256, 128), ("bf16", 128, 16), ("e4m3", 256, 32)])
def test_runs_of_many_tiles(pkg, kv, hd, page):
    """Sums that are put by and taken up again, at references that move (page scales, slopes), in sequences that a block has all
    of and in parts, with infinities among them."""
    ctx, nodes = (7003, 40, 5200, 2049, 4100), (7, 9, 3, 1, 20)
    pool = Pool(28, kv, 1, hd, page, ctx)
    for splits in ((1, 2), (3, 7)):
        tree_check(pkg, pool, nodes, 3, "f32", splits=splits)
    tree_check(pkg, pool, nodes, 3, "f32", splits=(1, 3), slopes=[0.05, 0.002, -0.004], starts=[3000, 0, 17, 1, 2047])
    if kv == "bf16":
        tree_check(pkg, pool, nodes, 3, "f16", splits=(1, 2))


@pytest.mark.parametrize("kv,hd,nodes", [("bf16", 64, 9), ("f16", 128, 5), ("e4m3", 128, 16), ("bf16", 256, 20)])
def test_many_runs_over_many_tiles(pkg, kv, hd, nodes):
    """Warps that are late or early where one sequence ends and the next begins: equal bits from every run, and no wait
    that gave up. Two KV heads, groups of 7: one or two units, some warps of them without a row."""
    import torch
    rng = np.random.default_rng(hd)
    n_seq, page, ctx = 5, 64, 2048
    per = ctx // page
    shape = (n_seq * per, page, 2, hd)
    vals = [rng.standard_normal(shape).astype(np.float32) for _ in range(2)]
    k, v = (tt(x).to(torch.float8_e4m3fn if kv == "e4m3" else dtype(kv)) for x in vals)
    scales = [torch.ones((n_seq * per, 2), device="cuda") for _ in range(2)] if kv == "e4m3" else []
    cache = pkg.PagedCache(k, v, *scales)
    table = tt(rng.permutation(n_seq * per).astype(np.int32).reshape(n_seq, per))
    pos = tt(np.int32([ctx - 1, 700, 100, ctx - 130, 1291]))
    q = tt(rng.standard_normal((n_seq * nodes, 14, hd)).astype(np.float32)).to(dtype("bf16" if kv == "bf16" else "f16"))
    pkg.attn_read_device_error()
    first = pkg.tree_decode_attention(cache, table, pos, q, n_splits=3)
    for _ in range(60):
        assert torch.equal(pkg.tree_decode_attention(cache, table, pos, q, n_splits=3), first)
    assert pkg.attn_read_device_error() == 0


def test_two_calls_at_once(pkg):
    """On two streams, each with its own trees over one cache: the bits of the calls alone."""
    import torch
    rng = np.random.default_rng(5)
    n_seq, page, per = 4, 32, 40
    shape = (n_seq * per, page, 2, 128)
    k, v = (tt(rng.standard_normal(shape).astype(np.float32)).half() for _ in range(2))
    cache = pkg.PagedCache(k, v)
    table = tt(rng.permutation(n_seq * per).astype(np.int32).reshape(n_seq, per))
    calls = [(tt(np.int32(p)), tt(rng.standard_normal((n_seq, n, 8, 128)).astype(np.float32)).half())
             for p, n in (([1279, 500, 64, 900], 6), ([1000, 31, 1200, 77], 30))]
    alone = [pkg.tree_decode_attention(cache, table, p, q) for p, q in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(20):
        for i, (p, q) in enumerate(calls):
            with torch.cuda.stream(streams[i]):
                got[i].append(pkg.tree_decode_attention(cache, table, p, q))
    torch.cuda.synchronize()
    for want, outs in zip(alone, got):
        assert all(torch.equal(x, want) for x in outs)
    assert pkg.attn_read_device_error() == 0


def test_a_query_of_nan_stays_alone(pkg):
    import torch
    for src in ("f32", "f16"):
        pool = Pool(17, "f16", 1, 128, 16, (140,))
        rng = np.random.default_rng(1)
        q = rng.standard_normal((10, 2, 128)).astype(np.float32)
        parents, sees, depths, mask = setup(3, (10,), 1)
        a = [tt(pool.table), tt(np.int32([139]))]
        kw = dict(mask=tt(mask), depths=tt(flat(depths)))
        clean = pkg.tree_decode_attention(pool.cache(pkg), *a, tt(q).to(dtype(src)), **kw)
        q[3, 1] = math.nan
        q[5, 0, 7] = math.inf
        out = pkg.tree_decode_attention(pool.cache(pkg), *a, tt(q).to(dtype(src)), **kw)
        keep = torch.ones(10, 2, dtype=torch.bool, device="cuda")
        keep[3, 1] = keep[5, 0] = False
        assert torch.equal(out[keep], clean[keep])
        assert bool(out[3, 1].isnan().all()) and not bool(out[5, 0].isfinite().all())


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_queries_that_are_not_finite_give_nan(pkg, kv, src, hd):
    """Infinities of either sign and NaN, alone in a row: NaN in all of its dimensions whatever the signs of K (keys of one sign
    make every score +inf or -inf), 0 where it sees no row, and the bits of the call without them elsewhere. With a cap the
    rows of a warp decide together which of two forms of tanh they take, each within the reference's bound of the result: so
    the other rows differ by twice that at most."""
    import torch
    ctx, n = 300, 12
    pool = Pool(25, kv, 1, hd, 16, (ctx,))
    if kv == "e4m3":
        pool.dev[0].view(torch.uint8).bitwise_and_(0x7F)
    else:
        pool.dev[0].abs_()
    parents, sees, depths, mask = setup(3, (n,), 1)
    q = np.random.default_rng(1).standard_normal((n, 4, hd)).astype(np.float32)
    a = [pool.cache(pkg), tt(pool.table), tt(np.int32([ctx - 1]))]
    kw = dict(mask=tt(mask), depths=tt(flat(depths)))
    wild = q.copy()
    put = [(0, 0, 0, -math.inf), (1, 3, hd - 1, math.inf), (4, 1, 7, math.nan), (7, 0, 40, -math.inf), (7, 1, 41, math.inf),
           (11, 2, hd // 2, -math.inf)]
    keep = torch.ones(n, 4, dtype=torch.bool, device="cuda")
    for t, h, d, x in put:
        wild[t, h, d] = x
        keep[t, h] = False
    k, v = ([np.abs(x) if i == 0 else x for x in pool.rows(i)] for i in range(2))
    bound = tree.attend([tt(q).to(dtype(src)).double().cpu().numpy()], sees, depths, k, v, hd ** -0.5, kv, src,
                        vmax=vmax_of(pool, v), softcap=20.0)[1][0]
    for extra in ({}, dict(softcap=20.0), dict(slopes=tt(np.full(4, 0.01, np.float32))), dict(starts=tt(np.int32([ctx - 1])))):
        for P in (0, 1, 3):
            clean, out = (pkg.tree_decode_attention(*a, tt(x).to(dtype(src)), n_splits=P, **kw, **extra) for x in (q, wild))
            assert bool(clean.isfinite().all())
            if "softcap" in extra:
                off = (out.double() - clean.double()).abs().cpu().numpy()
                assert (off <= 2 * bound)[keep.cpu().numpy()].all()
            else:
                assert torch.equal(out[keep], clean[keep]), (P, extra)
            for t, h, _, _ in put:
                if "starts" not in extra or n - 1 in sees[0][t]:
                    assert bool(out[t, h].isnan().all()), (t, h, P, extra)
                else:
                    assert bool((out[t, h] == 0).all()), (t, h, P, extra)


def test_same_bits_again_from_any_workspace_and_in_graphs(pkg):
    import torch
    pool = Pool(18, "e4m3", 2, 128, 64, (900, 333, 40))
    nodes = (30, 12, 40)
    cu = np.cumsum((0,) + nodes).astype(np.int32)
    parents, sees, depths, mask = setup(3, nodes, 2)
    rng = np.random.default_rng(1)
    q = tt(rng.standard_normal((82, 8, 128)).astype(np.float32)).bfloat16()
    cache, table, pos = pool.cache(pkg), tt(pool.table), tt(np.int32([899, 332, 39]))
    dm, dd, dcu = tt(mask), tt(flat(depths)), tt(cu)

    def call(out=None):
        return pkg.tree_decode_attention(cache, table, pos, q, mask=dm, depths=dd, cu_tokens=dcu, max_nodes=40, out=out)
    first = call()
    assert all(torch.equal(call(), first) for _ in range(3))
    need = pkg.attn_tree_plan(cache, table.shape[1], 3, 82, 40, pkg.ATTN_TYPE_BF16, 8)
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((max(need[1], 256),), fill, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        pkg.attn_decode_tree(cache, table, table.shape[1], pos, dcu, 3, 82, 40, q, out, pkg.ATTN_TYPE_BF16, 8, 128 ** -0.5,
                             dm, 2, dd, workspace=ws)
        assert torch.equal(out, first)
    out = torch.empty_like(q)                                     # the library's own workspace
    pkg.attn_decode_tree(cache, table, table.shape[1], pos, dcu, 3, 82, 40, q, out, pkg.ATTN_TYPE_BF16, 8, 128 ** -0.5, dm, 2, dd)
    assert torch.equal(out, first)
    # two graphs, replayed on two streams while the positions change
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        o = torch.empty_like(q)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call(o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(o)
        outs.append(o)
        graphs.append(g)
    for shift in (0, 7):
        pos.copy_(tt(np.int32([899 - 9 * shift, 332 - shift, 39])))
        want = call()
        torch.cuda.synchronize()
        for _ in range(5):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("kv,hd", [("e4m3", 128), ("bf16", 64), ("f16", 256)])
@pytest.mark.parametrize("P", [1, 4])
def test_sums_on_the_way_in_any_workspace_and_in_graphs(pkg, kv, hd, P):
    """Float32 queries over more rows than one sum takes: equal bits from every run, from workspaces that held anything and the
    library's own, and from graphs on two streams at once; a workspace that is too small is refused, one of a split too."""
    import torch
    ctx, nodes = (9001, 300, 2177, 4500), (20, 1, 33, 7)
    pool = Pool(29, kv, 2, hd, 64, ctx)
    parents, sees, depths, mask = setup(3, nodes, 2)
    t, cu = sum(nodes), np.cumsum((0,) + nodes).astype(np.int32)
    q = tt(np.random.default_rng(1).standard_normal((t, 6, hd)).astype(np.float32))
    cache, table, pos = pool.cache(pkg), tt(pool.table), tt(np.int32(ctx) - 1)
    dm, dd, dcu = tt(mask), tt(flat(depths)), tt(cu)

    def call(out=None):
        return pkg.tree_decode_attention(cache, table, pos, q, mask=dm, depths=dd, cu_tokens=dcu, max_nodes=33, n_splits=P, out=out)
    pkg.attn_read_device_error()
    first = call()
    assert all(torch.equal(call(), first) for _ in range(30))
    shape = (cache, table, table.shape[1], pos, dcu, 4, t, 33, q)
    rest = (pkg.ATTN_TYPE_F32, 6, hd ** -0.5, dm, 2, dd)
    need = pkg.attn_tree_plan(cache, table.shape[1], 4, t, 33, pkg.ATTN_TYPE_F32, 6, P)[1]
    assert need > 0
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        pkg.attn_decode_tree(*shape, out, *rest, n_splits=P, workspace=ws, workspace_bytes=need)
        assert torch.equal(out, first)
        assert bool((ws[need:] == fill).all())
    with pytest.raises(pkg.AttnError) as e:
        pkg.attn_decode_tree(*shape, out, *rest, n_splits=P, workspace=ws, workspace_bytes=need - 256)
    assert e.value.status == pkg.ATTN_ERR_WORKSPACE
    out = torch.empty_like(q)
    pkg.attn_decode_tree(*shape, out, *rest, n_splits=P)          # the library's own
    assert torch.equal(out, first)
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        o = torch.empty_like(q)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call(o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(o)
        outs.append(o)
        graphs.append(g)
    for shift in (0, 2100):
        pos.copy_(tt(np.int32(ctx) - 1 - np.int32([shift, 0, 0, shift])))
        want = call()
        torch.cuda.synchronize()
        for _ in range(5):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    assert pkg.attn_read_device_error() == 0


# ---------------------------------------------------------------------------
# The append at a tree's depths.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("src,out", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_of_trees(pkg, kv, src, out, interleaved):
    import torch
    for hd, page, past, nodes in ((128, 32, (5, 31, 32, 0), (7, 40, 1, 33)), (64, 16, (100,), (64,)), (256, 64, (63, 2), (5, 90))):
        rng = np.random.default_rng(hd)
        parents, sees, depths, mask = setup(hd, nodes, 3)
        ctx, t, pad = [a + b for a, b in zip(past, nodes)], sum(nodes), 2
        pool = Pool(hd, kv, 2, hd, page, ctx)
        q, kn, vn = (tt(rng.standard_normal((t + pad, h, hd)).astype(np.float32)).to(dtype(src)) for h in (6, 2, 2))
        rope = pkg.Rope(hd, interleaved=interleaved)
        q_out = torch.full((t + pad, 6, hd), -7.0, device="cuda", dtype=dtype(out))
        dep = flat(depths)
        pkg.rope_append(pool.cache(pkg), tt(pool.table), tt(np.int32(ctx) - 1), kn, vn, q=q, q_out=q_out, rope=rope,
                        cu_tokens=tt(np.cumsum((0,) + nodes).astype(np.int32)),
                        depths=tt(np.concatenate([dep, np.full(pad, 3, np.int32)])))
        place = dep + np.repeat(past, nodes)
        freq = ref.frequencies(hd, 10000.0)

        def turned(x):
            return ref.rotate(x[:t].double().cpu().numpy(), place, freq, interleaved)

        def slack(x):                                             # as in test_paged_gpu.append_check
            return 3 * 2.0 ** -22 * np.abs(x[:t].double().cpu().numpy()).max(axis=-1, keepdims=True)
        want = turned(q)
        check(q_out[:t], want, slack(q) + tree.HALF[out] * np.abs(want) + 2.0 ** -25, "q")
        assert bool((q_out[t:] == -7.0).all())
        for i, rows, sl in ((0, turned(kn), slack(kn)), (1, vn[:t].double().cpu().numpy(), 0 * slack(vn))):
            host, scale = pool.host[i].copy(), None if kv != "e4m3" else pool.scale[i].copy()
            ref.append(host, scale, rows, pool.table, [c - 1 for c in ctx], nodes)
            if kv == "e4m3":
                np.testing.assert_array_equal(pool.dscale[i].double().cpu().numpy(), scale)
                got = ref.VALUES[pool.dev[i].view(torch.uint8).cpu().numpy()] * scale[:, None, :, None]
                val = ref.VALUES[host] * scale[:, None, :, None]
                off = (got != val) & ~(np.isnan(got) & np.isnan(val))
                step = np.maximum(np.abs(val) * 2.0 ** -3, 2.0 ** -9 * scale[:, None, :, None])
                assert (np.abs(got - val)[off] <= (step + sl.max())[off]).all() and off.sum() <= max(4, 1e-4 * t * 2 * hd)
            else:
                got = pool.dev[i].double().cpu().numpy()
                err = np.abs(got - host)
                live = ~np.isnan(host)
                assert (np.isnan(got) == ~live).all()
                assert (err <= np.abs(host) * tree.HALF[kv] + sl.max() + 2.0 ** -25)[live].all()


@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_of_trees_in_place(pkg, kv, src, interleaved):
    """q_out may be q itself, where they are of one type: the bits of the call with another."""
    import torch
    for hd, n_head, past, nodes in ((128, 6, (5, 31, 0), (7, 40, 1)), (64, 32, (100,), (700,)), (256, 1, (63, 2), (5, 90))):
        parents, sees, depths, mask = setup(hd, nodes, 32)
        ctx, t = [a + b for a, b in zip(past, nodes)], sum(nodes)
        rng = np.random.default_rng(hd)
        q, kn, vn = (tt(rng.standard_normal((t + 1, h, hd)).astype(np.float32)).to(dtype(src)) for h in (n_head, 2, 2))
        cu = tt(np.cumsum((0,) + nodes).astype(np.int32))
        dep = tt(np.concatenate([flat(depths), np.int32([3])]))
        outs = []
        for q_out in (torch.empty_like(q), q.clone()):
            pool = Pool(hd, kv, 2, hd, 32, ctx)
            q_out[t:] = q[t:]
            given = q_out if outs else q
            got = pkg.rope_append(pool.cache(pkg), tt(pool.table), tt(np.int32(ctx) - 1), kn, vn, q=given, q_out=q_out,
                                  rope=pkg.Rope(hd, interleaved=interleaved), cu_tokens=cu, depths=dep)
            assert got is q_out
            outs.append((q_out, pool.dev[0].view(torch.uint8), pool.dev[1].view(torch.uint8)))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*outs))


def test_a_tree_that_is_a_chain_appends_the_same(pkg):
    """Depths 0, 1, ...: the bits of the call without depths (16-bit caches: every row's angle is its own there too)."""
    import torch
    for kv in ("f16", "bf16"):
        a, b = (Pool(3, kv, 2, 128, 32, (60, 41)) for _ in range(2))
        rng = np.random.default_rng(2)
        q, kn, vn = (tt(rng.standard_normal((30, h, 128)).astype(np.float32)) for h in (4, 2, 2))
        rope, pos = pkg.Rope(128), tt(np.int32([59, 40]))
        outs = [pkg.rope_append(p.cache(pkg), tt(p.table), pos, kn, vn, q=q, rope=rope, depths=d)
                for p, d in ((a, None), (b, tt(np.int32(list(range(15)) * 2))))]
        assert torch.equal(*outs)
        for i in range(2):
            assert torch.equal(a.dev[i].view(torch.int16), b.dev[i].view(torch.int16))


# ---------------------------------------------------------------------------
# Kept rows.
# ---------------------------------------------------------------------------
def keep_check(pkg, pool, base, path, counts):
    import torch
    before = [d.view(torch.uint8).clone() for d in pool.dev]
    most = max(max(counts), 1)
    p = np.full((len(counts), most), -3, np.int32)
    for s, x in enumerate(path):
        p[s, :len(x)] = x
    pkg.keep_rows(pool.cache(pkg), tt(pool.table), tt(np.int32(base)), tt(p), tt(np.int32(counts)))
    for i in range(2):
        host, scale = pool.host[i].copy(), None if pool.kv != "e4m3" else pool.scale[i].copy()
        touched = np.zeros(host.shape[:2], bool)
        for s, n in enumerate(counts):
            if n:
                touched |= tree.keep(host, scale, pool.table[s], base[s], path[s], n)
        now = pool.dev[i].view(torch.uint8)
        assert torch.equal(now[tt(~touched)], before[i][tt(~touched)])
        if pool.kv == "e4m3":
            np.testing.assert_array_equal(pool.dscale[i].double().cpu().numpy(), scale)
            np.testing.assert_array_equal(now.cpu().numpy()[touched], host[touched])
            pool.host[i], pool.scale[i] = now.cpu().numpy(), scale
        else:
            got = pool.dev[i].double().cpu().numpy()
            np.testing.assert_array_equal(got[touched], host[touched])
            pool.host[i] = got


@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("hd,page,n_kv", [(64, 16, 3), (128, 64, 2), (256, 48, 1), (128, 256, 2)])
def test_kept_rows(pkg, kv, hd, page, n_kv):
    rng = np.random.default_rng(page)
    ctx = (1, 40, 64, 100, 400, 300, 17)
    base = [0, 16, 60, 64, 37, 48, 16]
    counts = [1, 5, 0, 36, 200, 252, 1]
    path = [sorted(rng.choice(c - b, n, replace=False).tolist()) for c, b, n in zip(ctx, base, counts)]
    path[5] = list(range(252))                                    # every row stays
    pool = Pool(hd + page, kv, n_kv, hd, page, ctx)
    pkg.attn_read_device_error()
    keep_check(pkg, pool, base, path, counts)
    keep_check(pkg, pool, base, [list(range(n)) for n in counts], counts)    # again: nothing moves
    assert pkg.attn_read_device_error() == 0


@pytest.mark.parametrize("order", ["heads", "joint"])
def test_kept_rows_of_other_orders(pkg, order):
    for kv in ("e4m3", "bf16"):
        pool = Pool(4, kv, 3, 128, 32, (90, 200), order=order)
        keep_check(pkg, pool, [20, 100], [[3, 9, 30, 31, 69], list(range(1, 100, 3))], [5, 33])


def test_wrong_paths_and_pages_are_left_alone(pkg):
    import torch
    for kv in ("f16", "e4m3"):
        pool = Pool(5, kv, 1, 64, 16, (60,) * 8)
        before = [d.view(torch.uint8).clone() for d in pool.dev]
        pkg.attn_read_device_error()
        cap = pool.max_pages * 16
        path = np.int32([[1, 1, 5], [2, 1, 5], [-1, 2, 5], [0, 4, cap - 20], [0, 1, 2], [0, 1, 2], [3, 4, 9], [0, 0, 0]])
        pkg.keep_rows(pool.cache(pkg), tt(pool.table), tt(np.int32([20, 20, 20, 20, -1, 20, 20, 20])), tt(path),
                      tt(np.int32([3, 3, 3, 3, 3, 4, -1, 0])))
        assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_BAD_REQUEST
        assert all(torch.equal(d.view(torch.uint8), b) for d, b in zip(pool.dev, before))
        # rows from and to pages that are not there
        pool.table[0, 2] = -1
        pkg.keep_rows(pool.cache(pkg), tt(pool.table[:1]), tt(np.int32([20])), tt(np.int32([[1, 14, 30]])), tt(np.int32([3])))
        assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_BAD_PAGE
        p = int(pool.table[0, 1])
        for i in range(2):
            now = pool.dev[i].view(torch.uint8)
            if kv == "f16":
                a, b = now[p, 20 - 16], before[i][p, 21 - 16]
                assert torch.equal(a, b)
                assert torch.equal(now[p, 21 - 16], before[i][p, 21 - 16])      # from a page that is not there
                assert torch.equal(now[p, 22 - 16], before[i][int(pool.table[0, 3]), 50 - 48])


# ---------------------------------------------------------------------------
# A step of decoding, several times.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kv,hd,src", [("e4m3", 128, "bf16"), ("bf16", 64, "f32"), ("f16", 256, "f16")])
def test_steps_with_trees(pkg, kv, hd, src):
    """Pages for the tree, its append, attention, the accepted path, pages given back, forks: held at every step to
    a cache kept by the reference from what the device's cache held before."""
    import torch
    rng = np.random.default_rng(1)
    page, n_seq, n_kv, group, n = 16, 4, 2, 3, 12
    n_pages, max_pages = 64, 12
    refs = np.zeros(n_pages, np.int32)
    table = np.full((n_seq, max_pages), -1, np.int32)
    rows = np.int32([20, 33, 0, 0])
    pools = []
    for _ in range(2):
        x = tt(rng.standard_normal((n_pages, page, n_kv, hd)).astype(np.float32))
        pools.append(x.to(torch.float8_e4m3fn if kv == "e4m3" else dtype(kv)))
    scales = [tt(np.ones((n_pages, n_kv), np.float32)) if kv == "e4m3" else None for _ in range(2)]
    cache = pkg.PagedCache(*pools, *scales)
    book = pkg.PageBook(tt(refs), tt(table), page)
    pkg.attn_read_device_error()
    zero = np.zeros(n_seq, np.int32)
    book.resize(tt(zero), tt(rows))
    tree.resize(refs, table, page, zero, rows)
    rope = pkg.Rope(hd)

    def values(i, s, upto):
        x = pools[i].view(torch.uint8).view(torch.float8_e4m3fn) if kv == "e4m3" else pools[i]
        v = x.double().cpu().numpy()
        if kv == "e4m3":
            v = v * scales[i].double().cpu().numpy()[:, None, :, None]
        return np.array([v[table[s, j // page], j % page] for j in range(upto)]).reshape(upto, n_kv, hd)
    for step in range(5):
        if step == 2:                                             # two more sequences begin as forks
            src_, dst_, r_ = np.int32([0, 1]), np.int32([2, 3]), rows[:2].copy()
            copies = book.fork(tt(src_), tt(dst_), tt(r_))
            pkg.copy_pages(cache, copies)
            want, err = tree.fork(refs, table, page, src_, dst_, r_)
            np.testing.assert_array_equal(copies.cpu().numpy(), want)
            rows[2:] = r_
            for i in range(2):
                for s in range(2):
                    np.testing.assert_array_equal(values(i, s, rows[s]), values(i, s + 2, rows[s]))
        nodes = [n if r else 0 for r in rows]
        cu = np.cumsum([0] + nodes).astype(np.int32)
        parents, sees, depths, mask = setup(step, nodes, 1)
        grown = (rows + np.int32(nodes)).astype(np.int32)
        book.resize(tt(rows), tt(grown))
        tree.resize(refs, table, page, rows, grown)
        t = int(cu[-1])
        qn, kn, vn = (tt(rng.standard_normal((t, h, hd)).astype(np.float32)).to(dtype(src)) for h in (n_kv * group, n_kv, n_kv))
        dm, dd = pkg.tree_rules(tt(flat(parents)), cu_tokens=tt(cu), max_nodes=n)
        np.testing.assert_array_equal(dm.cpu().numpy(), mask)
        pos = tt(grown - 1)
        q = pkg.rope_append(cache, book.block_table, pos, kn, vn, q=qn, q_out=torch.empty_like(qn), rope=rope,
                            cu_tokens=tt(cu), depths=dd)
        out = pkg.tree_decode_attention(cache, book.block_table, pos, q, mask=dm, depths=dd, cu_tokens=tt(cu), max_nodes=n)
        np.testing.assert_array_equal(book.block_table.cpu().numpy(), table)
        k, v = ([values(i, s, grown[s]) for s in range(n_seq)] for i in range(2))
        qh = q.double().cpu().numpy()
        vm = [448.0 * float(scales[1].max()) if kv == "e4m3" else max(np.abs(x).max(initial=0.0), 1.0) for x in v]
        want, bound = tree.attend([qh[cu[s]:cu[s + 1]] for s in range(n_seq)], sees, depths, k, v, hd ** -0.5, kv, src, vmax=vm)
        check(out, np.concatenate(want), np.concatenate(bound), "step %d" % step)
        # the path to some node is accepted
        path = [sorted(sees[s][nodes[s] - 1 - step]) if nodes[s] else [] for s in range(n_seq)]
        counts = np.int32([len(p) for p in path])
        pad = np.full((n_seq, max(counts)), -1, np.int32)
        for s, p in enumerate(path):
            pad[s, :len(p)] = p
        kept = [[values(i, s, grown[s])[[rows[s] + y for y in path[s]]] for s in range(n_seq)] for i in range(2)]
        pkg.keep_rows(cache, book.block_table, tt(rows), tt(pad), tt(counts))
        after = (rows + counts).astype(np.int32)
        book.resize(tt(grown), tt(after))
        assert tree.resize(refs, table, page, grown, after) == 0
        for i in range(2):
            for s in range(n_seq):
                got = values(i, s, after[s])[rows[s]:]
                # values that were moved to a larger scale may have been rounded again: half a step of e4m3, or of its
                # smallest at the page's scale
                lim = np.abs(kept[i][s]) * 2.0 ** -4 + 2.0 ** -10 * float(scales[i].max()) if kv == "e4m3" else 0.0
                assert (np.abs(got - kept[i][s]) <= lim).all()
        rows = after
        np.testing.assert_array_equal(book.refs.cpu().numpy(), refs)
        np.testing.assert_array_equal(book.block_table.cpu().numpy(), table)
    assert pkg.attn_read_device_error() == 0
