"""GPU: the paged-cache operators against the 64-bit restatement in paged_reference.py.

Attention is held to the element-wise bound that the reference derives from the inputs. Append: a
16-bit element to half a step of its type plus the rotation's 32-bit error; an e4m3 element to half a
step at the page's scale plus the same; scales, rescaled rows and everything that must
not change exactly.
"""
import math

import numpy as np
import pytest

import paged_reference as ref
from harness import ABS_TOL, REL_TOL

pytestmark = pytest.mark.gpu

EPS_PAIR = {"f16": 2.0 ** -22, "bf16": 2.0 ** -24, "e4m3": 2.0 ** -22}    # two or three parts of q and p


@pytest.fixture(scope="module")
def pkg():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import decode_attention_gqa_gb300 as p
    from decode_attention_gqa_gb300 import build
    build.build()
    p.load()
    p.attn_read_device_error()
    return p


def tt(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


class Pool:
    """A paged cache with scattered pages; rows that no sequence has hold NaN."""

    def __init__(self, seed, kv, n_kv, hd, page, ctx, spare=2, gain=1.0, order="rows", extra_pages=0):
        import torch
        rng = np.random.default_rng(seed)
        self.kv, self.page, self.ctx = kv, page, [int(c) for c in ctx]
        used = [-(-c // page) for c in self.ctx]
        self.max_pages = max(max(used), 1) + extra_pages
        self.n_pages = sum(used) + spare
        ids = rng.permutation(self.n_pages)
        # entries past a sequence's last page are never looked at
        self.table = rng.choice([-1, -2 ** 31, 2 ** 31 - 1, self.n_pages],
                                (len(ctx), self.max_pages)).astype(np.int32)
        at = 0
        for s, n in enumerate(used):
            self.table[s, :n] = ids[at:at + n]
            at += n
        shape = (self.n_pages, page, n_kv, hd)
        live = np.zeros(shape[:2], bool)
        for s, c in enumerate(self.ctx):
            for j in range(c):
                live[self.table[s, j // page], j % page] = True
        self.host, self.scale, self.dev, self.dscale = [], [], [], []
        for _ in range(2):
            x = rng.standard_normal(shape) * gain
            if kv == "e4m3":
                sc = 2.0 ** rng.integers(-4, 3, (self.n_pages, n_kv)).astype(np.float64)
                codes = ref.to_e4m3(x * rng.choice([1.0, 20.0, 100.0], (self.n_pages, 1, n_kv, 1)))
                codes[~live] = 0x7F
                self.host.append(codes)
                self.scale.append(sc)
                d = tt(codes).view(torch.float8_e4m3fn)
                self.dscale.append(tt(sc.astype(np.float32)))
            else:
                d = tt(x).to(torch.float16 if kv == "f16" else torch.bfloat16)
                d[tt(~live)] = math.nan
                self.host.append(d.double().cpu().numpy())
                self.scale.append(None)
                self.dscale.append(None)
            if order == "heads":
                d = self._as(d, (0, 2, 1, 3))
            elif order == "joint":                    # k and v pages side by side in one allocation
                big = torch.zeros(self.n_pages, 2, *shape[1:], dtype=torch.uint8 if kv == "e4m3" else d.dtype,
                                  device="cuda")
                part = big[:, len(self.dev)]
                part.copy_(d.view(torch.uint8) if kv == "e4m3" else d)
                d = part.view(torch.float8_e4m3fn) if kv == "e4m3" else part
            self.dev.append(d)

    def _as(self, d, perm):
        import torch
        u = d.view(torch.uint8) if self.kv == "e4m3" else d
        u = u.permute(*perm).contiguous().permute(*perm)
        return u.view(torch.float8_e4m3fn) if self.kv == "e4m3" else u

    def cache(self, pkg):
        return pkg.PagedCache(self.dev[0], self.dev[1], self.dscale[0], self.dscale[1])

    def rows(self, i, ctx=None):
        """Per sequence float64 [ctx, n_kv, hd]; rows of pages that are not there NaN."""
        out = []
        for s, c in enumerate(self.ctx if ctx is None else ctx):
            x = np.empty((c,) + self.host[i].shape[2:])
            for j in range(c):
                p = self.table[s, j // self.page]
                if not 0 <= p < self.n_pages:
                    x[j] = math.nan
                elif self.kv == "e4m3":
                    x[j] = ref.VALUES[self.host[i][p, j % self.page]] * self.scale[i][p][:, None]
                else:
                    x[j] = self.host[i][p, j % self.page]
            out.append(x)
        return out


def check(got, want, bound, what=""):
    got = got.double().cpu().numpy()
    err = np.abs(got - want)
    bad = ~(err <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, err / np.maximum(bound, 1e-300), -1)), err.shape)
        raise AssertionError("%s: %d of %d elements outside; at %s got %r want %r, bound %.3g" % (
            what, int(bad.sum()), bad.size, i, got[i], want[i], bound[i]))


def attend_check(pkg, pool, n_q, n_head, seed=1, splits=(0,), positions=None, ctx=None, what="", **rules):
    rng = np.random.default_rng(seed)
    hd = pool.host[0].shape[3]
    n_seq = len(pool.ctx)
    q = rng.standard_normal((n_seq, n_q, n_head, hd)).astype(np.float32)
    pos = np.asarray(positions if positions is not None else [c - 1 for c in pool.ctx], np.int32)
    host = dict(rules)
    dev = dict(rules)
    if rules.get("slopes") is not None:
        host["slopes"] = np.asarray(rules["slopes"], np.float32)
        dev["slopes"] = tt(host["slopes"])
    if rules.get("starts") is not None:
        dev["starts"] = tt(np.asarray(rules["starts"], np.int32))
    want, bound = ref.attend(q, pool.rows(0, ctx), pool.rows(1, ctx), pos, hd ** -0.5,
                             eps_pair=EPS_PAIR[pool.kv], **host)
    cache, table, dpos, dq = pool.cache(pkg), tt(pool.table), tt(pos), tt(q)
    outs = []
    for P in splits:
        out = pkg.paged_decode_attention(cache, table, dpos, dq, n_splits=P, **dev)
        check(out, want, bound, "%s P=%d" % (what, P))
        outs.append(out)
    return outs


CTX = (0, 1, 15, 16, 17, 48, 63, 64, 65, 127, 200, 331)


@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("group,page", [(1, 16), (5, 48), (8, 64)])
def test_one_query_row(pkg, kv, hd, group, page):
    n_kv = 2
    pool = Pool(hd + group, kv, n_kv, hd, page, CTX)
    attend_check(pkg, pool, 1, group * n_kv, splits=(0, 1, 2, 7))
    assert pkg.attn_read_device_error() == 0


@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("n_q,group,page", [(2, 4, 32), (3, 5, 16), (5, 7, 128), (17, 3, 80), (1, 13, 16), (1, 64, 256)])
def test_several_query_rows_and_large_groups(pkg, kv, hd, n_q, group, page):
    ctx = (0, 1, 3, 16, 17, 30, 65, 130, 257)
    pool = Pool(hd + n_q, kv, 1, hd, page, ctx)
    attend_check(pkg, pool, n_q, group, splits=(0, 1, 3))
    assert pkg.attn_read_device_error() == 0


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("n_q,group,rules", [(2, 5, {}), (5, 7, {}), (1, 13, {}), (4, 8, dict(window=60, softcap=20.0)), (17, 3, {}),
                                             (4, 8, dict(softcap=20.0, slopes=True)), (2, 7, dict(starts=[0, 0, 69, 5, 900]))])
def test_large_groups_in_a_large_capacity(pkg, hd, n_q, group, rules):
    """8 bits: 16 slots a block where the capacity is large, whatever rows there are."""
    pool = Pool(hd + n_q, "e4m3", 2, hd, 64, (0, 1, 70, 333, 1000), extra_pages=4000)
    r = dict(rules)
    if r.get("slopes"):
        r["slopes"] = [2.0 ** -(h + 1) for h in range(group * 2)]
    attend_check(pkg, pool, n_q, group * 2, splits=(0, 1, 3), **r)
    assert pkg.attn_read_device_error() == 0


@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("n_q,group", [(1, 2), (4, 4)])
def test_many_tiles_a_block(pkg, kv, hd, n_q, group):
    """Blocks that go round their stages and descriptor buffers many times, across sequences, also with a
    window that begins late."""
    pool = Pool(hd + n_q, kv, 1, hd, 32, (2900, 0, 1411, 33, 800))
    attend_check(pkg, pool, n_q, group, splits=(1, 2, 5, 0))
    attend_check(pkg, pool, n_q, group, splits=(1, 3), window=1300)
    assert pkg.attn_read_device_error() == 0


def test_more_sequences_than_a_launch_takes(pkg):
    rng = np.random.default_rng(0)
    pool = Pool(1, "e4m3", 1, 64, 16, [int(x) for x in rng.integers(0, 70, 300)])
    attend_check(pkg, pool, 1, 2, splits=(0, 1, 5))
    attend_check(pkg, pool, 2, 2, splits=(0,), starts=[int(x) for x in rng.integers(0, 40, 300)], window=30)
    assert pkg.attn_read_device_error() == 0


@pytest.mark.parametrize("kv,hd,n_q,group", [("f16", 64, 1, 2), ("bf16", 128, 3, 4), ("e4m3", 256, 1, 1)])
def test_blocks_that_cross_many_sequences(pkg, kv, hd, n_q, group):
    """Long, short and empty sequences in turn, over few and many blocks: every place a boundary can fall."""
    rng = np.random.default_rng(hd)
    ctx = [int(x) for x in rng.choice([0, 1, 40, 64, 200, 700, 1500], 40)]
    pool = Pool(hd, kv, 1, hd, 64, ctx)
    attend_check(pkg, pool, n_q, group, splits=(0, 1, 2, 3, 7, 31, 100, 300))
    attend_check(pkg, pool, n_q, group, splits=(0, 5, 40), window=150, starts=[int(x) for x in rng.choice([0, 30, 650], 40)])
    assert pkg.attn_read_device_error() == 0


RULES = [
    dict(softcap=20.0), dict(window=1), dict(window=40), dict(window=100000), dict(slopes=True),
    dict(starts=True), dict(softcap=5.0, window=33, slopes=True, starts=True), dict(window=70, starts=True),
]


@pytest.mark.parametrize("kv,hd", [("e4m3", 128), ("e4m3", 64), ("bf16", 256), ("f16", 128)])
@pytest.mark.parametrize("n_q,group", [(1, 4), (4, 3), (1, 12)])
@pytest.mark.parametrize("rules", RULES)
def test_score_rules(pkg, kv, hd, n_q, group, rules):
    ctx = (0, 1, 2, 17, 64, 100, 193, 300)
    n_kv = 2
    pool = Pool(hd + n_q, kv, n_kv, hd, 32, ctx)
    r = dict(rules)
    if r.get("slopes"):
        r["slopes"] = [2.0 ** (-8 * (h + 1) / (group * n_kv)) for h in range(group * n_kv)]
    if r.get("starts"):
        r["starts"] = [0, 1, 0, 5, 63, 100, 64, 130]      # some at or past the last row: nothing to see
    attend_check(pkg, pool, n_q, group * n_kv, splits=(0, 1, 3), what=str(rules), **r)
    assert pkg.attn_read_device_error() == 0


def test_rows_and_pages_that_nothing_sees_are_not_read(pkg):
    """Pages below the window or the start have no entry at all."""
    ctx = (300, 290, 120)
    for rules, gone in ((dict(window=50), (240, 224, 64)), (dict(starts=[200, 1, 119]), (192, 0, 112))):
        pool = Pool(5, "e4m3", 2, 128, 16, ctx)
        for s, g in enumerate(gone):
            pool.table[s, :g // 16] = -9
        attend_check(pkg, pool, 1, 8, splits=(0, 1, 4), **rules)
        assert pkg.attn_read_device_error() == 0


@pytest.mark.parametrize("kv", ["e4m3", "f16"])
def test_pages_that_are_not_there(pkg, kv):
    """A used entry outside the pool: flagged, its rows not attended."""
    pool = Pool(6, kv, 2, 128, 32, (200, 64, 33))
    pool.table[0, 2] = -1
    pool.table[0, 5] = pool.n_pages
    pool.table[1, :2] = 2 ** 31 - 1                       # nothing left: 0
    pool.table[2, 0] = -2 ** 31
    outs = attend_check(pkg, pool, 1, 8, splits=(0, 1, 3))
    assert float(outs[0][1].abs().max()) == 0.0
    assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_BAD_PAGE
    attend_check(pkg, pool, 3, 8, splits=(0,), window=60)
    pkg.attn_read_device_error()


def test_positions_out_of_range(pkg):
    pool = Pool(7, "e4m3", 2, 128, 16, (64, 64, 64))      # max_pages 4: capacity 64
    attend_check(pkg, pool, 1, 8, positions=[63, 1000, -1], ctx=[64, 64, 0], splits=(0, 1))
    assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_POSITION_CLAMPED
    attend_check(pkg, pool, 2, 8, positions=[-5, 10, -2 ** 31], ctx=[0, 11, 0], splits=(0, 2))
    assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_POSITION_CLAMPED


@pytest.mark.parametrize("order", ["heads", "joint"])
@pytest.mark.parametrize("kv,hd", [("e4m3", 64), ("e4m3", 256), ("f16", 128)])
def test_other_orders_and_parts_of_an_allocation(pkg, order, kv, hd):
    pool = Pool(8, kv, 3, hd, 48, (1, 50, 333, 96), order=order)
    attend_check(pkg, pool, 1, 6, splits=(0, 3))
    attend_check(pkg, pool, 4, 6, splits=(0,))


def test_scales_of_any_size(pkg):
    """Scales far apart between pages, zero, negative and no power of two."""
    pool = Pool(9, "e4m3", 2, 128, 16, (160, 90, 16))
    rng = np.random.default_rng(0)
    for i in range(2):
        sc = np.float32(2.0 ** rng.integers(-28, 12, pool.scale[i].shape) * rng.uniform(0.5, 1, pool.scale[i].shape))
        if i == 0:
            sc = np.minimum(sc, np.float32(0.02))
        sc[0], sc[1] = 0.0, -sc[1]
        pool.scale[i] = sc.astype(np.float64)
        pool.dscale[i] = tt(sc)
    attend_check(pkg, pool, 1, 8, splits=(0, 1, 3))
    attend_check(pkg, pool, 3, 4, splits=(0,), softcap=30.0)
    # V scales of one page far below the others', whose scores carry the weight
    pool = Pool(10, "e4m3", 1, 128, 16, (64,))
    for e in (-55, -20, 20, 55):
        sc = np.full(pool.scale[1].shape, 2.0 ** e)
        pool.scale[1], pool.dscale[1] = sc, tt(sc.astype(np.float32))
        attend_check(pkg, pool, 1, 8, splits=(0, 1))


def test_unseen_infinities_and_nan(pkg):
    """A row that a later query row sees may hold anything for an earlier one."""
    for kv in ("f16", "e4m3"):
        pool = Pool(11, kv, 1, 128, 16, (70,))
        p = int(pool.table[0, 69 // 16])
        o = 69 % 16
        for i in range(2):
            d = pool.dev[i].view(__import__("torch").uint8) if kv == "e4m3" else pool.dev[i]
            d[p, o] = 0x7F if kv == "e4m3" else (math.inf if i else math.nan)
        rng = np.random.default_rng(2)
        q = rng.standard_normal((1, 3, 4, 128)).astype(np.float32)
        k, v = pool.rows(0), pool.rows(1)
        k[0], v[0] = k[0][:69], v[0][:69]
        want, bound = ref.attend(q[:, :2], k, v, [68], 128 ** -0.5, eps_pair=EPS_PAIR[kv])
        for P in (0, 1):
            out = pkg.paged_decode_attention(pool.cache(pkg), tt(pool.table), tt(np.int32([69])), tt(q), n_splits=P)
            check(out[:, :2], want, bound, kv)


def test_same_as_the_dense_call(pkg):
    """Consecutive page numbers over a dense cache: what decode_attention computes."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    for dt, n_q in ((torch.float16, 1), (torch.bfloat16, 1), (torch.float16, 4)):
        k = torch.randn(3, 512, 4, 128, generator=g, device="cuda").to(dt)
        v = torch.randn(3, 512, 4, 128, generator=g, device="cuda").to(dt)
        q = torch.randn(3, n_q, 28, 128, generator=g, device="cuda")
        pos = torch.tensor([511, 100, 7], dtype=torch.int32, device="cuda")
        table = torch.arange(24, dtype=torch.int32, device="cuda").view(3, 8)
        cache = pkg.PagedCache(k.view(24, 64, 4, 128), v.view(24, 64, 4, 128))
        got = pkg.paged_decode_attention(cache, table, pos, q)
        want = pkg.decode_attention(q if n_q > 1 else q[:, 0].contiguous(), k, v, pos).view_as(got)
        assert bool(((got - want).abs() <= ABS_TOL + REL_TOL * want.abs()).all())


def test_long_context_and_far_pages(pkg):
    """100,000 rows, in a pool whose elements lie past 2^32 bytes."""
    import torch
    page, n_kv, hd, n = 256, 4, 128, 100001
    n_pages = 40000                                        # 5.2 GB a pool
    used = -(-n // page)
    pools = [torch.empty(n_pages, page, n_kv, hd, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((n_pages, n_kv), 0.0625, device="cuda") for _ in range(2)]
    ids = torch.arange(n_pages - used, n_pages, device="cuda").flip(0)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = [torch.randn(used, page, n_kv, hd, generator=g, device="cuda").mul(16).to(torch.float8_e4m3fn)
         for _ in range(2)]
    for i in range(2):
        pools[i][ids] = x[i].view(torch.uint8)
    cache = pkg.PagedCache(*[p.view(torch.float8_e4m3fn) for p in pools], *scales)
    q = torch.randn(1, 16, hd, generator=g, device="cuda")
    pos = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    out = pkg.paged_decode_attention(cache, ids.int()[None].contiguous(), pos, q)
    k, v = (t.double().view(-1, n_kv, hd)[:n] * 0.0625 for t in x)
    s = torch.einsum("kgd,nkd->kgn", q[0].double().view(n_kv, 4, hd), k) * hd ** -0.5
    want = torch.einsum("kgn,nkd->kgd", torch.softmax(s, -1), v).view(1, 16, hd)
    # scores: magnitudes up to sum |q k| = A; the mean of 1e5 rows moves by 2 (A (8 + 4) 2^-23 + 2^-20) of |v|
    A = float((q[0].double().view(n_kv, 4, hd).abs() @ k.abs().amax(0)[:, :, None]).max()) * hd ** -0.5
    assert float((out.double() - want).abs().max()) <= float(v.abs().max()) * 2 * (A * 12 * 2.0 ** -23 + 2.0 ** -20)
    # append at the same far pages
    kn = torch.randn(1, n_kv, hd, generator=g, device="cuda")
    pkg.rope_append(cache, ids.int()[None].contiguous(), pos, kn, kn)
    last = pools[1][ids[(n - 1) // page], (n - 1) % page].view(torch.float8_e4m3fn).float() * \
        scales[1][ids[(n - 1) // page]][:, None]
    assert bool(((last - kn[0]).abs() <= kn[0].abs() * 2.0 ** -4 + 2.0 ** -10 * 0.0625).all())


def test_same_bits_again_and_from_any_workspace(pkg):
    import torch
    pool = Pool(12, "e4m3", 2, 128, 64, (500, 77))
    a = attend_check(pkg, pool, 1, 8)[0]
    b = attend_check(pkg, pool, 1, 8)[0]
    assert torch.equal(a, b)
    # the library-owned workspace and a given one through the C names
    rng = np.random.default_rng(1)
    q = tt(rng.standard_normal((2, 1, 8, 128)).astype(np.float32))
    table, pos, cache = tt(pool.table), tt(np.int32([499, 76])), pool.cache(pkg)
    P, need = pkg.attn_paged_plan(cache, pool.max_pages, 2, 1, 8)
    assert P > 1
    out = torch.full_like(q, math.nan)
    pkg.attn_decode_paged(cache, table, pool.max_pages, pos, q, out, 2, 1, 8, 128 ** -0.5)
    assert torch.equal(out, a)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, math.nan)
    pkg.attn_decode_paged(cache, table, pool.max_pages, pos, q, out, 2, 1, 8, 128 ** -0.5, workspace=ws)
    assert torch.equal(out, a)
    with pytest.raises(pkg.AttnError) as e:
        pkg.attn_decode_paged(cache, table, pool.max_pages, pos, q, out, 2, 1, 8, 128 ** -0.5, workspace=ws,
                              workspace_bytes=need - 256)
    assert e.value.status == pkg.ATTN_ERR_WORKSPACE


def test_pages_that_sequences_share(pkg):
    """A prefix that several sequences have in common, held once; one page twice in a sequence."""
    for kv in ("e4m3", "bf16"):
        pool = Pool(13, kv, 2, 128, 16, (200, 150, 90, 64))
        pool.table[1, :4] = pool.table[0, :4]
        pool.table[2, :5] = pool.table[0, :5]
        pool.table[3, :4] = pool.table[3, 0]
        attend_check(pkg, pool, 1, 8, splits=(0, 1, 4))
        attend_check(pkg, pool, 4, 4, splits=(0,))
    assert pkg.attn_read_device_error() == 0


@pytest.mark.parametrize("kv", ["e4m3", "f16"])
def test_many_query_rows_and_the_largest_pages(pkg, kv):
    pool = Pool(14, kv, 1, 64, 1024, (1500, 1030, 700))
    attend_check(pkg, pool, 1024, 2, splits=(0,), window=300)
    attend_check(pkg, pool, 1024, 1, splits=(0, 3))
    assert pkg.attn_read_device_error() == 0


def test_a_query_row_of_nan_stays_alone(pkg):
    import torch
    pool = Pool(15, "e4m3", 2, 128, 32, (300, 40))
    cache, table, pos = pool.cache(pkg), tt(pool.table), tt(np.int32([299, 39]))
    for n_q, n_head in ((1, 8), (3, 12)):
        q = tt(np.random.default_rng(3).standard_normal((2, n_q, n_head, 128)).astype(np.float32))
        want = pkg.paged_decode_attention(cache, table, pos, q)
        q[0, 0, 1] = math.nan
        q[1, n_q - 1, n_head - 1, 5] = math.nan
        got = pkg.paged_decode_attention(cache, table, pos, q)
        bad = torch.zeros(2, n_q, n_head, dtype=torch.bool, device="cuda")
        bad[0, 0, 1] = bad[1, n_q - 1, n_head - 1] = True
        assert bool(got[bad].isnan().all())
        assert torch.equal(got[~bad], want[~bad])


def test_one_kv_head_and_one_page_with_strides_of_no_meaning(pkg):
    import torch
    pool = Pool(16, "f16", 1, 64, 48, (40,), spare=0)
    for i in range(2):
        pool.dev[i] = torch.as_strided(pool.dev[i], (1, 48, 1, 64), (1, 64, 7, 1))
    attend_check(pkg, pool, 1, 4)
    k = torch.ones(1, 1, 64, device="cuda")
    pkg.rope_append(pool.cache(pkg), tt(pool.table), tt(np.int32([39])), k, k)
    assert bool((pool.dev[1][0, 39] == 1).all()) and pkg.attn_read_device_error() == 0


def test_numbers_past_32_bits_are_refused(pkg):
    pool = Pool(18, "f16", 1, 64, 16, (40,))
    for bad in (dict(window=1 << 31), dict(window=(1 << 32) + 5), dict(n_splits=1 << 32), dict(n_splits=-1)):
        with pytest.raises(ValueError):
            pkg.paged_decode_attention(pool.cache(pkg), tt(pool.table), tt(np.int32([39])),
                                       tt(np.zeros((1, 2, 64), np.float32)), **bad)


def test_calls_on_several_streams_at_once(pkg):
    """Eager calls of different shapes, interleaved on streams, each with the workspace torch gives it."""
    import torch
    jobs = []
    for i, (kv, ctx) in enumerate((("e4m3", (3000, 5)), ("f16", (900, 900)), ("bf16", (2048,)))):
        pool = Pool(40 + i, kv, 2, 128, 64, ctx)
        cache, table, pos = pool.cache(pkg), tt(pool.table), tt(np.int32([c - 1 for c in ctx]))
        q = tt(np.random.default_rng(i).standard_normal((len(ctx), 8, 128)).astype(np.float32))
        jobs.append((cache, table, pos, q, pkg.paged_decode_attention(cache, table, pos, q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for cache, table, pos, q, want, stream in jobs:
            with torch.cuda.stream(stream):
                outs.append((pkg.paged_decode_attention(cache, table, pos, q), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)


# ---------------------------------------------------------------------------
# Append.
# ---------------------------------------------------------------------------
SCALINGS = [dict(), dict(scaling=1, factor=4.0), dict(scaling=2, factor=4.0),
            dict(scaling=3, factor=8.0, low_turns=1.0, high_turns=4.0, trained_len=2048)]


def append_check(pkg, kv, src, n_kv, group, hd, page, past, new, rot, interleaved, scaling={}, mscale=1.0,
                 fused=False, pad=0, cu="given", order="rows", with_q=True, positions=None, seed=0):
    """Sequences with `past` rows get `new` more; returns the pool after (host side updated)."""
    import torch
    rng = np.random.default_rng(seed)
    n_seq, t, n_head = len(new), sum(new), n_kv * group
    ctx = [p + n for p, n in zip(past, new)]
    pool = Pool(seed, kv, n_kv, hd, page, ctx, order=order)
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[src]
    if fused:
        x = tt(rng.standard_normal((t + pad, n_head + 2 * n_kv, hd)).astype(np.float32)).to(dt)
        q, kn, vn = x[:, :n_head], x[:, n_head:n_head + n_kv], x[:, n_head + n_kv:]
    else:
        q, kn, vn = (tt(rng.standard_normal((t + pad, h, hd)).astype(np.float32) * g).to(dt)
                     for h, g in ((n_head, 1), (n_kv, 3.0), (n_kv, 0.7)))
    pos = np.asarray(positions if positions is not None else [c - 1 for c in ctx], np.int32)
    rope = pkg.Rope(rot, interleaved=interleaved, mscale=mscale, **scaling) if rot else None
    before = [d.view(torch.uint8).clone() for d in pool.dev]
    q_out = torch.full((t + pad, n_head, hd), -7.0, device="cuda")
    dcu = tt(np.cumsum([0] + list(new)).astype(np.int32)) if cu == "given" else None
    cache = pool.cache(pkg)
    got_q = pkg.rope_append(cache, tt(pool.table), tt(pos), kn, vn, q=q if with_q else None,
                            q_out=q_out if with_q else None, rope=rope, cu_tokens=dcu)
    torch.cuda.synchronize()
    tok_pos = np.concatenate([np.arange(p + 1 - n, p + 1) for p, n in zip(pos.astype(np.int64), new)] or [[]])
    freq = ref.frequencies(rot, 10000.0, *[scaling.get(k, d) for k, d in (
        ("scaling", 0), ("factor", 1.0), ("low_turns", 0.0), ("high_turns", 0.0), ("trained_len", 0))]) if rot else []

    def turned(x):
        x = x[:t].double().cpu().numpy()
        return ref.rotate(x, tok_pos, np.asarray(freq), interleaved, mscale) if rot else x

    # 32-bit rotation: the sine and cosine to 2^-22 (the angle in 2^-26 turns, sincospi, mscale), two products
    # and a sum: of the pair's magnitude, at most (4.5 sigma here) the row's largest
    def slack(x):
        m = np.abs(x[:t].double().cpu().numpy()).max(axis=-1, keepdims=True) * abs(mscale)
        return 3 * 2.0 ** -22 * m if rot else 0 * m
    if with_q:
        assert got_q is q_out
        check(q_out[:t], turned(q), slack(q) + 1e-30, "q")
        assert bool((q_out[t:] == -7.0).all())
    else:
        assert got_q is None
    for i, rows, sl in ((0, turned(kn), slack(kn)), (1, vn[:t].double().cpu().numpy(), 0 * slack(vn))):
        host = pool.host[i].copy()
        scale = None if kv != "e4m3" else pool.scale[i].copy()
        touched = ref.append(host, scale, rows, pool.table, pos, new)
        now = pool.dev[i].view(torch.uint8)
        keep = tt(~touched)
        assert torch.equal(now[keep], before[i][keep]), "rows that are not the call's changed"
        sfull = np.zeros(host.shape[:2] + (host.shape[2], 1))
        at = 0
        for s, n in enumerate(new):                        # the slack of each written row
            for j in range(n):
                p = int(pos[s]) + 1 - n + j
                if 0 <= p < pool.table.shape[1] * page and 0 <= pool.table[s, p // page] < pool.n_pages:
                    sfull[pool.table[s, p // page], p % page] = sl[at + j]
            at += n
        if kv == "e4m3":
            np.testing.assert_array_equal(pool.dscale[i].double().cpu().numpy(), scale)
            got = ref.VALUES[now.cpu().numpy()] * scale[:, None, :, None]
            want = ref.VALUES[host] * scale[:, None, :, None]
            # the same code, or a neighbour where the value lies within the slack of the border
            exact = got == want
            off = touched[:, :, None, None] & ~exact & ~(np.isnan(got) & np.isnan(want))
            step = np.maximum(np.abs(want) * 2.0 ** -3, 2.0 ** -9 * scale[:, None, :, None])
            assert (np.abs(got - want)[off] <= (step + np.broadcast_to(sfull, got.shape))[off]).all()
            assert off.sum() <= max(4, 1e-4 * touched.sum() * host.shape[2] * host.shape[3])
            pool.host[i], pool.scale[i] = now.cpu().numpy(), scale
        else:
            got = pool.dev[i].double().cpu().numpy()
            half = 2.0 ** -11 if kv == "f16" else 2.0 ** -8
            err = np.abs(got - host)[touched]
            lim = (np.abs(host) * half + sfull + 2.0 ** -25)[touched]
            assert (err <= lim).all(), float((err / lim).max())
            pool.host[i] = got
    return pool, q_out


@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hd,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 64), (256, 256), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_prompts(pkg, kv, src, hd, rot, interleaved):
    if rot == 0 and interleaved:
        pytest.skip("no rotation has no layout")
    append_check(pkg, kv, src, 2, 3, hd, 32, (0, 5, 31, 32, 0, 64, 7), (40, 1, 2, 33, 0, 64, 100), rot, interleaved,
                 SCALINGS[(hd + rot) // 16 % 4], mscale=1.0 if rot % 32 else 1.25, fused=(src != "f32"), pad=3)
    assert pkg.attn_read_device_error() == 0


@pytest.mark.parametrize("kv", ["e4m3", "bf16"])
def test_append_steps(pkg, kv):
    """One token a sequence, and the same number each, without offsets."""
    append_check(pkg, kv, "bf16", 4, 7, 128, 64, (0, 63, 64, 100, 8000), (1,) * 5, 128, False, cu=None)
    append_check(pkg, kv, "f32", 1, 8, 256, 16, (0, 15, 16, 10), (5,) * 4, 64, True, cu=None, order="heads")
    append_check(pkg, kv, "f16", 2, 1, 64, 48, (3, 47), (130, 130), 32, False, cu=None, with_q=False)
    append_check(pkg, kv, "f16", 2, 4, 64, 1024, (3, 1000), (1, 1500), 64, False, order="joint")
    assert pkg.attn_read_device_error() == 0


def test_append_many_sequences(pkg):
    """Offsets that the search has to find its way through, empty sequences among them."""
    rng = np.random.default_rng(3)
    new = [int(x) for x in rng.choice([0, 0, 1, 1, 2, 17, 40], 1100)]
    new[0] = new[-1] = 0
    append_check(pkg, "e4m3", "bf16", 1, 1, 64, 16, [int(x) for x in rng.integers(0, 40, 1100)], new, 64, False)
    append_check(pkg, "f16", "bf16", 1, 1, 64, 16, [int(x) for x in rng.integers(0, 40, 1100)], new, 64, False)


def test_append_far_positions(pkg):
    """The angle at a far position loses nothing: the same bound as at the first."""
    import torch
    pos = [0, 131071, 2 ** 24 + 1, 2 ** 30 - 7]
    q = tt(np.random.default_rng(1).standard_normal((4, 2, 64)).astype(np.float32))
    k = torch.zeros(4, 1, 64, device="cuda")
    pool = Pool(0, "f16", 1, 64, 16, (16,) * 4)
    rope = pkg.Rope(64, base=10000.0)
    out = pkg.rope_append(pool.cache(pkg), tt(pool.table), tt(np.int32(pos)), k, k, q=q, rope=rope)
    # the steps are the definition here: their fixed-point angle in exact integers
    steps = pkg.attn_rope_steps(64, 10000.0)
    turns = np.array([[(p * s % 2 ** 64) / 2.0 ** 64 for s in steps] for p in pos])
    x = q.double().cpu().numpy()
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    want = np.concatenate([x[..., :32] * c - x[..., 32:] * s, x[..., 32:] * c + x[..., :32] * s], -1)
    check(out, want, np.full(want.shape, 3 * 2.0 ** -22 * np.abs(x).max()), "far")
    assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_POSITION_CLAMPED


@pytest.mark.parametrize("kv", ["e4m3", "f16"])
def test_append_bad_pages_idle_sequences_and_positions(pkg, kv):
    import torch
    kw = dict(hd=64, page=16, rot=64, interleaved=False)
    # an idle sequence (position -1) is not flagged and writes nothing
    append_check(pkg, kv, "f16", 2, 2, past=(10, 4), new=(1, 1), positions=[10, -1], **kw)
    assert pkg.attn_read_device_error() == 0
    # past the capacity, and tokens before position 0
    append_check(pkg, kv, "f16", 2, 2, past=(20, 20), new=(4, 4), positions=[33, 23], **kw)
    assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_POSITION_CLAMPED
    append_check(pkg, kv, "f16", 2, 2, past=(20, 20), new=(4, 4), positions=[1, 23], **kw)
    assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_POSITION_CLAMPED
    # a page that is not there
    pool = Pool(1, kv, 2, 64, 16, (40, 20))
    pool.table[0, 1] = pool.n_pages
    pool.table[1, 0] = -1
    before = [d.view(torch.uint8).clone() for d in pool.dev]
    x = torch.ones(42, 2, 64, device="cuda").half()
    pkg.rope_append(pool.cache(pkg), tt(pool.table), tt(np.int32([33, 7])), x, x,
                    cu_tokens=tt(np.int32([0, 34, 42])))
    assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_BAD_PAGE
    written = np.zeros((pool.n_pages, 16), bool)
    written[pool.table[0, 0]] = True
    written[pool.table[0, 2], :2] = True
    for d, b in zip(pool.dev, before):
        same = (d.view(torch.uint8) == b).flatten(2).all(-1).cpu().numpy()
        assert same[~written].all() and not same[written].any()


def test_append_rescales_kept_rows(pkg):
    """A page whose later rows are larger: its first rows move to the larger scale, codes that fall below
    the smallest normal one rounded to even, and the scale never shrinks until a page starts anew."""
    import torch
    pool = Pool(2, "e4m3", 1, 64, 16, (16,))
    cache, table = pool.cache(pkg), tt(pool.table)
    host = [pool.host[0].copy(), pool.host[1].copy()]
    scale = [pool.scale[0].copy(), pool.scale[1].copy()]
    rng = np.random.default_rng(0)
    for j, size in enumerate([1e-3, 1.0, 1.0, 700.0, 5.0, 0.0, 1e4, 1e-8, 3e4]):
        x = (rng.standard_normal((1, 1, 64)) * size).astype(np.float32)
        pkg.rope_append(cache, table, tt(np.int32([j])), tt(x), tt(-x))
        for i, sign in ((0, 1), (1, -1)):
            ref.append(host[i], scale[i], sign * x.astype(np.float64), pool.table, [j], [1])
            np.testing.assert_array_equal(pool.dscale[i].double().cpu().numpy(), scale[i])
            np.testing.assert_array_equal(pool.dev[i].view(torch.uint8).cpu().numpy(), host[i])
    x = np.full((1, 1, 64), 1e-5, np.float32)              # the page starts anew
    pkg.rope_append(cache, table, tt(np.int32([0])), tt(x), tt(x))
    assert float(pool.dscale[0][pool.table[0, 0], 0]) == ref.scale_for(float(np.float32(1e-5)))


def test_append_infinities_and_nan(pkg):
    import torch
    pool = Pool(3, "e4m3", 1, 64, 16, (16,))
    x = np.ones((2, 1, 64), np.float32)
    x[0, 0, 3], x[0, 0, 4], x[1, 0, 5] = math.inf, -math.inf, math.nan
    pkg.rope_append(pool.cache(pkg), tt(pool.table), tt(np.int32([1])), tt(x), tt(x))
    p = int(pool.table[0, 0])
    sc = float(pool.dscale[1][p, 0])
    assert sc == ref.scale_for(1.0)
    got = ref.VALUES[pool.dev[1].view(torch.uint8)[p, :2, 0].cpu().numpy()] * sc
    assert got[0, 3] == 448 * sc and got[0, 4] == -448 * sc and math.isnan(got[1, 5])
    rest = np.ones((2, 64), bool)
    rest[0, 3] = rest[0, 4] = rest[1, 5] = False
    assert (got[rest] == 1.0).all()


@pytest.mark.parametrize("kv", ["e4m3", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_at_addresses_of_16_bytes(pkg, kv, interleaved):
    """Tensors and a pool that start 16 bytes past a multiple of 32 give what aligned ones give."""
    import torch
    rng = np.random.default_rng(8)
    dt, es = (torch.uint8, 1) if kv == "e4m3" else (torch.float16, 2)

    def shifted(x):
        n, by = x.numel(), 16 // x.element_size()
        base = torch.zeros(n + 2 * by, dtype=x.dtype, device="cuda")
        out = base[by:by + n].view(x.shape)
        out.copy_(x)
        assert out.data_ptr() % 32 == 16
        return out

    x = [tt(rng.standard_normal((5, h, 128)).astype(np.float32)) for h in (4, 2, 2)]
    table, pos, cu = tt(np.int32([[1, 0], [2, 3]])), tt(np.int32([17, 1])), tt(np.int32([0, 3, 5]))
    rope, got = pkg.Rope(96, interleaved=interleaved), []
    for place in (lambda t: t, shifted):
        pools = [place(torch.zeros(4, 16, 2, 128, dtype=dt, device="cuda")) for _ in range(2)]
        scales = [torch.zeros(4, 2, device="cuda") if es == 1 else None for _ in range(2)]
        view = [p.view(torch.float8_e4m3fn) if es == 1 else p for p in pools]
        q_out = place(torch.zeros(5, 4, 128, device="cuda"))
        cache = pkg.PagedCache(view[0], view[1], scales[0], scales[1])
        pkg.rope_append(cache, table, pos, place(x[1]), place(x[2]), q=place(x[0]), q_out=q_out, rope=rope, cu_tokens=cu)
        got.append([q_out] + pools + [s for s in scales if s is not None] +
                   [pkg.paged_decode_attention(cache, table, pos, place(torch.ones(2, 4, 128, device="cuda")))])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert pkg.attn_read_device_error() == 0


def test_append_nothing_and_in_place(pkg):
    import torch
    pool = Pool(17, "e4m3", 2, 64, 16, (20, 3))
    cache, table, pos = pool.cache(pkg), tt(pool.table), tt(np.int32([19, 2]))
    before = [d.view(torch.uint8).clone() for d in pool.dev]
    none = torch.zeros(0, 2, 64, device="cuda")
    out = pkg.rope_append(cache, table, pos, none, none, q=torch.zeros(0, 4, 64, device="cuda"), rope=pkg.Rope(64),
                          cu_tokens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64)
    # a padded batch without a token: everything lies behind the last sequence
    pad = torch.ones(4, 2, 64, device="cuda")
    pkg.rope_append(cache, table, pos, pad, pad, cu_tokens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert all(torch.equal(d.view(torch.uint8), b) for d, b in zip(pool.dev, before))
    # q turned where it is
    q = tt(np.random.default_rng(1).standard_normal((2, 4, 64)).astype(np.float32))
    k = torch.ones(2, 2, 64, device="cuda")
    want = pkg.rope_append(cache, table, pos, k, k, q=q, rope=pkg.Rope(64))
    same = pkg.rope_append(cache, table, pos, k, k, q=q, q_out=q, rope=pkg.Rope(64))
    assert same is q and torch.equal(q, want)
    with pytest.raises(ValueError):                          # q_out would be allocated on another stream
        pkg.rope_append(cache, table, pos, k, k, q=q, stream=torch.cuda.Stream())
    assert pkg.attn_read_device_error() == 0


# ---------------------------------------------------------------------------
# Together.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kv,hd,rules", [("e4m3", 128, {}), ("e4m3", 64, dict(window=50, softcap=30.0)),
                                         ("bf16", 128, dict(starts=True)), ("f16", 256, {})])
def test_prompt_then_steps_then_drafts(pkg, kv, hd, rules):
    """What a server does: prompts of different length, single steps captured once and replayed while the
    positions advance on the device, then a few draft rows at once -- each answer against the 64-bit
    attention over the rows that were appended."""
    import torch
    n_kv, group, page, max_pages = 2, 4, 16, 12
    n_head = n_kv * group
    new = (33, 1, 70)
    n_seq = 3
    n_pages = n_seq * max_pages
    rng = np.random.default_rng(5)
    dt = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.uint8}[kv]
    pools = [torch.zeros(n_pages, page, n_kv, hd, dtype=dt, device="cuda") for _ in range(2)]
    if kv == "e4m3":
        pools = [p.view(torch.float8_e4m3fn) for p in pools]
    scales = [torch.zeros(n_pages, n_kv, device="cuda") if kv == "e4m3" else None for _ in range(2)]
    cache = pkg.PagedCache(pools[0], pools[1], scales[0], scales[1])
    ids = rng.permutation(n_pages).reshape(n_seq, max_pages).astype(np.int32)
    table = tt(ids)
    rope = pkg.Rope(hd, interleaved=True)
    dev = dict(rules)
    host = dict(rules)
    if rules.get("starts"):
        host["starts"] = [3, 0, 64]
        dev["starts"] = tt(np.int32(host["starts"]))

    def rows(i, n):
        out = []
        for s in range(n_seq):
            p = pools[i]
            if kv == "e4m3":
                x = ref.VALUES[p.view(torch.uint8).cpu().numpy()[ids[s]]]
                x = x * scales[i].double().cpu().numpy()[ids[s]][:, None, :, None]
            else:
                x = p.double().cpu().numpy()[ids[s]]
            out.append(x.reshape(-1, n_kv, hd)[:n[s]])
        return out

    def check_rows(q, out, n):
        want, bound = ref.attend(q.double().cpu().numpy(), rows(0, n), rows(1, n), None, hd ** -0.5,
                                 eps_pair=EPS_PAIR[kv], **host)
        check(out, want, bound, "rows %s" % (n,))

    t = sum(new)
    x = [tt(rng.standard_normal((t, h, hd)).astype(np.float32)).bfloat16() for h in (n_head, n_kv, n_kv)]
    pos = tt(np.int32([n - 1 for n in new]))
    pkg.rope_append(cache, table, pos, x[1], x[2], q=x[0], rope=rope, cu_tokens=tt(np.int32(np.cumsum((0,) + new))))
    # the key of the first prompt's row 20 is the rotated one
    want = ref.rotate(x[1].double().cpu().numpy()[20:21], [20], ref.frequencies(hd, 10000.0), True)[0]
    got = rows(0, list(new))[0][20]
    assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -4 + 0.02).all()

    xs = [torch.zeros(n_seq, h, hd, device="cuda") for h in (n_head, n_kv, n_kv)]
    q_rot, out = torch.zeros(n_seq, n_head, hd, device="cuda"), torch.zeros(n_seq, n_head, hd, device="cuda")

    def step():
        pos.add_(1)
        pkg.rope_append(cache, table, pos, xs[1], xs[2], q=xs[0], q_out=q_rot, rope=rope)
        pkg.paged_decode_attention(cache, table, pos, q_rot, out=out, **dev)

    n = list(new)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    n = [a + 1 for a in n]
    check_rows(q_rot[:, None], out[:, None], n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(20):
        for a in xs:
            a.copy_(tt(rng.standard_normal(tuple(a.shape)).astype(np.float32) * (1 + i % 4)))
        graph.replay()
        torch.cuda.synchronize()
        n = [a + 1 for a in n]
        if i % 5 == 0 or i == 19:
            check_rows(q_rot[:, None], out[:, None], n)
    # three draft rows a sequence at once
    xs3 = [tt(rng.standard_normal((n_seq * 3, h, hd)).astype(np.float32)) for h in (n_head, n_kv, n_kv)]
    pos.add_(3)
    q3 = pkg.rope_append(cache, table, pos, xs3[1], xs3[2], q=xs3[0], rope=rope).view(n_seq, 3, n_head, hd)
    o3 = pkg.paged_decode_attention(cache, table, pos, q3, **dev)
    n = [a + 3 for a in n]
    check_rows(q3, o3, n)
    assert pkg.attn_read_device_error() == 0


def test_two_graphs_at_once(pkg):
    """Two captured calls replayed on two streams at the same time hold workspaces of their own."""
    import torch
    pools = [Pool(20 + i, "e4m3", 2, 128, 64, (3000, 100)) for i in range(2)]
    calls = []
    for i, pool in enumerate(pools):
        cache, table = pool.cache(pkg), tt(pool.table)
        pos = tt(np.int32([2999, 99]))
        q = tt(np.random.default_rng(i).standard_normal((2, 8, 128)).astype(np.float32))
        out = torch.zeros_like(q)
        want = pkg.paged_decode_attention(cache, table, pos, q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkg.paged_decode_attention(cache, table, pos, q, out=out)
        calls.append((g, out, want, (cache, table, pos, q)))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(50):
        for (g, _, _, _), s in zip(calls, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, out, want, _ in calls:
        assert torch.equal(out, want)


def test_a_stream_of_the_callers(pkg):
    import torch
    pool = Pool(30, "f16", 2, 128, 16, (100,))
    cache, table, pos = pool.cache(pkg), tt(pool.table), tt(np.int32([99]))
    q = tt(np.random.default_rng(0).standard_normal((1, 8, 128)).astype(np.float32))
    want = pkg.paged_decode_attention(cache, table, pos, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = pkg.paged_decode_attention(cache, table, pos, q, stream=s)
        k = torch.ones(1, 2, 128, device="cuda")
        pkg.rope_append(cache, table, pos, k, k, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    assert bool((pool.dev[0][pool.table[0, 6], 99 % 16] == 1).all())
    with pytest.raises(ValueError):
        pkg.paged_decode_attention(cache, table, pos, q, stream=s)


# ---------------------------------------------------------------------------
# What an append finds in a page, angles at their borders, weights of small scales.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n_kv", [1, 40])             # K and V in jobs of their own, or together
def test_append_onto_pages_of_any_scale(pkg, n_kv, interleaved):
    """Pages filled elsewhere, with scales of 0, negative or no power of two, get a row: the rows that they
    hold keep their values, as near as a code at the new scale comes. With old scale o and the rows' own
    smallest power of two n, the new scale is max(|o|, n) and each kept code the rounding of value * (o / new),
    a product rounded to 32 bits."""
    import torch
    rng = np.random.default_rng(n_kv)
    old = np.float32([0.0, -0.0, -0.5, -0.3, 0.3, 7.0, -7.0, 2.0 ** -60, -2.0 ** -60, 2.0 ** 60, -2.0 ** 60, 0.25, 1e-3])
    n, hd, page, at = len(old), 64, 16, 5
    for size in (1e-4, 100.0, 1e5):
        x = np.clip(rng.standard_normal((n, n_kv, hd)), -3, 3).astype(np.float32) * np.float32(size)
        codes = [rng.integers(0, 256, (n, page, n_kv, hd)).astype(np.uint8) for _ in range(2)]
        scales = [np.repeat(old[:, None], n_kv, 1), np.repeat(np.roll(old, 3)[:, None], n_kv, 1)]
        dev, dsc = [tt(c) for c in codes], [tt(s) for s in scales]
        cache = pkg.PagedCache(dev[0].view(torch.float8_e4m3fn), dev[1].view(torch.float8_e4m3fn), *dsc)
        table = tt(np.arange(n, dtype=np.int32)[:, None])
        # position 0 turns nothing but goes through the rotation: the angle of the row's own position is 0
        rope = pkg.Rope(hd, interleaved=interleaved)
        rope.steps.zero_()
        pkg.rope_append(cache, table, tt(np.full(n, at, np.int32)), tt(x), tt(-x), rope=rope)
        for i, rows in ((0, x), (1, -x)):
            want, now = codes[i].copy(), np.zeros((n, n_kv), np.float32)
            for p in range(n):
                for h in range(n_kv):
                    o = scales[i][p, h]
                    now[p, h] = max(abs(o), np.float32(ref.scale_for(float(np.abs(rows[p, h]).max()))))
                    kept = np.float32(ref.VALUES[codes[i][p, :at, h]]) * np.float32(o / now[p, h])
                    new = ref.to_e4m3(kept)
                    # a NaN code stays one, whatever its sign
                    nan = np.isnan(ref.VALUES[codes[i][p, :at, h]])
                    want[p, :at, h] = np.where(nan, 0x7F, new)
                    want[p, at, h] = ref.to_e4m3(rows[p, h] / now[p, h])
            got = dev[i].cpu().numpy()
            was_nan = (codes[i] & 0x7F) == 0x7F
            was_nan[:, at:] = False
            got = np.where(was_nan & ((got & 0x7F) == 0x7F), 0x7F, got)
            # nothing to rescale: the codes are left as they are
            same = (now == scales[i])[:, None, :, None] & (np.arange(page) < at)[None, :, None, None]
            want = np.where(same & ~was_nan, codes[i], want)
            np.testing.assert_array_equal(dsc[i].cpu().numpy(), now)
            zero = lambda c: np.where((c & 0x7F) == 0, 0, c)                # the sign of a 0 is not looked at
            np.testing.assert_array_equal(zero(got), zero(want), err_msg="size %g, tensor %d" % (size, i))
    assert pkg.attn_read_device_error() == 0


def test_angles_at_every_border(pkg):
    """A step of any 64-bit number at position 1: the angle is that number of 2^-64 turns, also beside the
    eighths of a turn where the kernel goes from one quarter to the next."""
    import torch
    edges = [(e << 61) + d for e in range(8) for d in (-(1 << 33), -(1 << 32), -1, 0, 1, 1 << 32, 1 << 33)]
    steps = [e % (1 << 64) for e in edges] + [0x5A << 56, 0x6B << 56, 0x7F << 56, 0xE1 << 56, 3, (1 << 64) - 3] * 2
    steps = (steps + [0] * 128)[:128]
    rope = pkg.Rope(256)
    rope.steps.copy_(torch.tensor([s - (1 << 64) if s >> 63 else s for s in steps]))
    pool = Pool(0, "f16", 1, 256, 16, (16,))
    q = np.zeros((1, 1, 256), np.float32)
    q[..., :128] = 1.0                                     # (1, 0) turned is (cos, sin)
    k = torch.zeros(1, 1, 256, device="cuda")
    for pos in (1, 3, 5):
        out = pkg.rope_append(pool.cache(pkg), tt(pool.table), tt(np.int32([pos])), k, k, q=tt(q), rope=rope)
        turns = np.array([(pos * s % 2 ** 64) / 2.0 ** 64 for s in steps])
        want = np.concatenate([np.cos(2 * np.pi * turns), np.sin(2 * np.pi * turns)])[None, None]
        # 2 pi 2^-32 for the half of the angle that is left off; three roundings of the remainder of at most pi / 4
        # (to 24 bits, the constant, their product: 2^-24 of it each); the series: half a 2^-24 for the result (at most
        # 1) and, for the terms added to x or 1 before (together below 0.5, four roundings each), 1.5 times 2^-24
        bound = 2 * np.pi * 2.0 ** -32 + 3 * np.pi / 4 * 2.0 ** -24 + 2 * 2.0 ** -24
        check(out, want, np.full(want.shape, bound), "pos %d" % pos)


@pytest.mark.parametrize("spread", [0, 8, 20, 28])
@pytest.mark.parametrize("hd,n_q,group", [(64, 1, 4), (128, 1, 8), (128, 3, 4), (256, 2, 8)])
def test_weights_under_small_scales_by_dimension(pkg, spread, hd, n_q, group):
    """Dimensions that only pages of a small V scale fill, beside pages of a scale 2^spread times as large
    that hold 0 there. A row's weight times its V scale is carried to 2^-22 of itself or 2^-31 of the largest
    such product (the f16 parts end at 2^-25, the largest lies at 2^6 or above), so that, with w the
    normalised weights and d the error of a score, a dimension is off by at most
        (e^2d - 1 + 2^-22 + 2^-21 + 2^-20) sum_j w_j |v_j|  +  2^-31 max_j(w_j vs_j) sum_j |code_j|,
    2^-21 for the exponential and 2^-20 for the sums."""
    page, ctx, n_kv = 16, 96, 2
    pool = Pool(60 + spread, "e4m3", n_kv, hd, page, (ctx,))
    rng = np.random.default_rng(spread)
    small = pool.table[0, 1::2]
    small = small[(small >= 0) & (small < pool.n_pages)]
    large = pool.table[0, 0:ctx // page:2]
    # scores of about 1, so that pages of both kinds weigh
    kc = ref.to_e4m3(rng.standard_normal(pool.host[0].shape) * 20)
    pool.host[0], pool.scale[0] = kc, np.full(pool.scale[0].shape, 2.0 ** -4)
    codes = pool.host[1]
    codes[large, :, :, hd // 2:] = 0
    codes[small, :, :, hd // 2:] = ref.to_e4m3(rng.uniform(50, 400, codes[small, :, :, hd // 2:].shape))
    pool.scale[1] = np.ones_like(pool.scale[1])
    pool.scale[1][small] = 2.0 ** -spread
    import torch
    pool.dev = [tt(c).view(torch.float8_e4m3fn) for c in pool.host]
    pool.dscale = [tt(c.astype(np.float32)) for c in pool.scale]
    n_head = n_kv * group
    q = rng.standard_normal((1, n_q, n_head, hd)).astype(np.float32)
    out = pkg.paged_decode_attention(pool.cache(pkg), tt(pool.table), tt(np.int32([ctx - 1])), tt(q))
    k, v = pool.rows(0)[0], pool.rows(1)[0]
    vs = np.repeat(pool.scale[1][pool.table[0, :ctx // page]], page, 0)
    want, bound = np.zeros(q.shape), np.zeros(q.shape)
    for t in range(n_q):
        seen = ctx - n_q + t + 1
        for h in range(n_head):
            x, kk, vv, s = q[0, t, h].astype(np.float64), k[:seen, h // group], v[:seen, h // group], vs[:seen, h // group]
            sc = kk @ x * hd ** -0.5
            mag = (np.abs(kk) @ np.abs(x)).max() * hd ** -0.5
            d = mag * (2.0 ** -22 + (hd / 16 + 4) * 2.0 ** -23) + 2.0 ** -22 * np.abs(sc).max()
            w = np.exp(sc - sc.max())
            w /= w.sum()
            want[0, t, h] = w @ vv
            bound[0, t, h] = (math.expm1(2 * d) + 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -20) * (w @ np.abs(vv)) + \
                2.0 ** -31 * (w * s).max() * np.abs(vv / s[:, None]).sum(0)
    check(out, want, bound, "spread %d" % spread)
    assert pkg.attn_read_device_error() == 0


def test_the_public_names_of_torch(pkg, monkeypatch):
    """Where torch lacks the short ways to its allocator, device and stream, their public names give the same,
    eagerly, on another stream and in a captured graph."""
    import torch
    pool = Pool(61, "e4m3", 2, 128, 64, (3000, 5))
    cache, table, pos = pool.cache(pkg), tt(pool.table), tt(np.int32([2999, 4]))
    q = tt(np.random.default_rng(1).standard_normal((2, 8, 128)).astype(np.float32))
    want = pkg.paged_decode_attention(cache, table, pos, q)
    short = {n: getattr(pkg, n) for n in ("_torch", "_alloc", "_free", "_device", "_raw_stream")}
    try:
        with monkeypatch.context() as m:
            m.setattr(torch, "_C", object())
            pkg._torch = None
            pkg._torch_module()
        assert pkg._device is torch.cuda.current_device and pkg._free is torch.cuda.caching_allocator_delete
        assert pkg._alloc.__module__ == pkg._raw_stream.__module__ == pkg.__name__
        assert torch.equal(pkg.paged_decode_attention(cache, table, pos, q), want)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = pkg.paged_decode_attention(cache, table, pos, q)
        side.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = pkg.paged_decode_attention(cache, table, pos, q)
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    finally:
        for n, f in short.items():
            setattr(pkg, n, f)
    assert pkg.attn_read_device_error() == 0


@pytest.mark.parametrize("hd,rot,page,n_kv,interleaved", [(128, 128, 64, 2, False), (64, 64, 1024, 1, True),
                                                          (256, 64, 128, 8, False)])
def test_a_prompt_at_once_or_row_by_row(pkg, hd, rot, page, n_kv, interleaved):
    """The pages hold the same scales and V codes either way, where no row needs a larger scale than the first
    of its page. K too, but for elements so near to the middle of two codes that the rotations' rounding decides:
    a row by itself is turned by its own angle (a sine and cosine within 4.4 2^-24 + 2 pi 2^-32), of a page's rows three
    in four by the row before's and a fixed step. As complex numbers both are off by 6.3 2^-24, each of three
    products adds as much and 1.4 2^-24 of rounding, the rotation itself 1.4 2^-24: 31 2^-24 of the pair's magnitude,
    which is at most sqrt 2 times the row's largest element -- 11 2^-22 of it."""
    import torch
    n = 2 * page + 7
    x = np.random.default_rng(page).standard_normal((2, n, n_kv, hd)).astype(np.float32)
    x[:, ::page] *= 4 / np.abs(x[:, ::page]).max(-1, keepdims=True)
    x[:, ::page, :, 0] = 6                     # turned, at least 6 / sqrt 2; the other rows at most 2 sqrt 2
    y = np.clip(x, -2, 2)
    y[:, ::page] = x[:, ::page]
    k, v = tt(y[0]), tt(y[1])
    table = tt(np.arange(3, dtype=np.int32)[None])
    rope = pkg.Rope(rot, interleaved=interleaved)
    got = []
    for steps in ([n], [1] * n):
        pools = [torch.zeros(3, page, n_kv, hd, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(3, n_kv, device="cuda") for _ in range(2)]
        cache = pkg.PagedCache(*[p.view(torch.float8_e4m3fn) for p in pools], *scales)
        at = 0
        for m in steps:
            pkg.rope_append(cache, table, tt(np.int32([at + m - 1])), k[at:at + m], v[at:at + m], rope=rope)
            at += m
        got.append([t.cpu().numpy() for t in pools + scales])
    (ka, va, *sa), (kb, vb, *sb) = got
    np.testing.assert_array_equal(va, vb)
    np.testing.assert_array_equal(np.stack(sa), np.stack(sb))
    a, b = (ref.VALUES[c.reshape(-1, n_kv, hd)[:n]] for c in (ka, kb))
    scale = np.repeat(sa[0].astype(np.float64), page, 0)[:n, :, None]
    freq = np.array([2 * math.pi * s / 2.0 ** 64 for s in pkg.attn_rope_steps(rot, 10000.0)])
    want = ref.rotate(y[0].astype(np.float64), np.arange(n), freq, interleaved) / scale
    far = np.abs(want - (a + b) / 2) > 11 * 2.0 ** -22 * np.abs(y[0]).max(-1, keepdims=True) / scale
    assert not (far & (a != b)).any()
    assert (np.abs(a - b) <= np.maximum(np.abs(want) * 2.0 ** -3 * (1 + 2.0 ** -4), 2.0 ** -9)).all()
    assert pkg.attn_read_device_error() == 0
