"""Trees and page bookkeeping without a GPU: refusals of the C entry points (all before any CUDA call) and of the torch
forms, plans for a given SM count, and the restatement that the GPU tests compare with, against closed forms."""
import ctypes
import math
import re

import numpy as np
import pytest

import decode_attention_gqa_gb300 as pkg
import tree_reference as tree
from decode_attention_gqa_gb300 import build as cuda_build
from test_paged_host import CACHE_FAULTS, _addr, _cache, _pool_and_ids, door     # noqa: F401  (door is a fixture)

INVALID, UNSUPPORTED, OK = pkg.ATTN_ERR_INVALID_ARG, pkg.ATTN_ERR_UNSUPPORTED, pkg.ATTN_OK
F32, F16, BF16, E4M3 = range(4)


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return pkg.load()


def _rules(lib, **kw):
    a = dict(parents=16, cu=None, n_seq=1, n_tokens=4, most=4, mask=16, depths=16)
    a.update(kw)
    return lib.attn_tree_rules(a["parents"], a["cu"], a["n_seq"], a["n_tokens"], a["most"], a["mask"], a["depths"], None)


def _tree(lib, cache=None, rules=None, **kw):
    a = dict(table=16, max_pages=8, pos=16, cu=None, n_seq=1, n_tokens=4, most=4, q=16, out=16, q_type=F32, n_head=8,
             scale=0.1, mask=16, words=1, depths=16, P=0, ws=None, ws_bytes=0)
    a.update(kw)
    c = cache if cache is not None else _cache()
    return lib.attn_decode_tree(_addr(c), a["table"], a["max_pages"], a["pos"], a["cu"], a["n_seq"], a["n_tokens"], a["most"],
                                a["q"], a["out"], a["q_type"], a["n_head"], a["scale"], a["mask"], a["words"], a["depths"],
                                _addr(rules), a["P"], a["ws"], a["ws_bytes"], None)


def _append(lib, cache=None, **kw):
    a = dict(table=16, max_pages=8, pos=16, cu=None, n_seq=1, n_tokens=1, q=16, k=16, v=16, qs=0, ks=0, vs=0, t=F16, q_out=32,
             out_type=F32, n_head=8, depths=16)
    a.update(kw)
    c = cache if cache is not None else _cache()
    return lib.attn_rope_append_tree(_addr(c), a["table"], a["max_pages"], a["pos"], a["cu"], a["n_seq"], a["n_tokens"],
                                     a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["t"], a["q_out"], a["out_type"],
                                     a["n_head"], None, a["depths"], None)


def _keep(lib, cache=None, **kw):
    a = dict(table=16, max_pages=8, base=16, path=16, counts=16, n_seq=1, most=4)
    a.update(kw)
    c = cache if cache is not None else _cache()
    return lib.attn_keep_rows(_addr(c), a["table"], a["max_pages"], a["base"], a["path"], a["counts"], a["n_seq"], a["most"],
                              None)


def _resize(lib, **kw):
    a = dict(refs=16, n_pages=4, table=16, max_pages=8, page=16, have=16, want=16, n_seq=1)
    a.update(kw)
    return lib.attn_pages_resize(a["refs"], a["n_pages"], a["table"], a["max_pages"], a["page"], a["have"], a["want"],
                                 a["n_seq"], None)


def _fork(lib, **kw):
    a = dict(refs=16, n_pages=4, table=16, max_pages=8, page=16, n_seq=2, src=16, dst=16, rows=16, n=1, copies=16)
    a.update(kw)
    return lib.attn_pages_fork(a["refs"], a["n_pages"], a["table"], a["max_pages"], a["page"], a["n_seq"], a["src"], a["dst"],
                               a["rows"], a["n"], a["copies"], None)


@pytest.mark.parametrize("fault,want", CACHE_FAULTS)
def test_a_wrong_pool_is_refused(lib, fault, want):
    c = _cache(**fault)
    assert _tree(lib, c) == want
    assert _append(lib, c) == want
    assert _keep(lib, c) == want
    assert lib.attn_pages_copy(_addr(c), 16, 1, None) == want


def test_rules_refuse_wrong_arguments(lib):
    for kw in (dict(parents=None), dict(mask=None), dict(depths=None), dict(parents=2), dict(mask=6), dict(depths=1),
               dict(cu=2), dict(n_seq=-1), dict(n_seq=70000), dict(n_tokens=-1), dict(n_tokens=1 << 31), dict(most=0),
               dict(most=1025), dict(n_seq=3), dict(n_seq=0), dict(most=3), dict(n_seq=0, cu=16)):
        assert _rules(lib, **kw) == INVALID, kw
    assert _rules(lib, n_tokens=0, parents=None, mask=None, depths=None) == OK
    assert _rules(lib, n_seq=0, n_tokens=0) == OK


def test_attention_refuses_wrong_arguments(lib):
    assert lib.attn_decode_tree(None, 16, 8, 16, None, 1, 1, 1, 16, 16, 0, 8, 0.1, None, 0, None, None, 0, None, 0, None) == INVALID
    for kw in (dict(table=None), dict(pos=None), dict(q=None), dict(out=None), dict(q=8), dict(out=20), dict(table=18),
               dict(pos=17), dict(mask=2), dict(depths=6), dict(cu=1), dict(max_pages=0), dict(max_pages=1 << 26),
               dict(n_seq=-1), dict(n_seq=70000), dict(n_seq=3), dict(n_seq=0), dict(n_tokens=-4), dict(n_tokens=1 << 31),
               dict(most=0), dict(most=3), dict(most=1025), dict(most=33), dict(words=0), dict(words=1025), dict(q_type=E4M3),
               dict(q_type=-1), dict(n_head=0), dict(n_head=7), dict(n_head=70000), dict(scale=math.nan),
               dict(scale=math.inf), dict(P=-1), dict(P=5000), dict(ws=128)):
        assert _tree(lib, **kw) == INVALID, kw
    assert _tree(lib, n_head=130) == UNSUPPORTED                        # 65 query heads a KV head
    assert _tree(lib, scale=3e38) == INVALID                            # past 32 bits with log2 e
    assert _tree(lib, scale=1e30, rules=pkg._RulesStruct(1e-10, 0, 0, 0)) == INVALID
    for r in ((-1.0, 0, 0, 0), (math.nan, 0, 0, 0), (math.inf, 0, 0, 0), (0.0, -1, 0, 0), (0.0, 0, 2, 0),
              (0.0, 0, 0, 3), (1e-20, 0, 0, 0), (1e30, 0, 0, 0)):
        assert _tree(lib, rules=pkg._RulesStruct(*r)) == INVALID, r
    # distances need the nodes' depths; a chain has them
    assert _tree(lib, depths=None, rules=pkg._RulesStruct(0.0, 5, 0, 0)) == INVALID
    assert _tree(lib, depths=None, rules=pkg._RulesStruct(0.0, 0, 16, 0)) == INVALID
    assert _tree(lib, n_tokens=0, n_seq=0, table=None, pos=None, q=None, out=None, mask=None, depths=None) == OK
    assert _tree(lib, n_tokens=0) == OK


def test_append_refuses_wrong_arguments(lib):
    for kw in (dict(depths=2), dict(out_type=BF16), dict(out_type=E4M3), dict(out_type=-1), dict(t=F32, out_type=F16),
               dict(table=None), dict(q_out=None), dict(k=8), dict(n_seq=2, n_tokens=3), dict(q=32), dict(q=32, t=F32, qs=1032)):
        assert _append(lib, **kw) == INVALID, kw
    assert _append(lib, n_tokens=0, n_seq=0, table=None, pos=None, k=None, v=None) == OK


def test_keep_refuses_wrong_arguments(lib):
    for kw in (dict(table=None), dict(base=None), dict(path=None), dict(counts=None), dict(table=2), dict(base=1), dict(path=6),
               dict(counts=3), dict(n_seq=-1), dict(n_seq=70000), dict(most=-1), dict(max_pages=0)):
        assert _keep(lib, **kw) == INVALID, kw
    assert _keep(lib, n_seq=0, table=None, base=None, path=None, counts=None) == OK
    assert _keep(lib, most=0, path=None) == OK


def test_bookkeeping_refuses_wrong_arguments(lib):
    for kw in (dict(refs=None), dict(table=None), dict(have=None), dict(want=None), dict(refs=8), dict(table=2), dict(have=1),
               dict(want=2), dict(n_pages=0), dict(max_pages=0), dict(max_pages=1 << 27), dict(page=0), dict(page=8),
               dict(page=24), dict(page=1040), dict(n_seq=-1), dict(n_seq=70000)):
        assert _resize(lib, **kw) == INVALID, kw
    assert _resize(lib, n_seq=8193) == UNSUPPORTED
    assert _resize(lib, n_seq=0, refs=None, table=None, have=None, want=None) == OK
    for kw in (dict(refs=None), dict(table=None), dict(src=None), dict(dst=None), dict(rows=None), dict(copies=None),
               dict(refs=8), dict(table=2), dict(src=1), dict(dst=2), dict(rows=3), dict(copies=8), dict(n_pages=0),
               dict(max_pages=0), dict(page=24), dict(n_seq=-1), dict(n=-1)):
        assert _fork(lib, **kw) == INVALID, kw
    assert _fork(lib, n=4097) == UNSUPPORTED
    assert _fork(lib, n=0, refs=None, table=None, src=None, dst=None, rows=None, copies=None) == OK
    for kw in ((None, 1), (8, 1), (16, -1)):
        assert lib.attn_pages_copy(_addr(_cache()), *kw, None) == INVALID
    assert lib.attn_pages_copy(_addr(_cache()), None, 0, None) == OK


def test_bookkeeping_of_more_pages_than_it_counts_is_refused(lib):
    assert _resize(lib, n_pages=(1 << 30) + 1) == UNSUPPORTED
    assert _fork(lib, n_pages=(1 << 31) - 1) == UNSUPPORTED


def test_resizing_a_table_of_more_entries_than_it_counts_is_refused(lib):
    """What all sequences ask for is summed in 32 bits."""
    assert _resize(lib, n_seq=8192, max_pages=1 << 18) == UNSUPPORTED
    assert _resize(lib, n_seq=17, max_pages=(1 << 27) - 1025) == UNSUPPORTED


@pytest.mark.parametrize("hd,nodes,splits,workspace", [
    # 8 KV heads, groups of 4: 128 slots hold 32 nodes; an SM a block, 152 of them
    (128, 32, 19, 19 * 2 * 8 * 128 * (128 + 2) * 4 + 256),
    (128, 33, 9, 9 * 2 * 16 * 128 * (128 + 2) * 4 + 256),
    (256, 200, 10, 10 * 2 * 56 * 128 * (256 + 2) * 4 + 256),     # 56 units: two rounds' worth would leave a quarter idle: four rounds
])
def test_plan_fills_the_sms(hd, nodes, splits, workspace):
    """152 SMs, two sequences of up to 65536 rows."""
    c = _cache(head_dim=hd, n_kv_head=8)
    got = pkg.attn_tree_plan(ctypes.addressof(c), 65536 // c.page_size, 2, 2 * nodes, nodes, F16, 32, sm_count=152)
    assert tuple(got) == (splits, workspace)


@pytest.mark.parametrize("kv,q,hd,rows,workspace", [
    (E4M3, F32, 128, 4096, 16 * 128 * 128 * 4), (E4M3, F32, 128, 2048, 0), (F16, F32, 256, 2112, 16 * 128 * 256 * 4),
    (BF16, F32, 64, 2176, 16 * 128 * 64 * 4), (E4M3, F16, 128, 65536, 0), (BF16, BF16, 128, 65536, 0), (BF16, F16, 128, 16384, 0),
    (BF16, F16, 128, 32768, 16 * 128 * 128 * 4)])
def test_plan_of_one_split_has_room_for_sums_on_the_way(kv, q, hd, rows, workspace):
    """8 KV heads, 33 nodes of groups of 4: 16 units, a sum of 128 rows of f32 each where more rows than 2048 are added up
    (f16 queries over bf16: 16384)."""
    c = _cache(head_dim=hd, n_kv_head=8, kv_type=kv, page_size=64)
    got = pkg.attn_tree_plan(ctypes.addressof(c), rows // 64, 2, 66, 33, q, 32, 1, sm_count=152)
    assert tuple(got) == (1, workspace)


def test_plan_refuses_what_the_call_does():
    def plan(cache=None, max_pages=8, n_seq=1, n_tokens=4, most=4, q_type=F32, n_head=8, P=0):
        c = cache or _cache()
        return pkg.attn_tree_plan(ctypes.addressof(c), max_pages, n_seq, n_tokens, most, q_type, n_head, P, 152)
    assert plan()[0] >= 1
    for kw, st in ((dict(n_seq=0), INVALID), (dict(n_tokens=0), INVALID), (dict(most=0), INVALID), (dict(most=1025), INVALID),
                   (dict(n_head=3), INVALID), (dict(q_type=3), INVALID), (dict(P=-2), INVALID), (dict(n_head=130), UNSUPPORTED),
                   (dict(cache=_cache(head_dim=32)), UNSUPPORTED), (dict(max_pages=0), INVALID)):
        with pytest.raises(pkg.AttnError) as e:
            plan(**kw)
        assert e.value.status == st, kw


def test_torch_forms_refuse_before_any_call():
    torch = pytest.importorskip("torch")
    i32 = dict(dtype=torch.int32)
    k = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    cache = pkg.PagedCache(k, k.clone())
    table, pos = torch.zeros(2, 2, **i32), torch.zeros(2, **i32)
    with pytest.raises(ValueError):
        pkg.tree_rules(torch.zeros(2, 3, **i32))                        # not on a GPU
    with pytest.raises(ValueError):
        pkg.keep_rows(cache, table, pos, torch.zeros(2, 3, **i32), pos)
    with pytest.raises(ValueError):
        pkg.copy_pages(cache, torch.zeros(2, 4, **i32))
    with pytest.raises(ValueError):
        pkg.PageBook(torch.zeros(4, **i32), table, 16)
    q = torch.zeros(4, 4, 64)
    for args, kw, err in (((q,), {}, ValueError), ((q.double(),), {}, TypeError), ((q.half()[0],), {}, ValueError),
                          ((torch.zeros(2, 2, 4, 64),), dict(cu_tokens=pos), ValueError)):
        with pytest.raises(err):
            pkg.tree_decode_attention(cache, table, pos, *args, **kw)
    with pytest.raises(ValueError):
        pkg.rope_append(cache, table, pos, torch.zeros(2, 2, 64), torch.zeros(2, 2, 64), depths=torch.zeros(2, **i32))


def test_a_window_is_refused_whatever_was_called_before(door):     # noqa: F811
    """The plan does not depend on the window, so a call of the same shape must not let one past 32 bits through, which would
    arrive as another: 2^32 as none."""
    import torch
    cache, table, pos = _pool_and_ids()
    q = torch.zeros(3, 4, 64)
    for _ in range(2):
        n = len(door.calls)
        for window in (2 ** 31, 2 ** 32, 2 ** 32 + 16, -1, -2 ** 32):
            with pytest.raises(ValueError, match="window"):
                pkg.tree_decode_attention(cache, table, pos, q, window=window)
        assert len(door.calls) == n
        pkg.tree_decode_attention(cache, table, pos, q)
        pkg.tree_decode_attention(cache, table, pos, q, window=2 ** 31 - 1)
        assert door.calls[-1][0] == "attn_decode_tree"


def test_a_mask_of_too_few_words_is_refused(door):                # noqa: F811
    """One of no words has no address, and would stand for chains."""
    import torch
    cache, table, pos = _pool_and_ids()
    i32 = dict(dtype=torch.int32)
    depths = torch.zeros(33, **i32)
    for mask in (torch.zeros(33, 0, **i32), torch.zeros(33, 1, **i32), torch.zeros(33, **i32)):
        with pytest.raises(ValueError, match="mask"):
            pkg.tree_decode_attention(cache, table, pos, torch.zeros(33, 4, 64), mask=mask, depths=depths)
    assert not door.calls
    pkg.tree_decode_attention(cache, table, pos, torch.zeros(33, 4, 64), mask=torch.zeros(33, 2, **i32), depths=depths)
    assert door.calls[-1][1][13] and door.calls[-1][1][14] == 2


def test_headers_and_binding_agree(lib):
    text = "".join(open(cuda_build.ROOT + "/include/%s.h" % h).read() for h in ("attn_tree", "attn_pages"))
    for name, value in re.findall(r"#define (ATTN_\w+) (0x[0-9A-Fa-f]+)u", text):
        assert getattr(pkg, name) == int(value, 16)
    names = re.findall(r"^attn_status (attn_\w+)\(", text, re.M)
    assert len(names) == 8
    for n in names:
        assert hasattr(lib, n) and callable(getattr(pkg, n)) and n in pkg.__all__


def test_the_restatement_of_rules():
    sees, depths, wrong = tree.rules([-1, 0, 0, 1, -1, 4])
    assert sees == [[0], [1, 0], [2, 0], [3, 1, 0], [4], [5, 4]] and depths == [0, 1, 1, 2, 0, 1] and not wrong
    assert tree.rules([1, 0])[2] and tree.rules([2, -1])[2]
    w = tree.words([[0, 31, 32, 63]], 2).view(np.uint32)
    assert w.tolist() == [[1 | 1 << 31, 1 | 1 << 31]]


def test_the_restatement_of_attention():
    """One visible row gives that row; equal keys give the mean of the visible rows; a chain of one node sees all."""
    rng = np.random.default_rng(0)
    k, v = np.ones((6, 1, 8)), rng.standard_normal((6, 1, 8))
    q = [rng.standard_normal((3, 2, 8))]
    out, bound = tree.attend(q, [[[0], [0, 1], [2]]], [[0, 1, 0]], [k], [v], 1.0, "f16", "f32")
    np.testing.assert_allclose(out[0][1, 0], v[[0, 1, 2, 3, 4], 0].mean(0))
    np.testing.assert_allclose(out[0][2, 1], v[[0, 1, 2, 5], 0].mean(0))
    out, _ = tree.attend(q, [[[0], [0, 1], [2]]], [[0, 1, 0]], [k], [v], 1.0, "f16", "f32", window=1)
    np.testing.assert_allclose(out[0][1, 0], v[4, 0])
    np.testing.assert_allclose(out[0][2, 0], v[5, 0])
    out, _ = tree.attend(q, [[[], [0, 1], [2]]], [[0, 1, 0]], [k], [v], 1.0, "f16", "f32", starts=[4])
    assert (out[0][0] == 0).all()
    np.testing.assert_allclose(out[0][1, 0], v[4, 0])
    assert (bound[0] >= 0).all()


def test_the_restatement_of_bookkeeping():
    refs, table = np.zeros(6, np.int32), np.full((3, 3), -1, np.int32)
    assert tree.resize(refs, table, 16, [0, 0, 0], [40, 16, 0]) == 0
    assert table.tolist() == [[0, 1, 2], [3, -1, -1], [-1, -1, -1]]
    copies, err = tree.fork(refs, table, 16, [0], [2], [40])
    assert err == 0 and copies.tolist() == [[2, 4, 8, 0]] and table[2].tolist() == [0, 1, 4]
    assert refs.tolist() == [2, 2, 1, 1, 1, 0]
    assert tree.resize(refs, table, 16, [40, 16, 40], [0, 48, 40]) == 0
    assert table.tolist() == [[-1] * 3, [3, 2, 5], [0, 1, 4]] and refs.tolist() == [1] * 6
    assert tree.resize(refs, table, 16, [0, 48, 40], [16, 48, 40]) == 16 and table[0, 0] == -1
