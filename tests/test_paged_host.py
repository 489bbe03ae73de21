"""The paged-cache operators without a GPU: refusals of the C entry points (all before any CUDA
call), of the torch forms, the split plan for a given SM count, and the rotary steps."""
import ctypes
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

import decode_attention_gqa_gb300 as pkg
import paged_reference as ref
from decode_attention_gqa_gb300 import build as cuda_build

INVALID, UNSUPPORTED, OK = pkg.ATTN_ERR_INVALID_ARG, pkg.ATTN_ERR_UNSUPPORTED, pkg.ATTN_OK


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return pkg.load()


def _cache(**kw):
    a = dict(k=256, v=256, k_scale=0, v_scale=0, page_stride=0, row_stride=0, head_stride=0, n_pages=4,
             page_size=64, n_kv_head=2, head_dim=128, kv_type=pkg.ATTN_TYPE_F16, reserved=0)
    a.update(kw)
    return pkg._CacheStruct(*[a[n] for n, _ in pkg._CacheStruct._fields_])


def _addr(s):
    return ctypes.addressof(s) if s is not None else None


CACHE_FAULTS = [
    (dict(k=0), INVALID), (dict(v=8), INVALID), (dict(k_scale=256, v_scale=256), INVALID),
    (dict(kv_type=pkg.ATTN_TYPE_E4M3), INVALID),                       # no scales
    (dict(kv_type=pkg.ATTN_TYPE_E4M3, k_scale=256), INVALID),
    (dict(kv_type=pkg.ATTN_TYPE_E4M3, k_scale=256, v_scale=258), INVALID),
    (dict(kv_type=pkg.ATTN_TYPE_F32), INVALID), (dict(kv_type=4), INVALID), (dict(reserved=1), INVALID),
    (dict(n_pages=0), INVALID), (dict(n_kv_head=0), INVALID), (dict(n_kv_head=70000), INVALID),
    (dict(page_size=0), INVALID), (dict(page_size=8), INVALID), (dict(page_size=24), INVALID),
    (dict(page_size=1040), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=8), UNSUPPORTED),
    (dict(head_dim=0), INVALID),
    (dict(page_stride=64 * 256, row_stride=256), INVALID),             # head stride missing
    (dict(page_stride=64 * 256, row_stride=256, head_stride=132), INVALID),      # 264 bytes
    (dict(page_stride=64 * 256, row_stride=-256, head_stride=128), INVALID),
    (dict(page_stride=1 << 40, row_stride=256, head_stride=128), INVALID),
]


def _attend(lib, cache=None, rules=None, **kw):
    a = dict(table=16, max_pages=8, pos=16, q=16, out=16, n_seq=1, n_q=1, n_head=8, scale=0.1, P=0, ws=None,
             ws_bytes=0)
    a.update(kw)
    c = cache if cache is not None else _cache()
    return lib.attn_decode_paged(_addr(c), a["table"], a["max_pages"], a["pos"], a["q"], a["out"], a["n_seq"],
                                 a["n_q"], a["n_head"], a["scale"], _addr(rules), a["P"], a["ws"], a["ws_bytes"],
                                 None)


def _append(lib, cache=None, rope=None, **kw):
    a = dict(table=16, max_pages=8, pos=16, cu=None, n_seq=1, n_tokens=1, q=16, k=16, v=16, qs=0, ks=0, vs=0,
             t=pkg.ATTN_TYPE_F16, q_out=32, n_head=8)
    a.update(kw)
    c = cache if cache is not None else _cache()
    return lib.attn_rope_append(_addr(c), a["table"], a["max_pages"], a["pos"], a["cu"], a["n_seq"], a["n_tokens"],
                                a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["t"], a["q_out"], a["n_head"],
                                _addr(rope), None)


@pytest.mark.parametrize("fault,want", CACHE_FAULTS)
def test_a_wrong_pool_is_refused(lib, fault, want):
    assert _attend(lib, _cache(**fault)) == want
    assert _append(lib, _cache(**fault)) == want


def test_attention_refuses_wrong_arguments(lib):
    assert lib.attn_decode_paged(None, 16, 8, 16, 16, 16, 1, 1, 8, 0.1, None, 0, None, 0, None) == INVALID
    for kw in (dict(table=None), dict(pos=None), dict(q=None), dict(out=None), dict(q=8), dict(out=20),
               dict(table=18), dict(pos=17), dict(max_pages=0), dict(max_pages=1 << 26), dict(n_seq=-1),
               dict(n_seq=70000), dict(n_q=0), dict(n_q=1025), dict(n_head=0), dict(n_head=7),
               dict(scale=math.nan), dict(scale=math.inf), dict(P=-1), dict(P=5000), dict(ws=128)):
        assert _attend(lib, **kw) == INVALID, kw
    assert _attend(lib, n_head=130) == UNSUPPORTED                      # 65 query heads a KV head
    assert _attend(lib, scale=3e38) == INVALID                          # past 32 bits with log2 e
    assert _attend(lib, scale=1e30, rules=pkg._RulesStruct(1e-10, 0, 0, 0)) == INVALID
    for r in ((-1.0, 0, 0, 0), (math.nan, 0, 0, 0), (math.inf, 0, 0, 0), (0.0, -1, 0, 0), (0.0, 0, 2, 0),
              (0.0, 0, 0, 3), (1e-20, 0, 0, 0), (1e30, 0, 0, 0)):
        assert _attend(lib, rules=pkg._RulesStruct(*r)) == INVALID, r
    assert _attend(lib, n_seq=0, table=None, pos=None, q=None, out=None) == OK


def test_append_refuses_wrong_arguments(lib):
    assert lib.attn_rope_append(None, 16, 8, 16, None, 1, 1, 16, 16, 16, 0, 0, 0, 1, 32, 8, None, None) == INVALID
    for kw in (dict(table=None), dict(pos=None), dict(k=None), dict(v=None), dict(q=None), dict(q_out=None),
               dict(k=8), dict(v=4), dict(q=24), dict(q_out=8), dict(cu=2), dict(t=pkg.ATTN_TYPE_E4M3),
               dict(t=9), dict(n_seq=-1), dict(n_seq=70000), dict(n_tokens=-1), dict(n_seq=2, n_tokens=3),
               dict(n_seq=0, n_tokens=1), dict(n_head=0), dict(max_pages=0), dict(qs=100), dict(qs=1028),
               dict(ks=128), dict(vs=260), dict(q=32, q_out=32)):
        assert _append(lib, **kw) == INVALID, kw
    for r in ((0, 128, 0, 1.0, 0), (24, 128, 0, 1.0, 0), (16, 0, 0, 1.0, 0), (16, 24, 0, 1.0, 0),
              (16, 144, 0, 1.0, 0), (16, 128, 2, 1.0, 0), (16, 128, 0, math.nan, 0), (16, 128, 0, 1.0, 1)):
        assert _append(lib, rope=pkg._RopeStruct(*r)) == INVALID, r
    assert _append(lib, n_tokens=0, n_seq=0, table=None, pos=None, k=None, v=None) == OK
    assert _append(lib, n_tokens=0, cu=16) == OK


def test_plan_for_a_given_sm_count(lib):
    def plan(cache=None, max_pages=128, n_seq=1, n_q=1, n_head=8, window=0, P=0, sms=152):
        c = cache or _cache()
        return pkg.attn_paged_plan(ctypes.addressof(c), max_pages, n_seq, n_q, n_head, window, P, sms)
    def ws(P, units, slots=8, n_seq=1, hd=128):
        parts = P * 2 * units * slots
        return -(-parts * hd * 4 // 256) * 256 + -(-parts * 8 // 256) * 256 + -(-min(n_seq, 128) * 8 // 256) * 256
    # one sequence, 2 KV heads, 8192 rows: 2 x 152 resident blocks, but no more than there are 64-row tiles
    assert plan() == (128, ws(128, 2))
    assert plan(n_seq=2) == (152, ws(152, 2, n_seq=2))
    assert plan(n_seq=1000) == (152, ws(152, 2, n_seq=1000))
    # a window bounds the rows that a sequence can need, and so the blocks
    assert plan(window=300)[0] < 8 and plan(window=100)[0] == 1
    # 16 (query row, head) slots a block, several blocks a KV head
    assert plan(n_q=4, n_seq=9) == (152, ws(152, 2, 16, 9)) and plan(n_q=12, n_seq=9)[0] == 50
    # 8 bits: 8 slots a block while the blocks have few rows, or 16
    e8 = dict(kv_type=pkg.ATTN_TYPE_E4M3, k_scale=256, v_scale=256)
    assert plan(cache=_cache(**e8), n_q=4, n_seq=3) == (114, ws(114, 4, 8, 3))
    assert plan(cache=_cache(**e8), n_q=4, n_seq=9) == (152, ws(152, 2, 16, 9))
    assert plan(cache=_cache(**e8), n_q=5, n_seq=99) == (76, ws(76, 6, 8, 99))      # 20 slots: the second 16 half empty
    # a third block an SM only where it has more than two tiles
    assert plan(cache=_cache(n_kv_head=4, **e8), n_head=28) == (64, ws(64, 4))
    # units just over half of the resident blocks: four rounds; far more units than blocks: one block each
    assert plan(cache=_cache(n_kv_head=160), n_head=160, n_seq=2)[0] == 7
    assert plan(cache=_cache(n_kv_head=2000), n_head=2000) == (1, 0)
    assert plan(P=7) == (7, ws(7, 2)) and plan(P=1) == (1, 0)
    for kw, st in ((dict(n_seq=0), INVALID), (dict(n_head=3), INVALID), (dict(window=-1), INVALID),
                   (dict(P=-2), INVALID), (dict(n_head=130), UNSUPPORTED),
                   (dict(cache=_cache(head_dim=32)), UNSUPPORTED), (dict(max_pages=0), INVALID)):
        with pytest.raises(pkg.AttnError) as e:
            plan(**kw)
        assert e.value.status == st, kw
    # only the pool's shape is looked at
    assert plan(cache=_cache(k=0, v=0)) == plan()


def test_torch_forms_refuse_wrong_tensors(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    k = torch.zeros(3, 16, 2, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        pkg.PagedCache(k.float(), k.float())
    with pytest.raises(TypeError):
        pkg.PagedCache(k, k.bfloat16())
    with pytest.raises(ValueError):
        pkg.PagedCache(k, torch.zeros(3, 16, 2, 128, dtype=torch.float16))
    with pytest.raises(ValueError):
        pkg.PagedCache(k, torch.zeros(3, 2, 16, 64, dtype=torch.float16).transpose(1, 2))   # other strides
    with pytest.raises(ValueError):
        pkg.PagedCache(k, k.clone(), torch.ones(3, 2), torch.ones(3, 2))                    # scales of a 16-bit cache
    k8 = torch.zeros(3, 16, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        pkg.PagedCache(k8, k8)
    with pytest.raises(ValueError):
        pkg.PagedCache(k8, k8, torch.ones(3, 1), torch.ones(3, 2))
    with pytest.raises(TypeError):
        pkg.PagedCache(k8, k8, torch.ones(3, 2).double(), torch.ones(3, 2))
    c = pkg.PagedCache(k, k.clone())
    table, pos = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64)
    with pytest.raises(ValueError):                                    # host tensors
        pkg.paged_decode_attention(c, table, pos, q)
    with pytest.raises(ValueError):
        pkg.rope_append(c, table, pos, k[0, :1], k[0, :1])
    # the checks behind the device's
    monkeypatch.setattr(pkg, "_same_device", lambda d: None)
    for bad in (dict(q=q.double()), dict(q=q[0]), dict(q=torch.zeros(2, 4, 64)), dict(q=torch.zeros(1, 4, 32)),
                dict(q=torch.zeros(1, 64, 4).transpose(1, 2)), dict(table=table.long()), dict(table=table[0]),
                dict(pos=pos.long()), dict(pos=torch.zeros(2, dtype=torch.int32)), dict(out=torch.zeros(1, 4, 32)),
                dict(out=torch.zeros(1, 4, 64).half()), dict(slopes=torch.zeros(3)), dict(slopes=torch.zeros(4).half()),
                dict(starts=torch.zeros(1)), dict(starts=torch.zeros(2, dtype=torch.int32))):
        a = dict(table=table, pos=pos, q=q)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            pkg.paged_decode_attention(c, a.pop("table"), a.pop("pos"), a.pop("q"), **a)
    x = torch.zeros(1, 2, 64)
    for bad in (dict(k=x.double()), dict(k=x.long()), dict(v=x.half()), dict(v=torch.zeros(2, 2, 64)),
                dict(k=torch.zeros(1, 3, 64)), dict(k=torch.zeros(1, 64, 2).transpose(1, 2)), dict(q=x[0]),
                dict(q=torch.zeros(1, 4, 64), q_out=torch.zeros(1, 4, 64).half()), dict(q_out=x),
                dict(q=torch.zeros(1, 4, 64), q_out=torch.zeros(1, 2, 64)), dict(cu_tokens=pos),
                dict(cu_tokens=torch.zeros(2))):
        a = dict(k=x, v=x)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            pkg.rope_append(c, table, pos, a.pop("k"), a.pop("v"), **a)


PI = Decimal("3.14159265358979323846264338327950288419716939937510")


@pytest.mark.parametrize("rot,base,scaling,kw", [
    (128, 10000.0, 0, {}), (64, 500000.0, 0, {}), (16, 1.0, 0, {}), (256, 1e6, 1, dict(factor=8.0)),
    (128, 10000.0, 2, dict(factor=4.0)),
    (128, 500000.0, 3, dict(factor=8.0, low_turns=1.0, high_turns=4.0, trained_len=8192))])
def test_rope_steps(lib, rot, base, scaling, kw):
    """Against 50-digit arithmetic: the angle at a far position is within pos * f * 2^-50 radians."""
    getcontext().prec = 50
    got = pkg.attn_rope_steps(rot, base, scaling, **kw)
    assert len(got) == rot // 2
    factor = Decimal(kw.get("factor", 1.0))
    b = Decimal(base) * (factor ** (Decimal(rot) / Decimal(rot - 2)) if scaling == 2 else 1)
    for i, step in enumerate(got):
        f = b ** (Decimal(-2 * i) / Decimal(rot))
        if scaling == 1:
            f = f / factor
        if scaling == 3:
            n = Decimal(kw["trained_len"]) * f / (2 * PI)
            lo, hi = Decimal(kw["low_turns"]), Decimal(kw["high_turns"])
            keep = min(max((n - lo) / (hi - lo), Decimal(0)), Decimal(1))
            f = keep * f + (1 - keep) * f / factor
        want = f / (2 * PI) * Decimal(2) ** 64
        assert abs(Decimal(step) - want) <= want * Decimal(2) ** -50 + Decimal("0.5"), i


def test_rope_steps_refusals(lib):
    buf = (ctypes.c_uint64 * 128)()
    a = ctypes.addressof(buf)
    inf, nan = math.inf, math.nan
    for args in ((0, 1e4, 0, 1, 0, 0, 0), (24, 1e4, 0, 1, 0, 0, 0), (272, 1e4, 0, 1, 0, 0, 0),
                 (64, 0.5, 0, 1, 0, 0, 0), (64, nan, 0, 1, 0, 0, 0), (64, inf, 0, 1, 0, 0, 0),
                 (64, 1e4, 4, 1, 0, 0, 0), (64, 1e4, -1, 1, 0, 0, 0), (64, 1e4, 1, 0.0, 0, 0, 0),
                 (64, 1e4, 1, nan, 0, 0, 0), (64, 1e4, 1, 0.01, 0, 0, 0),      # more than a turn per position
                 (64, 1e4, 3, 8, 4, 4, 10), (64, 1e4, 3, 8, 1, 4, 0), (64, 1e4, 3, 8, nan, 4, 10)):
        assert lib.attn_rope_steps(*args, a) == INVALID, args
    assert lib.attn_rope_steps(64, 1e4, 0, 1.0, 0.0, 0.0, 0, None) == INVALID
    assert all(x == 0 for x in buf)                                    # nothing written on a refusal


def test_reference_codes():
    """The tests' own e4m3: exact on every code, ties to even, against torch's cast."""
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.VALUES, want)
    fin = codes[np.isfinite(ref.VALUES)]
    np.testing.assert_array_equal(ref.to_e4m3(ref.VALUES[fin]), fin)
    x = np.random.default_rng(0).standard_normal(20000) * np.exp(np.random.default_rng(1).uniform(-8, 5, 20000))
    mid = (ref.VALUES[:126] + ref.VALUES[1:127]) / 2                   # ties
    x = np.concatenate([x, mid, -mid]).clip(-448, 448)
    got = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.to_e4m3(x.astype(np.float32)), got)
    for a in (1.0, 447.9, 448.0, 448.1, 3e-5, 1e30, 0.0):
        s = ref.scale_for(a)
        assert (a <= 448 * s or s == 2.0 ** 60) and (a > 224 * s or s == 2.0 ** -60)


def test_the_header_is_plain_c(tmp_path):
    import os
    import subprocess
    src = tmp_path / "t.c"
    src.write_text("#include \"attn_paged.h\"\nint main(void) { attn_paged_cache c = {0}; attn_rope r = {0};\n"
                   "attn_score_rules s = {0}; return (int)(sizeof c + sizeof r + sizeof s) == 0; }\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(root, "include"), "-c", str(src),
                    "-o", str(tmp_path / "t.o")], check=True)
    # the binding's structures have the header's sizes
    probe = tmp_path / "p.c"
    probe.write_text("#include <stdio.h>\n#include \"attn_paged.h\"\nint main(void) { printf(\"%zu %zu %zu\\n\", "
                     "sizeof(attn_paged_cache), sizeof(attn_rope), sizeof(attn_score_rules)); return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(probe), "-o", str(tmp_path / "p")], check=True)
    sizes = [int(x) for x in subprocess.run([str(tmp_path / "p")], capture_output=True, text=True).stdout.split()]
    assert sizes == [ctypes.sizeof(x) for x in (pkg._CacheStruct, pkg._RopeStruct, pkg._RulesStruct)]


def test_paged_constants_match_the_header():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "attn_paged.h")).read()
    found = re.findall(r"^#define (ATTN_(?:TYPE|ROPE|DEVERR)_\w+)\s+(0x[0-9a-fA-F]+|\d+)u?\b", text, flags=re.M)
    assert len(found) == 9
    for name, val in found:
        assert getattr(pkg, name) == int(val, 0), name


# ---------------------------------------------------------------------------
# The torch forms up to the library's door: host tensors that say they are on device 0, and a
# recorder in place of the library, so that valid arguments get through and each refusal is the
# check's own.
# ---------------------------------------------------------------------------
class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return pkg.ATTN_OK
        return call


@pytest.fixture
def door(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    rec = Recorder()
    pkg._torch_module()
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(pkg, "_same_device", lambda d: None)
    monkeypatch.setattr(pkg, "_device", lambda: 0)
    monkeypatch.setattr(pkg, "_raw_stream", lambda i: 0)
    monkeypatch.setattr(pkg, "_alloc", lambda size, stream: 1 << 20)
    monkeypatch.setattr(pkg, "_free", lambda p: None)
    monkeypatch.setattr(pkg, "attn_paged_plan", lambda *a: (4, 4096))
    monkeypatch.setattr(pkg, "_lib", rec)
    return rec


def _pool_and_ids():
    import torch
    k = torch.zeros(3, 16, 2, 64, dtype=torch.float16)
    return (pkg.PagedCache(k, k.clone()), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_tokens_that_overlap_are_refused(door):
    """A row repeated by expand has a stride of 0, which the C call takes for dense: it would be read
    past its end. Strides below a token's elements are refused with it."""
    import torch
    cache, table, pos = _pool_and_ids()
    good = {"k_new": torch.zeros(4, 2, 64), "v_new": torch.zeros(4, 2, 64), "q": torch.zeros(4, 4, 64)}
    pkg.rope_append(cache, table, pos, **good)
    wide = torch.zeros(4, 8, 64)
    pkg.rope_append(cache, table, pos, k_new=wide[:, 4:6], v_new=wide[:, 6:], q=wide[:, :4])
    assert [c[1][10:13] for c in door.calls] == [(256, 128, 128), (512, 512, 512)]
    for name, x in good.items():
        for bad in (x[:1].expand(4, -1, -1), torch.zeros(4 * 64 * 4).as_strided(x.shape, (64, 64, 1))):
            with pytest.raises(ValueError, match="%s must not have tokens that overlap" % name):
                pkg.rope_append(cache, table, pos, **dict(good, **{name: bad}))
    assert len(door.calls) == 2
    # one token has no stride
    one = {n: x[:1].as_strided(x[:1].shape, (0, 64, 1)) for n, x in good.items()}
    pkg.rope_append(cache, table, pos, **one)
    assert door.calls[-1][1][10:13] == (0, 0, 0)


def test_pools_whose_rows_overlap_are_refused(lib):
    """A pool expanded from one row has three strides of 0, which the C call takes for a dense pool: an
    append would write past its allocation. Pages, rows or heads that lie on each other are refused alike."""
    torch = pytest.importorskip("torch")
    shape = (3, 16, 2, 64)
    row = torch.zeros(64, dtype=torch.float16)
    for bad in (row.expand(shape), torch.zeros(1, 16, 2, 64, dtype=torch.float16).expand(shape),
                torch.zeros(3, 1, 2, 64, dtype=torch.float16).expand(shape),
                torch.zeros(3, 16, 1, 64, dtype=torch.float16).expand(shape),
                torch.zeros(9999, dtype=torch.float16).as_strided(shape, (2048, 128, 32, 1)),
                row.view(torch.uint8)[:64].expand(shape).view(torch.float8_e4m3fn)):
        scales = (torch.ones(3, 2), torch.ones(3, 2)) if bad.dtype == torch.float8_e4m3fn else ()
        with pytest.raises(ValueError, match="must not overlap"):
            pkg.PagedCache(bad, bad, *scales)
    # a dimension of one element has no stride, and any other order of the three is fine
    pkg.PagedCache(row.expand(1, 1, 1, 64), row.expand(1, 1, 1, 64))
    k = torch.zeros(3, 2, 16, 64, dtype=torch.float16).transpose(1, 2)
    pkg.PagedCache(k, k)


def test_a_softcap_that_32_bits_take_for_none_is_refused(door):
    """Below the smallest 32-bit number a cap would arrive as 0, which stands for no cap."""
    import torch
    cache, table, pos = _pool_and_ids()
    q = torch.zeros(1, 4, 64)
    for softcap in (0.0, 2.0 ** -40, 30.0):
        pkg.paged_decode_attention(cache, table, pos, q, softcap=softcap)
        pkg.attn_decode_paged(cache, table, 1, pos, q, q, 1, 1, 4, 0.1, (softcap, 0, None, None), stream=0)
    n = len(door.calls)
    for softcap in (1e-50, -1e-50, 5e-324):
        with pytest.raises(ValueError, match="softcap"):
            pkg.paged_decode_attention(cache, table, pos, q, softcap=softcap)
        with pytest.raises(ValueError, match="softcap"):
            pkg.attn_decode_paged(cache, table, 1, pos, q, q, 1, 1, 4, 0.1, (softcap, 0, None, None), stream=0)
    assert len(door.calls) == n


def test_rope_steps_of_an_enlarged_base_past_64_bits(lib):
    """base * factor^(rot_dim / (rot_dim - 2)) that overflows would leave every pair but the first unturned."""
    buf = (ctypes.c_uint64 * 128)()
    a = ctypes.addressof(buf)
    assert lib.attn_rope_steps(128, 1e300, pkg.ATTN_ROPE_BASE, 1e10, 0.0, 0.0, 0, a) == INVALID
    assert lib.attn_rope_steps(16, 1e4, pkg.ATTN_ROPE_BASE, 1e300, 0.0, 0.0, 0, a) == INVALID
    assert all(x == 0 for x in buf)
    assert lib.attn_rope_steps(128, 1e300, pkg.ATTN_ROPE_BASE, 1e6, 0.0, 0.0, 0, a) == OK
    assert buf[1] > 0


def _each_refused(call, good, cases, door):
    """`call` with `good` reaches the library; with each of `cases` it raises that error first."""
    call(**good)
    n = len(door.calls)
    for bad, error, message in cases:
        with pytest.raises(error, match=message):
            call(**dict(good, **bad))
        assert len(door.calls) == n, bad
    call(**good)
    assert len(door.calls) == n + 1


def test_each_refusal_of_the_attention_call(door):
    import torch
    cache, table, pos = _pool_and_ids()
    i32, f16 = torch.int32, torch.float16
    good = dict(block_table=table, positions=pos, q=torch.zeros(1, 4, 64), out=torch.zeros(1, 4, 64),
                slopes=torch.zeros(4), starts=torch.zeros(1, dtype=i32), window=5, n_splits=3)
    disagree = "disagree on n_seq or head_dim"
    _each_refused(lambda **a: pkg.paged_decode_attention(cache, **a), good, [
        (dict(q=torch.zeros(4, 64)), ValueError, "q must be .n_seq"),
        (dict(q=torch.zeros(1, 1, 1, 4, 64)), ValueError, "q must be .n_seq"),
        (dict(q=good["q"].double()), TypeError, "q must be float32"),
        (dict(q=good["q"].half()), TypeError, "q must be float32"),
        (dict(q=torch.zeros(2, 4, 64)), ValueError, disagree),
        (dict(q=torch.zeros(1, 4, 32)), ValueError, disagree),
        (dict(q=torch.zeros(1, 64, 4).transpose(1, 2)), ValueError, "q must be contiguous"),
        (dict(block_table=table.long()), TypeError, "block_table must be int32"),
        (dict(block_table=table[0]), ValueError, "block_table must be .n_seq, max_pages"),
        (dict(block_table=torch.zeros(1, 4, dtype=i32)[:, ::2]), ValueError, "block_table must be contiguous"),
        (dict(positions=pos.long()), TypeError, "positions must be int32"),
        (dict(positions=torch.zeros(2, dtype=i32)), ValueError, "positions .n_seq"),
        (dict(positions=torch.zeros(1, 1, dtype=i32)), ValueError, "positions .n_seq"),
        (dict(out=torch.zeros(1, 4, 32)), ValueError, "out must have the shape of q"),
        (dict(out=torch.zeros(1, 4, 64, dtype=f16)), TypeError, "out must be float32"),
        (dict(out=torch.zeros(1, 64, 4).transpose(1, 2)), ValueError, "out must be contiguous"),
        (dict(slopes=torch.zeros(3)), ValueError, "slopes must be .n_head"),
        (dict(slopes=torch.zeros(4, dtype=f16)), TypeError, "slopes must be float32"),
        (dict(slopes=torch.zeros(8)[::2]), ValueError, "slopes must be contiguous"),
        (dict(starts=torch.zeros(1)), TypeError, "starts must be int32"),
        (dict(starts=torch.zeros(2, dtype=i32)), ValueError, "starts must be .n_seq"),
        (dict(window=-1), ValueError, "window and n_splits"),
        (dict(window=1 << 31), ValueError, "window and n_splits"),
        (dict(n_splits=-1), ValueError, "window and n_splits"),
        (dict(n_splits=1 << 32), ValueError, "window and n_splits"),
        (dict(stream=7), ValueError, "stream must be the current stream"),
    ], door)


def test_each_refusal_of_the_append_call(door, monkeypatch):
    import torch
    cache, _, _ = _pool_and_ids()
    i32, f16 = torch.int32, torch.float16
    table, pos = torch.zeros(2, 1, dtype=i32), torch.zeros(2, dtype=i32)
    x = torch.zeros(2, 2, 64)
    q = torch.zeros(2, 4, 64)
    rope = pkg.Rope(64, device="cpu")
    assert rope._index == 0
    far = pkg.Rope(64, device="cpu")
    far._index = 1
    good = dict(block_table=table, positions=pos, k_new=x, v_new=x, q=q, q_out=torch.zeros(2, 4, 64), rope=rope,
                cu_tokens=torch.tensor([0, 1, 2], dtype=i32))
    shape = "k_new and v_new must be .n_tokens"
    _each_refused(lambda **a: pkg.rope_append(cache, **a), good, [
        (dict(k_new=x.double()), TypeError, "k_new must be float32, float16 or bfloat16"),
        (dict(k_new=x.long()), TypeError, "k_new must be float32, float16 or bfloat16"),
        (dict(v_new=x.half()), TypeError, "v_new must be float32"),
        (dict(v_new=torch.zeros(3, 2, 64)), ValueError, shape),
        (dict(k_new=torch.zeros(2, 3, 64), v_new=torch.zeros(2, 3, 64)), ValueError, shape),
        (dict(k_new=torch.zeros(2, 2, 32), v_new=torch.zeros(2, 2, 32)), ValueError, shape),
        (dict(k_new=torch.zeros(2, 64, 2).transpose(1, 2)), ValueError, "dense within a token"),
        (dict(v_new=torch.zeros(2, 4, 64)[:, ::2]), ValueError, "dense within a token"),
        (dict(block_table=table.long()), TypeError, "block_table must be int32"),
        (dict(block_table=table[0]), ValueError, "block_table must be .n_seq, max_pages"),
        (dict(positions=pos.long()), TypeError, "positions must be int32"),
        (dict(positions=torch.zeros(3, dtype=i32)), ValueError, "positions .n_seq"),
        (dict(q=q[0]), ValueError, "q must be .n_tokens"),
        (dict(q=torch.zeros(3, 4, 64)), ValueError, "q must be .n_tokens"),
        (dict(q=q.half()), TypeError, "q must be float32"),
        (dict(q=torch.zeros(2, 64, 4).transpose(1, 2)), ValueError, "q must be .n_tokens"),
        (dict(q_out=torch.zeros(2, 4, 64, dtype=f16)), TypeError, "q_out must be float32"),
        (dict(q_out=torch.zeros(2, 2, 64)), ValueError, "q_out must have the shape of q"),
        (dict(q_out=torch.zeros(2, 64, 4).transpose(1, 2)), ValueError, "q_out must be contiguous"),
        (dict(q=None), ValueError, "q_out without q"),
        (dict(q_out=None, stream=7), ValueError, "q_out must be given"),
        (dict(cu_tokens=torch.zeros(3)), TypeError, "cu_tokens must be int32"),
        (dict(cu_tokens=torch.zeros(2, dtype=i32)), ValueError, "cu_tokens must be .n_seq"),
        (dict(cu_tokens=torch.zeros(6, dtype=i32)[::2]), ValueError, "cu_tokens must be contiguous"),
        (dict(rope=far), ValueError, "rope must be on the cache's device"),
    ], door)
    # another device than the current one
    monkeypatch.setattr(pkg, "_device", lambda: 1)
    for call in (lambda: pkg.rope_append(cache, **good), lambda: pkg.paged_decode_attention(cache, table, pos, q)):
        n = len(door.calls)
        with pytest.raises(ValueError):
            call()
        assert len(door.calls) == n


@pytest.mark.parametrize("rot,base", [(128, 1e4), (128, 1e6), (96, 1e6), (256, 1e9), (64, 1e30)])
def test_rope_steps_round_to_half_a_step(lib, rot, base):
    """A step is the 64-bit floating-point f_i 2^64 / 2 pi to half a step, pi 2^-64 radians a position: more than
    f_i 2^-50 where f_i lies below some 2e-4. f_i itself: the exponent's rounding (none where rot is a power of
    two) moves it by 2^-53 times the logarithm of base^(2i / rot), power, 2 pi and two divisions by 2^-51 at most."""
    getcontext().prec = 50
    exact = rot & (rot - 1) == 0
    over = 0
    for i, step in enumerate(pkg.attn_rope_steps(rot, base)):
        f = Decimal(base) ** (Decimal(-2 * i) / Decimal(rot))
        own = Decimal(2) ** -51 + (0 if exact else -f.ln() * Decimal(2) ** -53)
        off = abs(Decimal(step) * 2 * PI / Decimal(2) ** 64 - f)
        assert off <= f * own + PI * Decimal(2) ** -64 * (1 + Decimal(2) ** -40), i
        over += off > f * Decimal(2) ** -50
    assert over > 0                            # the rounding to steps is what far positions of slow pairs lose
