"""GPU: the page bookkeeping against the restatement in tree_reference.py: tables and counts are equal to the
last entry, copied pages to the last bit."""
import os
import subprocess
import sys

import numpy as np
import pytest

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tree_reference as tree
from test_paged_gpu import Pool, pkg, tt        # noqa: F401  (pkg is the fixture)

pytestmark = pytest.mark.gpu
CUDA_INCLUDE = "/usr/local/cuda/include"


def book(pkg, refs, table, page):
    return pkg.PageBook(tt(refs), tt(table), page)


def same(b, refs, table):
    np.testing.assert_array_equal(b.refs.cpu().numpy(), refs)
    np.testing.assert_array_equal(b.block_table.cpu().numpy(), table)


@pytest.mark.parametrize("n_seq,n_pages,max_pages,page", [(1, 1, 1, 16), (1, 5, 9, 16), (7, 40, 9, 32), (33, 300, 20, 64),
                                                          (1500, 20011, 16, 16), (8192, 70000, 9, 128), (40, 16384, 500, 16),
                                                          (40, 16385, 500, 1024)])
def test_resize(pkg, n_seq, n_pages, max_pages, page):
    rng = np.random.default_rng(n_seq)
    refs, table = np.zeros(n_pages, np.int32), np.full((n_seq, max_pages), -1, np.int32)
    b = book(pkg, refs, table, page)
    have = np.zeros(n_seq, np.int32)
    pkg.attn_read_device_error()
    for step in range(8):
        want = rng.integers(0, max_pages * page + 1, n_seq).astype(np.int32)
        want[rng.random(n_seq) < 0.2] = 0
        if step % 2:                                               # as many rows as there are, or one more or less
            want = np.clip(have + rng.integers(-1, 2, n_seq), 0, max_pages * page).astype(np.int32)
        if step == 4:
            want[:] = 0
        b.resize(tt(have), tt(want))
        err = tree.resize(refs, table, page, have, want)
        same(b, refs, table)
        assert pkg.attn_read_device_error() == err
        have = want


SMALLER = """
#include <cuda_runtime.h>
static int asked = 0;
extern "C" int times_asked() { return asked; }
namespace attn {
int cluster_slots(const void *, dim3, size_t, unsigned cluster_x) { ++asked; return cluster_x <= %d ? 1 : 0; }
}
"""


@pytest.mark.parametrize("most", [0, 1, 2, 8])
def test_resize_where_no_cluster_of_16_blocks_fits(most, tmp_path):
    """As on a share of a device: the question how many clusters it holds is answered by a library that is loaded before
    (0: by nobody), the same steps give the same tables, and it is asked once per size."""
    shim = tmp_path / "shim.so"
    (tmp_path / "shim.cpp").write_text(SMALLER % most)
    subprocess.run(["g++", "-shared", "-fPIC", "-I", CUDA_INCLUDE, str(tmp_path / "shim.cpp"), "-o", str(shim)], check=True)
    res = subprocess.run([sys.executable, __file__, str(shim)], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.abspath(__file__)))
    assert res.returncode == 0, res.stdout + res.stderr
    assert res.stdout.split() == ["asked", str({0: 4, 1: 4, 2: 4, 8: 2}[most])]


def _resize_with(shim):
    import ctypes
    lib = ctypes.CDLL(shim, mode=ctypes.RTLD_GLOBAL)
    import decode_attention_gqa_gb300 as package
    package.load()
    for shape in ((1, 5, 9, 16), (33, 300, 20, 64), (1500, 20011, 16, 16), (40, 16385, 500, 1024)):
        test_resize(package, *shape)
    print("asked", lib.times_asked())


def test_resize_out_of_range(pkg):
    refs, table = np.zeros(8, np.int32), np.full((4, 3), -1, np.int32)
    b = book(pkg, refs, table, 16)
    pkg.attn_read_device_error()
    b.resize(tt(np.int32([0, 0, 0, 0])), tt(np.int32([49, -1, 2 ** 31 - 1, 16])))
    assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_POSITION_CLAMPED
    tree.resize(refs, table, 16, [0] * 4, [48, 0, 48, 16])
    same(b, refs, table)
    # entries that are no held page: left out of the counting
    table[0, 1], table[2, 2], table[3, 0] = 99, -5, 7
    b.block_table.copy_(tt(table))
    refs[7] = 0
    b.refs.copy_(tt(refs))
    b.resize(tt(np.int32([48, 0, 48, 16])), tt(np.int32([0, 0, 0, 0])))
    assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_BAD_PAGE
    assert tree.resize(refs, table, 16, [48, 0, 48, 16], [0] * 4) == 4
    same(b, refs, table)


def test_a_cut_inside_a_shared_page_is_reported(pkg):
    refs, table = np.zeros(20, np.int32), np.full((3, 4), -1, np.int32)
    b = book(pkg, refs, table, 16)
    pkg.attn_read_device_error()
    have = np.int32([64, 0, 0])
    b.resize(tt(np.int32([0, 0, 0])), tt(have))
    tree.resize(refs, table, 16, [0] * 3, have)
    b.fork(tt(np.int32([0])), tt(np.int32([1])), tt(np.int32([64])))
    tree.fork(refs, table, 16, [0], [1], [64])
    same(b, refs, table)
    have = np.int32([64, 64, 0])
    for want, err in (((48, 64, 0), 0), ((48, 40, 0), pkg.ATTN_DEVERR_SHARED_PAGE), ((0, 40, 0), 0)):
        want = np.int32(want)
        b.resize(tt(have), tt(want))
        assert tree.resize(refs, table, 16, have, want) == err
        assert pkg.attn_read_device_error() == err
        same(b, refs, table)
        have = want


@pytest.mark.parametrize("n_seq,n_fork,n_pages,max_pages,page", [(2, 1, 4, 2, 16), (12, 8, 60, 9, 32), (300, 200, 900, 6, 16),
                                                                 (5000, 4096, 30000, 9, 64), (6, 4, 9, 4, 16)])
def test_fork(pkg, n_seq, n_fork, n_pages, max_pages, page):
    """Some of more forks than there are free pages for, in the last sizes."""
    rng = np.random.default_rng(n_fork)
    refs, table = np.zeros(n_pages, np.int32), np.full((n_seq, max_pages), -1, np.int32)
    parents = n_seq - n_fork
    have = np.zeros(n_seq, np.int32)
    have[:parents] = rng.integers(1, max_pages * page + 1, parents)
    b = book(pkg, refs, table, page)
    zero = np.zeros(n_seq, np.int32)
    b.resize(tt(zero), tt(have))
    tree.resize(refs, table, page, zero, have)
    src = rng.integers(0, parents, n_fork).astype(np.int32)
    dst = (parents + rng.permutation(n_fork)).astype(np.int32)
    rows = np.int32([rng.integers(0, have[s] + 1) for s in src])
    pkg.attn_read_device_error()
    copies = b.fork(tt(src), tt(dst), tt(rows))
    want, err = tree.fork(refs, table, page, src, dst, rows)
    same(b, refs, table)
    np.testing.assert_array_equal(copies.cpu().numpy(), want)
    assert pkg.attn_read_device_error() == err
    # and they end again
    have[dst] = rows
    b.resize(tt(have), tt(zero))
    tree.resize(refs, table, page, have, zero)
    same(b, refs, table)
    assert (refs == 0).all()
    pkg.attn_read_device_error()


def test_forks_that_are_none_are_skipped(pkg):
    refs, table = np.zeros(20, np.int32), np.full((8, 3), -1, np.int32)
    have = np.int32([40, 48, 0, 0, 0, 0, 0, 0])
    b = book(pkg, refs, table, 16)
    b.resize(tt(np.zeros(8, np.int32)), tt(have))
    tree.resize(refs, table, 16, [0] * 8, have)
    pkg.attn_read_device_error()
    src, dst, rows = np.int32([0, -1, 0, 8, 0, 1, 0]), np.int32([2, 3, 8, 4, 0, 5, 6]), np.int32([40, 5, 5, 5, 5, 49, -1])
    copies = b.fork(tt(src), tt(dst), tt(rows))
    want, err = tree.fork(refs, table, 16, src, dst, rows)
    assert err == 8 and pkg.attn_read_device_error() == err
    np.testing.assert_array_equal(copies.cpu().numpy(), want)
    same(b, refs, table)
    table[1, 0], table[1, 2] = -1, 99                              # entries of src that are no page
    b.block_table.copy_(tt(table))
    src, dst, rows = np.int32([1]), np.int32([7]), np.int32([40])
    copies = b.fork(tt(src), tt(dst), tt(rows))
    want, err = tree.fork(refs, table, 16, src, dst, rows)
    assert err == 4 and pkg.attn_read_device_error() == 4
    np.testing.assert_array_equal(copies.cpu().numpy(), want)
    same(b, refs, table)


def test_forks_that_end_in_the_same_sequence_or_in_a_source(pkg):
    """None of two with one dst, none whose dst is the src of another; an impossible fork counts for neither."""
    refs, table = np.zeros(40, np.int32), np.full((70, 3), -1, np.int32)
    have = np.zeros(70, np.int32)
    have[:3] = 40, 48, 17
    b = book(pkg, refs, table, 16)
    b.resize(tt(np.zeros(70, np.int32)), tt(have))
    tree.resize(refs, table, 16, [0] * 70, have)
    pkg.attn_read_device_error()
    src = np.int32([0, 1, 2, 1, 69, 0, 2, 0, 1])
    dst = np.int32([3, 3, 4, 69, 5, 33, 33, 65, 65])
    rows = np.int32([40, 20, 17, 48, 5, 40, 1, 20, 49])               # the last is none, so the one before it is
    copies = b.fork(tt(src), tt(dst), tt(rows))
    want, err = tree.fork(refs, table, 16, src, dst, rows)
    assert err & 8 and pkg.attn_read_device_error() == err
    np.testing.assert_array_equal(copies.cpu().numpy(), want)
    same(b, refs, table)
    assert (table[[3, 33, 69]] == -1).all() and (table[[4, 65], 0] >= 0).all()


@pytest.mark.parametrize("kv", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("order", ["rows", "heads", "joint"])
@pytest.mark.parametrize("hd,n_kv,page", [(64, 1, 16), (128, 3, 48), (256, 8, 64)])
def test_copy_pages(pkg, kv, order, hd, n_kv, page):
    import torch
    pool = Pool(3, kv, n_kv, hd, page, (page * 10,), order=order)
    c = np.int32([[0, 5, page, 7], [1, 6, 1, 0], [2, 7, page - 3, -9], [3, -1, 4, 0], [4, 8, 0, 0], [0, 9, page + 100, 0],
                  [-1, -1, 0, 0], [2, 10, -4, 0]])
    before = [d.view(torch.uint8).clone() for d in pool.dev]
    sc = [x.clone() if x is not None else None for x in pool.dscale]
    pkg.attn_read_device_error()
    pkg.copy_pages(pool.cache(pkg), tt(c))
    assert pkg.attn_read_device_error() == 0
    for i in range(2):
        want = before[i].clone()
        for f, t, r, _ in c.tolist():
            if t >= 0 and r > 0:
                want[t, :r] = before[i][f, :r]
                if sc[i] is not None:
                    sc[i][t] = sc[i][f]
        assert torch.equal(pool.dev[i].view(torch.uint8), want)
        if sc[i] is not None:
            assert torch.equal(pool.dscale[i], sc[i])
    # pages outside the pool
    now = [d.view(torch.uint8).clone() for d in pool.dev]
    pkg.copy_pages(pool.cache(pkg), tt(np.int32([[pool.n_pages, 0, 4, 0], [0, pool.n_pages, 4, 0], [-2, 1, 4, 0]])))
    assert pkg.attn_read_device_error() == pkg.ATTN_DEVERR_BAD_PAGE
    assert all(torch.equal(d.view(torch.uint8), b) for d, b in zip(pool.dev, now))


def test_bookkeeping_in_a_graph_and_on_a_stream_of_the_callers(pkg):
    import torch
    refs, table = np.zeros(200, np.int32), np.full((9, 8), -1, np.int32)
    b = book(pkg, refs, table, 16)
    have, want = tt(np.zeros(9, np.int32)), tt(np.zeros(9, np.int32))
    src, dst, rows = tt(np.int32([0, 1])), tt(np.int32([7, 8])), tt(np.int32([0, 0]))
    copies = torch.empty((2, 4), dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.resize(have, want, stream=s)
    b.fork(src, dst, rows, copies=copies, stream=s)
    torch.cuda.synchronize()
    with pytest.raises(ValueError):
        b.fork(src, dst, rows, stream=s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.resize(have, want)
        b.fork(src, dst, rows, copies=copies)
    rng = np.random.default_rng(1)
    h = np.zeros(9, np.int32)
    for _ in range(6):
        w = rng.integers(1, 129, 9).astype(np.int32)
        w[7:] = 0
        r = np.int32([rng.integers(0, w[0] + 1), rng.integers(0, w[1] + 1)])
        have.copy_(tt(h)), want.copy_(tt(w)), rows.copy_(tt(r))
        g.replay()
        tree.resize(refs, table, 16, h, w)
        c, _ = tree.fork(refs, table, 16, [0, 1], [7, 8], r)
        same(b, refs, table)
        np.testing.assert_array_equal(copies.cpu().numpy(), c)
        h = w
        h[7:] = r
    pkg.attn_read_device_error()


if __name__ == "__main__":
    _resize_with(sys.argv[1])
