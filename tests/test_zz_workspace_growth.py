"""GPU: the library-owned workspace grows under a captured graph that holds the smaller one.

Last in the order of files: it leaves a large workspace behind.
"""
import math

import pytest

from harness import make_case, to_device

pytestmark = pytest.mark.gpu


def test_a_graph_keeps_its_workspace_when_a_larger_call_follows():
    """A dense call captured over the library's buffer, then a paged one that needs more of it: the graph's partial
    results still go where they went, and nothing that was allocated since is written."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import decode_attention_gqa_gb300 as pkg
    from decode_attention_gqa_gb300 import build
    build.build()
    n_head, n_kv, hd, cap = 8, 2, 128, 256
    dev = to_device(make_case(24, 1, n_head, n_kv, hd, cap, (200,)))
    out = torch.empty_like(dev["q"])

    def dense(o):
        pkg.attn_decode_ex(dev["q"], dev["k"], dev["v"], dev["positions"], o, 1, n_head, n_kv, hd, 1 / math.sqrt(hd), cap,
                           n_splits=4)
    dense(out)
    torch.cuda.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dense(out)
    # 4096 splits of 8 KV heads of 256 dimensions: more than half a GB of parts
    k = torch.zeros(2, 16, 8, 256, dtype=torch.float16, device="cuda")
    cache = pkg.PagedCache(k, k)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([31], dtype=torch.int32, device="cuda")
    q = torch.ones(1, 8, 256, device="cuda")
    o = torch.ones(1, 8, 256, device="cuda")
    need = pkg.attn_paged_plan(cache, 2, 1, 1, 8, n_splits=4096)[1]
    assert need > 1 << 29
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    pkg.attn_decode_paged(cache, table, 2, pos, q, o, 1, 1, 8, 0.1, n_splits=4096)
    torch.cuda.synchronize()
    assert bool((o == 0).all())
    assert free - torch.cuda.mem_get_info()[0] >= need // 2        # it did grow
    guard = [torch.zeros(1 << 20, device="cuda") for _ in range(64)]
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(bool((g == 0).all()) for g in guard)
    dense(out)                                                     # over the larger one
    assert torch.equal(out, want)
    assert pkg.attn_read_device_error() == 0
