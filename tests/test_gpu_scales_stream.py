"""E4M3 scales given as numbers to a call on another stream than the current one:
the numbers are in memory before the kernel reads them, though the current
stream is busy."""

import pytest
import torch

from spec_support import TreeOnDevice, tree_workload

pytestmark = pytest.mark.gpu


def busy(seconds=0.05):
    """Keeps the current stream at work for about that long."""
    x = torch.randn(4096, 4096, device="cuda")
    for _ in range(int(seconds / 0.002)):
        x = torch.mm(x, x).clamp_(-1, 1)
    return x


def test_number_scales_on_a_side_stream():
    from paged_kv_cache_394_b200 import pagedkv as pk

    w = tree_workload([200, 31, 900], [20, 8, 64], 16, 2, 128, 16, "fp16", seed=71)
    t = TreeOnDevice(pk, w, scales=([0.0125] * 2, [0.01] * 2))
    t.run()
    t.check()
    first = t.out.clone()
    s = torch.cuda.Stream()
    for _ in range(3):
        # memory that held other values, free on the current stream
        for _ in range(4):
            torch.full((2,), 7.0, device="cuda")
        t.out.zero_()
        torch.cuda.synchronize()
        keep = busy()
        pk.paged_attn_tree_fp8(t.out, t.q, t.k_cache, t.v_cache, t.tables, t.lens, t.qstart,
                               t.parents, w.scale, 0.0125, 0.01, 2, 16, w.max_context_len,
                               t.max_nodes, dev_err=t.err, stream=s)
        s.synchronize()
        assert int(t.err.item()) == 0 and torch.equal(first, t.out)
        del keep


def test_number_scales_of_the_cache_write_and_decode_on_a_side_stream():
    from paged_kv_cache_394_b200 import pagedkv as pk

    w = tree_workload([64, 100, 30], [1, 1, 1], 8, 2, 64, 16, "fp16", seed=72)
    t = TreeOnDevice(pk, w, scales=([0.0125] * 2, [0.01] * 2))
    want = torch.empty_like(t.q)
    args = (t.q, t.k_cache, t.v_cache, t.tables, t.lens, w.scale)
    pk.paged_attn_decode_fp8(want, *args, t.ks, t.vs, 2, 16, w.max_context_len, dev_err=t.err)
    got = torch.zeros_like(want)
    k8, v8 = t.k_cache.clone(), t.v_cache.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = busy()
    pk.reshape_and_cache_fp8(t.key, t.value, k8, v8, t.slots, 0.0125, 0.01, dev_err=t.err,
                             stream=s)
    pk.paged_attn_decode_fp8(got, *args, 0.0125, 0.01, 2, 16, w.max_context_len, dev_err=t.err,
                             stream=s)
    s.synchronize()
    assert int(t.err.item()) == 0
    assert torch.equal(want, got) and torch.equal(k8, t.k_cache) and torch.equal(v8, t.v_cache)
    del keep
