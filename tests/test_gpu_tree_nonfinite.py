"""Infinities and NaN in V that a drafted tree's rows do see, whatever weight the
key has: the element's value is their sum (infinity, or NaN), as in 64 bits."""

import numpy as np
import pytest
import torch

from spec_support import TreeOnDevice, close, tree_workload
from support import dev_to_bits, widen_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_394_b200 import pagedkv
    return pagedkv


def bits(x, dtype):
    t = torch.tensor(float(x)).to(torch.float16 if dtype == "fp16" else torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16)


def special(dtype, fp8):
    """(infinity or NaN, minus infinity or NaN, NaN) as V's elements; E4M3 has NaN only."""
    if fp8:
        return 0x7F, 0xFF, 0x7F
    return (0x7C00, 0xFC00, 0x7E00) if dtype == "fp16" else (0x7F80, 0xFF80, 0x7FC0)


def put(t, w, i, pos, dims, what):
    b = w.block_tables[i, pos // w.block_size]
    t.v_ref[b, :, pos % w.block_size, dims] = what


# one sequence, cut into pieces whose maxima lie 150 nats apart
@pytest.mark.parametrize("heads,d", [(2, 128), (8, 64), (16, 128)])
@pytest.mark.parametrize("dtype,fp8", [("fp16", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("far_first", [False, True])
def test_infinite_v_of_a_node_in_a_piece_of_no_weight(pk, dtype, fp8, heads, d, far_first):
    h = 12000
    w = tree_workload([h], [6], heads, 2, d, 16, dtype, seed=61, kind="chain")
    w.q = np.broadcast_to(bits(1.0, dtype), w.q.shape).copy()
    low = -150.0 / (w.scale * d)
    scales = None
    if fp8:
        s = 2.0 ** -4 if d == 128 else 2.0 ** -3    # codes of low fit in 448
        scales = ([s, s], [0.01, 0.03])
    # the first half of the history at logit 0, the rest and the tree at -150, or
    # the other way round
    half = w.block_tables[0, :h // 32]
    w.k_cache[:] = bits(0.0 if far_first else low, dtype)
    w.k_cache[half] = bits(low if far_first else 0.0, dtype)
    w.key[:] = bits(0.0 if far_first else low, dtype)
    t = TreeOnDevice(pk, w, scales=scales)
    ref, mag = t.reference({(n, 0) for n in range(6)})
    inf, minus, nan = special(dtype, fp8)
    put(t, w, 0, h + 2, slice(0, None, 4), inf)
    put(t, w, 0, h + 3, slice(1, None, 4), minus)
    put(t, w, 0, h + 1, slice(2, None, 4), nan)
    t.upload()
    assert t.run() == 0
    got = widen_out(dev_to_bits(t.out), w)
    for n in range(6):
        for dims, node, what in ((slice(0, None, 4), 2, np.isposinf),
                                 (slice(1, None, 4), 3, np.isneginf),
                                 (slice(2, None, 4), 1, np.isnan)):
            if n >= node:
                assert (np.isnan if fp8 else what)(got[n, :, dims]).all(), (n, node)
            else:
                close(got[n, :1, dims], ref[n, :1, dims], mag[n, :1, dims], dtype)
        close(got[n, :1, 3::4], ref[n, :1, 3::4], mag[n, :1, 3::4], dtype)


# whole and cut units; one query tile, two in turn, two side by side
@pytest.mark.parametrize("hist,nodes,heads,d", [
    ([300], [8], 8, 128), ([70, 20], [40, 24], 2, 64), ([6000, 130], [5, 3], 4, 128),
    ([3000, 50], [64, 20], 16, 128), ([3000] * 30, [9] * 30, 8, 64)])
@pytest.mark.parametrize("dtype,fp8", [("fp16", False), ("bf16", False), ("fp16", True)])
def test_infinite_v_in_the_history(pk, hist, nodes, heads, d, dtype, fp8):
    w = tree_workload(hist, nodes, heads, 2, d, 16, dtype, seed=62)
    t = TreeOnDevice(pk, w, scales=([0.0125, 0.02], [0.01, 0.03]) if fp8 else None)
    first = int(w.query_start[1]) - 1
    rows = {(0, 0), (first, heads - 1), (first // 2, heads // 2)}
    if len(nodes) > 1:
        rows |= {(first + 1, 0), (len(w.q) - 1, heads - 1)}
    ref, mag = t.reference(rows)
    inf, minus, nan = special(dtype, fp8)
    h = hist[0]
    for pos, dims, what in ((0, 0, inf), (h - 1, 1, minus), (h // 2, 2, nan), (h // 3, 3, inf),
                            (h // 3 + 9, 3, minus), (h // 5, 4, inf), (h - 2, 4, inf)):
        put(t, w, 0, pos, slice(dims, None, 8), what)
    t.upload()
    assert t.run() == 0
    got = widen_out(dev_to_bits(t.out), w)
    own = got[:first + 1]
    for dims, what in ((0, np.isposinf), (1, np.isneginf), (2, np.isnan), (3, np.isnan),
                       (4, np.isposinf)):
        assert (np.isnan if fp8 else what)(own[:, :, dims::8]).all(), dims
    assert np.isfinite(own.reshape(-1, heads, d // 8, 8)[..., 5:]).all()
    assert np.isfinite(got[first + 1:]).all()
    for n, head in rows:
        at = np.arange(d) % 8 >= (5 if n <= first else 0)
        close(got[n, head, at], ref[n, head, at], mag[n, head, at], dtype)


# the infinity's weight underflows: far below the row's maximum, before and behind it
@pytest.mark.parametrize("hist,nodes,heads", [(700, 5, 4), (9000, 5, 4), (2000, 64, 16)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("peak", [0.1, 0.9])
def test_infinite_v_of_no_weight_in_the_history(pk, hist, nodes, heads, dtype, peak):
    d = 128
    w = tree_workload([hist], [nodes], heads, 2, d, 16, dtype, seed=63)
    w.q = np.broadcast_to(bits(1.0, dtype), w.q.shape).copy()
    low = bits(-150.0 / (w.scale * d), dtype)
    w.k_cache[:] = low
    w.key[:] = low
    at = int(hist * peak)
    w.k_cache[w.block_tables[0, at // 16], :, at % 16] = bits(0.0, dtype)
    t = TreeOnDevice(pk, w)
    inf, minus, nan = special(dtype, False)
    for pos, dims, what in ((5, 0, inf), (hist // 2, 1, minus), (hist - 3, 2, inf),
                            (at, 3, minus)):
        put(t, w, 0, pos, slice(dims, None, 8), what)
    t.upload()
    assert t.run() == 0
    got = widen_out(dev_to_bits(t.out), w)
    for dims, what in ((0, np.isposinf), (1, np.isneginf), (2, np.isposinf), (3, np.isneginf)):
        assert what(got[:, :, dims::8]).all(), dims
    assert np.isfinite(got.reshape(-1, heads, d // 8, 8)[..., 4:]).all()


@pytest.mark.parametrize("hist,nodes,heads", [(300, 8, 8), (9000, 6, 4), (3000, 64, 16)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_opposite_infinities_in_history_and_tree(pk, hist, nodes, heads, dtype):
    w = tree_workload([hist], [nodes], heads, 2, 64, 16, dtype, seed=64, kind="chain")
    t = TreeOnDevice(pk, w)
    inf, minus, _ = special(dtype, False)
    for base in (0, hist - 1):      # the first tile, and the one that the tree starts in
        put(t, w, 0, base, slice(0, None, 8), inf)
        put(t, w, 0, base, slice(1, None, 8), minus)
    put(t, w, 0, hist + 3, slice(0, None, 8), minus)
    put(t, w, 0, hist + 3, slice(1, None, 8), minus)
    put(t, w, 0, hist + 3, slice(2, None, 8), inf)
    t.upload()
    assert t.run() == 0
    got = widen_out(dev_to_bits(t.out), w)
    assert np.isposinf(got[:3, :, 0::8]).all() and np.isnan(got[3:, :, 0::8]).all()
    assert np.isneginf(got[:, :, 1::8]).all()
    assert np.isfinite(got[:3, :, 2::8]).all() and np.isposinf(got[3:, :, 2::8]).all()
    assert np.isfinite(got.reshape(nodes, heads, 8, 8)[..., 3:]).all()
