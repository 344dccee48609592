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
