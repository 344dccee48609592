"""Attention of drafted trees whose softmax is peaked: one key far above a long
tail whose weights are small one by one and count together."""

import numpy as np
import pytest
import torch

from oracle.dtypes import widen
from spec_support import TreeOnDevice, tree_workload
from support import dev_to_bits, widen_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_394_b200 import pagedkv
    return pagedkv


def bits(x, dtype):
    t = torch.as_tensor(np.asarray(x, dtype=np.float32))
    t = t.to(torch.float16 if dtype == "fp16" else torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16)


def peaked(pk, hist, nodes, group, d, dtype, fp8, gap, sink, v_sink, seed):
    """Every row's logit is 0 at key `sink` of a history and -gap (nats, up to the
    rounding of K, and of its scale) at every other: q is constant, K is -gap
    along it."""
    w = tree_workload(hist, nodes, 2 * group, 2, d, 16, dtype, seed=seed)
    scales = ([0.0125, 0.02], [0.01, 0.03]) if fp8 else None
    w.q = np.broadcast_to(bits(1.0, dtype), w.q.shape).copy()
    k = -gap / (w.scale * d)
    w.key[:] = bits(k, dtype)
    w.k_cache[:] = bits(k, dtype)
    for i, h in enumerate(hist):
        if h:
            b = w.block_tables[i, sink // 16]
            w.k_cache[b, :, sink % 16] = bits(0.0, dtype)
            w.v_cache[b, :, sink % 16] = bits(v_sink, dtype)
    return w, TreeOnDevice(pk, w, scales=scales)


def values(t, w, h, i):
    """float64 [C, D]: the V of sequence i's keys for query head h, by the table."""
    g = h // (w.num_heads // w.num_kv_heads)
    n = int(w.context_lens[i])
    at = np.arange(n)
    rows = t.v_ref[w.block_tables[i][at // 16], g, at % 16]
    if t.scales is None:
        return widen(rows, w.dtype)
    from oracle.fp8 import e4m3_decode
    return e4m3_decode(rows) * float(t.scales[1][g])


def check(t, w, rows, fp16_p):
    """Elementwise within what the roundings allow:
    * the output's, half a step of it and of the smallest subnormal;
    * of P, 2^-11 of each term (the terms' magnitudes sum to mag) while it is a
      normal fp16 number, else half of fp16's smallest step, 2^-25, where the
      largest P is at least 2^7 and so is the sum of P: 2^-32 of each |v|;
    * of the logits, below 2^5 here, 2^-12 of each term (128 2^-24 2^5 at worst,
      and the exponential's 2^-22)."""
    ref, mag = t.reference(rows)
    got = widen_out(dev_to_bits(t.out), w)
    eps = 2.0 ** -11 if w.dtype == "fp16" else 2.0 ** -8
    for node, h in rows:
        i = int(np.searchsorted(w.query_start, node, side="right")) - 1
        tail = 2.0 ** -32 * np.abs(values(t, w, h, i)).sum(axis=0) if fp16_p else 0.0
        r, m = ref[node, h], mag[node, h]
        bound = eps * np.abs(r) + (2.0 ** -11 + 2.0 ** -12) * m * (1 + eps) + tail + 2.0 ** -25
        err = np.abs(got[node, h] - r)
        assert (err <= bound).all(), (node, h, err.max(), bound.min())


# cut and whole units, one and two groups of softmax warps, each cache type
@pytest.mark.parametrize("hist,nodes,group,d", [
    ([32768], [3], 1, 128), ([32768, 40], [20, 5], 8, 64), ([1000, 600], [9, 4], 4, 128),
    ([16384] * 3, [64, 40, 8], 4, 128)])
@pytest.mark.parametrize("dtype,fp8", [("fp16", False), ("bf16", False), ("fp16", True),
                                       ("bf16", True)])
@pytest.mark.parametrize("gap", [12.0, 17.5, 21.0])
def test_a_long_tail_below_one_key(pk, hist, nodes, group, d, dtype, fp8, gap):
    w, t = peaked(pk, hist, nodes, group, d, dtype, fp8, gap, sink=5, v_sink=0.0, seed=51)
    # a tail of one sign, so that what it loses does not cancel
    t.v_ref &= np.uint8(0x7F) if fp8 else np.uint16(0x7FFF)
    t.upload()
    assert t.run() == 0
    check(t, w, {(0, 0), (nodes[0] - 1, 2 * group - 1), (sum(nodes) - 1, group)},
          fp16_p=fp8 or dtype == "fp16")


@pytest.mark.parametrize("dtype,fp8", [("fp16", False), ("fp16", True)])
@pytest.mark.parametrize("sink", [0, 70, 8191])
def test_the_peak_at_any_place_of_the_history(pk, dtype, fp8, sink):
    """The maximum comes first, later, and last: sums made before it are rescaled."""
    for gap in (5.0, 5.5, 9.0, 16.0):     # 2^8 is 5.55 nats
        w, t = peaked(pk, [8192], [6], 4, 128, dtype, fp8, gap, sink=sink, v_sink=1.0, seed=52)
        assert t.run() == 0
        check(t, w, {(0, 0), (5, 7)}, fp16_p=True)
