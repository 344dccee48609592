"""Helpers of the speculative-decoding tests: drafted trees over the workloads
of paged_kv_cache_394_b200.workloads, and the error bound of tree attention."""

import numpy as np
import torch

from oracle import cache_ops as OC
from oracle import fp8 as OF
from oracle import speculative as OS
from paged_kv_cache_394_b200 import workloads as W
from support import DeviceWorkload, dev_to_bits, widen_out


def random_parents(rng, n, kind="tree"):
    """int32 [n]: a tree (or chain, or star) in draft order; node 0 is its root."""
    if kind == "chain":
        return np.arange(-1, n - 1, dtype=np.int32)
    if kind == "star":
        return np.concatenate([[-1], np.zeros(max(n - 1, 0))]).astype(np.int32)[:n]
    if kind == "forest":   # every node a child of the history or of any earlier node
        return np.array([rng.integers(-1, j) if j else -1 for j in range(n)], dtype=np.int32)
    return np.array([-1] + [int(j * rng.random() ** 1.5) for j in range(1, n)],
                    dtype=np.int32)[:n]


def tree_workload(hist, nodes, heads, kv_heads, dim, block, dtype, seed, kind="tree"):
    w = W.build_prefill_workload(hist, nodes, heads, kv_heads, dim, block, dtype, seed)
    rng = np.random.default_rng(seed + 1)
    w.parents = (np.concatenate([random_parents(rng, n, kind) for n in nodes])
                 if sum(nodes) else np.zeros(0, dtype=np.int32)).astype(np.int32)
    return w


class TreeOnDevice(DeviceWorkload):
    """The workload on the device, its tree's K/V written (as 16-bit elements, or
    as E4M3 codes with the given scales), and the oracle's view of the caches."""

    def __init__(self, pk, w, scales=None):
        super().__init__(w)
        self.pk = pk
        self.parents = torch.from_numpy(w.parents).cuda()
        self.max_nodes = int(np.diff(w.query_start).max()) if w.num_seqs else 0
        self.scales = None
        if scales is None:
            pk.reshape_and_cache(self.key, self.value, self.k_cache, self.v_cache, self.slots,
                                 dev_err=self.err)
            self.k_ref, self.v_ref, _ = OC.reshape_and_cache(
                w.key, w.value, w.k_cache, w.v_cache, w.slot_mapping, w.block_size)
        else:
            ks, vs = (np.asarray(s, dtype=np.float32) for s in scales)
            self.scales = (ks, vs)
            self.k_ref = OF.quantize_cache(w.k_cache, w.dtype, ks)
            self.v_ref = OF.quantize_cache(w.v_cache, w.dtype, vs)
            self.k_ref, self.v_ref = OF.quantize_into_cache(
                w.key, w.value, self.k_ref, self.v_ref, w.slot_mapping, w.block_size, w.dtype,
                ks, vs)
            self.k_cache = torch.from_numpy(self.k_ref).cuda()
            self.v_cache = torch.from_numpy(self.v_ref).cuda()
            self.ks, self.vs = torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda()

    def upload(self):
        """The caches as k_ref / v_ref now are."""
        for dst, src in ((self.k_cache, self.k_ref), (self.v_cache, self.v_ref)):
            t = torch.from_numpy(np.ascontiguousarray(src).view(
                np.uint8 if src.dtype == np.uint8 else np.int16)).cuda()
            dst.copy_(t if src.dtype == np.uint8 else t.view(dst.dtype))

    def attend(self, scale=None, **more):
        w = self.w
        scale = w.scale if scale is None else scale
        args = (self.out, self.q, self.k_cache, self.v_cache, self.tables, self.lens, self.qstart,
                self.parents, scale)
        tail = (w.num_kv_heads, w.block_size, w.max_context_len, self.max_nodes)
        more.setdefault("dev_err", self.err)
        if self.scales is None:
            self.pk.paged_attn_tree(*args, *tail, **more)
        else:
            self.pk.paged_attn_tree_fp8(*args, self.ks, self.vs, *tail, **more)

    def run(self, **more):
        self.attend(**more)
        torch.cuda.synchronize()
        return int(self.err.item())

    def reference(self, rows=None, scale=None):
        """(the oracle's output, its terms' magnitudes sum_k p_k |v_k|)."""
        w = self.w
        both = []
        sign = np.uint8(0x7F) if self.scales is not None else np.uint16(0x7FFF)
        for v in (self.v_ref, self.v_ref & sign):
            both.append(OS.tree_attention(
                w.q, self.k_ref, v, w.block_tables, w.context_lens, w.query_start, w.parents,
                w.scale if scale is None else scale, w.num_kv_heads, w.block_size, w.dtype,
                rows=rows, k_scales=None if self.scales is None else self.scales[0],
                v_scales=None if self.scales is None else self.scales[1]))
        return both

    def check(self, rows=None, scale=None):
        ref, mag = self.reference(rows, scale)
        got = widen_out(dev_to_bits(self.out), self.w)
        close(got, ref, mag, self.w.dtype, rows)


def close(got, ref, mag, dtype, rows=None):
    """|got - ref| within what the roundings allow, elementwise:
    * the output's rounding, at most eps / 2 of it (fp16 2^-11, bf16 2^-8), and
      half a step of the smallest subnormal (fp16 2^-25);
    * a probability's rounding to fp16, at most 2^-11 of each of the terms whose
      magnitudes sum to mag;
    * a logit's fp32 sum over at most 128 products: |q . k| scale below 2^6 here,
      so at most 128 2^-24 2^6 = 2^-11 off in the worst case and about the root of
      that many half steps, 2^-14, in earnest, and the exponential's 2^-22, of
      each term.
    The terms' errors are held to 2^-11 + 2^-12 of mag together."""
    out_u = 2.0 ** -11 if dtype == "fp16" else 2.0 ** -8
    if rows is not None:
        at = tuple(np.array(sorted(rows)).T)
        got, ref, mag = got[at], ref[at], mag[at]
    assert np.isfinite(got).all(), "non-finite output"
    bound = out_u * np.abs(ref) + (2.0 ** -11 + 2.0 ** -12) * mag * (1 + out_u) + 2.0 ** -25
    err = np.abs(got - ref)
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), "off by %.3g, bound %.3g at %s (got %r, ref %r)" % (
        err[worst], bound[worst], worst, got[worst], ref[worst])
