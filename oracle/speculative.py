"""Speculative decoding in float64 — the oracle.  TEST INFRASTRUCTURE ONLY.

A draft proposes a tree of tokens per sequence.  The three device steps:

* ``tree_attention``: node j of a tree sees the sequence's history and the
  nodes on its path up to the history (itself among them).
* ``verify``: speculative sampling along the tree.  The kept tokens and the one
  that follows them are distributed as the target's own samples.
* ``compact``: the kept nodes' K/V move to the front of the tree's positions.

A tree's nodes are the last ``q_len`` cached tokens of its sequence, in draft
order; ``parents`` holds indices within the tree, -1 for a child of the history.
For verification node 0 is the root, the token sampled last.
"""

import numpy as np

from .attention import attend, kv_head_of
from .dtypes import widen
from .fp8 import e4m3_decode


def path_to(parents, j):
    """Node j and its ancestors, rising."""
    path = []
    while j != -1:
        path.append(j)
        if not -1 <= parents[j] < j:
            raise ValueError("a parent must come before its node")
        j = parents[j]
    return path[::-1]


def cached_rows(cache, table_row, positions, kv_head, block_size, dtype, scale=None):
    """float64 [len(positions), D]: the K (or V) rows of logical tokens.  A cache
    of uint8 codes holds E4M3 values times ``scale``."""
    t = np.asarray(positions, dtype=np.int64)
    rows = cache[np.asarray(table_row)[t // block_size], kv_head, t % block_size, :]
    if cache.dtype == np.uint8:
        return e4m3_decode(rows) * float(scale)
    return widen(rows, dtype)


def tree_attention(q_bits, k_cache, v_cache, block_tables, context_lens, query_start, parents,
                   scale, num_kv_heads, block_size, dtype, rows=None, k_scales=None,
                   v_scales=None):
    """float64 [T, H, D]; ``rows``: the (node, head) rows to compute (others NaN)."""
    total, num_heads, dim = q_bits.shape
    out = np.full((total, num_heads, dim), np.nan)
    wanted = None if rows is None else {(int(t), int(h)) for t, h in rows}
    for i in range(len(context_lens)):
        a, b = int(query_start[i]), int(query_start[i + 1])
        hist = int(context_lens[i]) - (b - a)
        for t in range(a, b):
            seen = list(range(hist)) + [hist + n for n in path_to(parents[a:b], t - a)]
            for h in range(num_heads):
                if wanted is not None and (t, h) not in wanted:
                    continue
                g = kv_head_of(h, num_heads, num_kv_heads)
                k, v = (cached_rows(c, block_tables[i], seen, g, block_size, dtype,
                                    None if s is None else s[g])
                        for c, s in ((k_cache, k_scales), (v_cache, v_scales)))
                out[t, h] = attend(widen(q_bits[t, h], dtype), k, v, scale)
    return out


def verify_one(parents, tokens, target, draft, accept_u, sample_u):
    """One tree: (kept nodes, next token).  target (and draft, or None) [n, V]
    float64, row j the distribution after node j."""
    n = len(parents)
    kept = [0]
    r, z = np.fmax(np.asarray(target[0], dtype=np.float64), 0.0), 1.0
    for j in range(1, n):
        cur = kept[-1]
        if parents[j] != cur:
            continue
        x = tokens[j]
        if draft is not None:
            q = np.fmax(np.asarray(draft[cur], dtype=np.float64), 0.0)
        else:
            q = np.zeros(len(r))
            q[x] = 1.0
        if float(accept_u[j]) * q[x] * z < r[x]:
            kept.append(j)
            r, z = np.fmax(np.asarray(target[j], dtype=np.float64), 0.0), 1.0
        elif draft is not None:
            with np.errstate(divide="ignore", invalid="ignore"):
                r = np.fmax(r / z - q, 0.0)
            z = r.sum()
        else:
            z -= r[x]
            r = r.copy()
            r[x] = 0.0
    if not r.sum() > 0:
        r = np.fmax(np.asarray(target[kept[-1]], dtype=np.float64), 0.0)
    c = np.cumsum(r)
    above = np.nonzero(c > float(sample_u) * c[-1])[0]
    return kept, int(above[0] if len(above) else np.nonzero(r)[0][-1])


def verify(query_start, parents, tokens, target, draft, accept_u, sample_u, width):
    """(accepted [S, width], num_accepted [S], next_token [S]) of a batch."""
    s = len(query_start) - 1
    accepted = np.full((s, width), -1, dtype=np.int32)
    count, nxt = np.zeros(s, dtype=np.int32), np.full(s, -1, dtype=np.int32)
    for i in range(s):
        a, b = int(query_start[i]), int(query_start[i + 1])
        if a == b:
            continue
        kept, nxt[i] = verify_one(parents[a:b], tokens[a:b], target[a:b],
                                  None if draft is None else draft[a:b], accept_u[a:b],
                                  sample_u[i])
        accepted[i, :len(kept)] = kept
        count[i] = len(kept)
    return accepted, count, nxt


def compact(k_cache, v_cache, block_tables, context_lens, query_start, accepted, num_accepted,
            block_size):
    """The caches after every tree's kept rows moved to its front (new arrays)."""
    out = []
    for cache in (k_cache, v_cache):
        new = cache.copy()
        for i in range(len(context_lens)):
            hist = int(context_lens[i]) - int(query_start[i + 1] - query_start[i])
            for d in range(int(num_accepted[i])):
                src, dst = hist + int(accepted[i, d]), hist + d
                row = block_tables[i]
                new[row[dst // block_size], :, dst % block_size] = \
                    cache[row[src // block_size], :, src % block_size]
        out.append(new)
    return out
