"""Draft verification next to a border: weights whose sums are exact in 64 bits, and
a drawn share that lies between two of them."""

import numpy as np
import pytest
import torch

from oracle import speculative as OS

pytestmark = pytest.mark.gpu


# clusters of 1, 2, 4 and 8 CTAs
@pytest.mark.parametrize("vocab", [300, 2048, 5000, 9001, 20000])
@pytest.mark.parametrize("nudge,want", [(0, "first"), (3, "second")])
def test_a_residual_is_summed_in_64_bits(vocab, nudge, want):
    """After the first rejection r = p - q.  Tokens 0 .. 3 weigh
    A = (1 + 2^-25 - 3 2^-52) / 2 together, two later ones
    B = (1 + 2^-25 - (5 - nudge) 2^-52) / 2, and the share is half of A + B: token 3
    is the smallest whose running sum is above it if A > B, else the next.  All
    sums are exact in 64 bits, in any order; the differences are not in 32."""
    from paged_kv_cache_394_b200 import pagedkv as pk

    p, q = np.zeros((2, vocab), np.float32), np.zeros((2, vocab), np.float32)
    p[0, :4] = np.array([1.0, 2.0 ** -26, 2.0 ** -26, 2.0 ** -26]) / 2
    q[0, :4] = np.array([2.0 ** -26, 2.0 ** -52, 2.0 ** -52, 2.0 ** -52]) / 2
    y = 4 + 8 * 9                   # another lane's
    p[0, y:y + 2] = np.array([1.0, 2.0 ** -25]) / 2
    q[0, y + 1] = (5 - nudge) * 2.0 ** -52 / 2
    q[0, 200] = 1.0                 # the drafted token: the target never takes it
    p[1, 7], q[1, 7] = 1.0, 1.0
    r = np.maximum(p[0].astype(np.float64) - q[0], 0)
    a, b = r[:4].sum(), r[y:y + 2].sum()
    assert a == (1 + 2.0 ** -25 - 3 * 2.0 ** -52) / 2 and a - b == (2 - nudge) * 2.0 ** -53
    par, qs, tok = np.array([-1, 0], np.int32), np.array([0, 2], np.int32), np.array([0, 200], np.int32)
    u, un = np.array([0.5, 0.5], np.float32), np.array([0.5], np.float32)
    ref = OS.verify(qs, par, tok, p.astype(np.float64), q.astype(np.float64), u, un, 2)
    assert ref[2][0] == (3 if want == "first" else y)
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    acc = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    count, nxt, err = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(3))
    pk.verify_draft(acc, count, nxt, dev(p), dev(tok), dev(par), dev(qs), dev(u), dev(un), 2,
                    draft_probs=dev(q), dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert acc.tolist() == ref[0].tolist() and count.tolist() == ref[1].tolist()
    assert nxt.tolist() == ref[2].tolist()
