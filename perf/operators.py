"""Speculative decoding over the paged KV cache, as measured: attention for a
tree of drafted tokens, verification of the drafted tokens, and compaction of
the accepted path in the cache.

A case is one call's shape.  ``prepare`` makes the inputs, ``run`` makes one
pass: with ``own`` false in elementary torch operations, with ``own`` true
through the library.  ``exact`` computes the same from the definitions in 64
bits, sequence by sequence.
"""

import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases -----------------------------------------------------------------
def listed():
    return [
        # one interactive user of a GQA model, a small tree: the call's latency
        dict(name="tree one user", op="tree", seqs=1, nodes_lo=8, nodes=8, ctx_lo=300, ctx=300,
             heads=32, kv_heads=8, dim=128, block=16, dtype="bf16", cache="16"),
        # a chat batch of a GQA model, ragged trees and contexts
        dict(name="tree gqa chat", op="tree", seqs=32, nodes_lo=5, nodes=32, ctx_lo=40, ctx=4096,
             heads=32, kv_heads=8, dim=128, block=32, dtype="bf16", cache="16"),
        # the LLaMA-7B attention layer (32 heads, no grouping), short drafts
        dict(name="tree llama7b", op="tree", seqs=32, nodes_lo=16, nodes=16, ctx_lo=128, ctx=2048,
             heads=32, kv_heads=32, dim=128, block=16, dtype="fp16", cache="16"),
        # few long documents, large trees over 8 heads a group: tensor cores and memory alike
        dict(name="tree long", op="tree", seqs=4, nodes_lo=64, nodes=64, ctx_lo=16384, ctx=32768,
             heads=64, kv_heads=8, dim=128, block=16, dtype="bf16", cache="16"),
        # an 8-bit cache, ordinary trees
        dict(name="tree e4m3", op="tree", seqs=16, nodes_lo=12, nodes=33, ctx_lo=512, ctx=8192,
             heads=32, kv_heads=8, dim=128, block=16, dtype="fp16", cache="e4m3"),
        # a small model: head_dim 64, two heads a group
        dict(name="tree small heads", op="tree", seqs=8, nodes_lo=3, nodes=25, ctx_lo=100,
             ctx=3000, heads=16, kv_heads=8, dim=64, block=16, dtype="fp16", cache="16"),
        # one user, a chain of four drafted tokens
        dict(name="verify one chain", op="verify", seqs=1, nodes=5, vocab=32000, chain=True,
             draft=True, dtype="fp32"),
        # a serving batch of chains over a large vocabulary
        dict(name="verify chains", op="verify", seqs=64, nodes=8, vocab=128000, chain=True,
             draft=True, dtype="fp32"),
        # trees sampled from the draft: rejected siblings leave residuals
        dict(name="verify trees", op="verify", seqs=16, nodes=24, vocab=50001, chain=False,
             draft=True, dtype="bf16"),
        # trees of the draft's best tokens (no draft probabilities)
        dict(name="verify best tokens", op="verify", seqs=32, nodes=32, vocab=100000, chain=False,
             draft=False, dtype="fp32"),
        # after a small batch's verification, 8-bit cache
        dict(name="compact few", op="compact", seqs=4, nodes=16, hist=70, kv_heads=8, dim=128,
             block=16, keep=4, dtype="bf16", cache="e4m3"),
        # after a large batch's verification, ungrouped heads
        dict(name="compact batch", op="compact", seqs=256, nodes=32, hist=45, kv_heads=32,
             dim=128, block=16, keep=8, dtype="fp16", cache="16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "verify", "compact"])
    if op == "tree":
        kv = rng.choice([1, 2, 4, 8, 8, 32])
        group = rng.choice([1, 2, 4, 8]) if kv < 32 else 1
        nodes = _spread(rng, 1, 64)
        dim = rng.choice([64, 128, 128])
        ctx = _spread(rng, max(nodes, 2), 32768)
        # no more cached values than the largest listed case has
        most = max(1, min(64, int(4 * 24576 * 8 * 128 / (ctx * kv * dim))))
        most = max(1, min(most, int(4 * 64 * 64 * 24576 / (kv * group * nodes * ctx))))
        return dict(op="tree", seqs=_spread(rng, 1, most), nodes_lo=rng.randint(1, nodes),
                    nodes=nodes, ctx_lo=rng.randint(nodes, ctx), ctx=ctx, heads=kv * group,
                    kv_heads=kv, dim=dim, block=rng.choice([16, 32]),
                    dtype=rng.choice(["fp16", "bf16"]), cache=rng.choice(["16", "16", "e4m3"]))
    if op == "verify":
        vocab = _spread(rng, 1000, 160000)
        nodes = rng.randint(1, 32)
        dtype = rng.choice(["fp32", "fp32", "fp16", "bf16"])
        most = max(1, min(128, int(64 * 8 * 128000 / (nodes * vocab))))
        return dict(op="verify", seqs=_spread(rng, 1, most), nodes=nodes, vocab=vocab,
                    chain=rng.random() < 0.5, draft=rng.random() < 0.6, dtype=dtype)
    nodes = _spread(rng, 2, 64)
    kv = rng.choice([1, 2, 8, 32])
    return dict(op="compact", seqs=_spread(rng, 1, 256), nodes=nodes,
                hist=_spread(rng, 1, 64), kv_heads=kv, dim=rng.choice([64, 128]),
                block=rng.choice([16, 32]), keep=rng.randint(1, min(nodes, 12)),
                dtype=rng.choice(["fp16", "bf16"]), cache=rng.choice(["16", "e4m3"]))


def _levels(lo, hi, n):
    """n whole numbers from lo to hi in equal steps: a batch's lengths, in any order."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _tree_sizes(case):
    nodes = _levels(case["nodes_lo"], case["nodes"], case["seqs"])
    ctx = _levels(case["ctx_lo"], case["ctx"], case["seqs"])
    return nodes, [max(c, n) for c, n in zip(ctx, nodes[::-1])]


def work(case):
    if case["op"] == "tree":
        nodes, ctx = _tree_sizes(case)
        elem = 1 if case["cache"] == "e4m3" else 2
        total = sum(nodes)
        cached = sum(ctx) * case["kv_heads"] * case["dim"] * 2 * elem
        rows = 2 * total * case["heads"] * case["dim"] * 2
        pairs = sum(n * (c - n + 1) for n, c in zip(nodes[::-1], ctx))  # at least itself each
        return {"bytes": cached + rows, "flops": 4 * case["dim"] * case["heads"] * pairs}
    if case["op"] == "verify":
        elem = 4 if case["dtype"] == "fp32" else 2
        rows = 2 if case["draft"] else 1  # the last node's row of the target, and of the draft
        return {"bytes": case["seqs"] * rows * elem * (case["vocab"] + case["nodes"]),
                "flops": case["seqs"] * case["vocab"] * rows}
    elem = 1 if case["cache"] == "e4m3" else 2
    moved = sum(max(0, k - 1) for k in _keeps(case))
    moved = moved if case["nodes"] > case["keep"] else 0
    return {"bytes": max(64, moved * case["kv_heads"] * case["dim"] * 2 * 2 * elem), "flops": 0}


def _keeps(case):
    return _levels(1, case["keep"], case["seqs"])


# ---- inputs ----------------------------------------------------------------
def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _parents(rng, n, chain=False):
    """A tree in draft order: node 0 is its root, a node follows its parent."""
    return [-1] + [j - 1 if chain else int(j * rng.random() ** 1.5) for j in range(1, n)]


def _paged(rng, ctx, block):
    """Block tables with the blocks anywhere in a pool a fifth larger than needed."""
    need = [-(-c // block) for c in ctx]
    pool = int(sum(need) * 1.2) + 1
    order = list(range(pool))
    rng.shuffle(order)
    width = max(max(need), 1)
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n] + [-1] * (width - n))
        at += n
    return _i32(rows), pool


def _cache(gen, shape, case):
    x = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(generator=gen)
    if case["cache"] == "e4m3":
        return (x.mul_(32.0)).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(DTYPES[case["dtype"]])


def _scales(gen, kv):
    return torch.empty(kv, dtype=torch.float32, device="cuda").uniform_(
        0.02, 0.045, generator=gen)


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"tree": _prepare_tree, "verify": _prepare_verify,
            "compact": _prepare_compact}[case["op"]](case, rng, gen)


def _prepare_tree(case, rng, gen):
    nodes, ctx = _tree_sizes(case)
    pairs = list(zip(nodes[::-1], ctx))
    rng.shuffle(pairs)
    nodes, ctx = [p[0] for p in pairs], [p[1] for p in pairs]
    tables, pool = _paged(rng, ctx, case["block"])
    shape = (pool, case["kv_heads"], case["block"], case["dim"])
    dt = DTYPES[case["dtype"]]
    q = torch.randn((sum(nodes), case["heads"], case["dim"]), generator=gen, device="cuda").to(dt)
    st = dict(case=case, q=q, out=torch.empty_like(q), k=_cache(gen, shape, case),
              v=_cache(gen, shape, case), tables=tables, ctx=_i32(ctx), qs=_i32(_starts(nodes)),
              parents=_i32(sum((_parents(rng, n) for n in nodes), [])),
              scale=1.0 / math.sqrt(case["dim"]), most_ctx=max(ctx), most_nodes=max(nodes),
              err=_i32([0]))
    if case["cache"] == "e4m3":
        st["ks"], st["vs"] = _scales(gen, case["kv_heads"]), _scales(gen, case["kv_heads"])
    return st


def _prepare_verify(case, rng, gen):
    s, n, v = case["seqs"], case["nodes"], case["vocab"]
    dt = DTYPES[case["dtype"]]
    par = [_parents(rng, n, case["chain"]) for _ in range(s)]
    logits = torch.randn((s * n, v), generator=gen, device="cuda")
    noise = torch.randn((s * n, v), generator=gen, device="cuda")
    draft = torch.softmax(logits.mul_(4.0).add(noise, alpha=0.8), dim=1)
    del noise
    target = torch.softmax(logits, dim=1).to(dt)
    del logits
    # each node's token drawn from its parent's draft distribution; the root's is any
    rows = torch.tensor([i * n + max(p, 0) for i in range(s) for p in par[i]], device="cuda")
    u = torch.rand((s * n, 1), generator=gen, device="cuda")
    tokens = torch.empty(s * n, dtype=torch.int32, device="cuda")
    for at in range(0, s * n, 64):
        c = torch.cumsum(draft[rows[at:at + 64]], dim=1)
        tokens[at:at + 64] = torch.searchsorted(c, u[at:at + 64] * c[:, -1:])[:, 0].clamp(
            max=v - 1).int()
    return dict(case=case, target=target, draft=draft.to(dt) if case["draft"] else None,
                tokens=tokens, parents=_i32(sum(par, [])), qs=_i32(_starts([n] * s)),
                u=torch.rand(s * n, generator=gen, device="cuda"),
                u_next=torch.rand(s, generator=gen, device="cuda"), nodes=n,
                accepted=torch.empty((s, n), dtype=torch.int32, device="cuda"),
                count=torch.empty(s, dtype=torch.int32, device="cuda"),
                next=torch.empty(s, dtype=torch.int32, device="cuda"), err=_i32([0]))


def _prepare_compact(case, rng, gen):
    s, n = case["seqs"], case["nodes"]
    keeps = _keeps(case)
    rng.shuffle(keeps)
    hist = _levels(max(0, case["hist"] - 16), case["hist"], s)
    rng.shuffle(hist)
    ctx = [h + n for h in hist]
    tables, pool = _paged(rng, ctx, case["block"])
    # the root, then the kept nodes past it: a path that leaves at once wherever it can
    paths = []
    for k in keeps:
        k = min(k, n)
        low = 2 if n > case["keep"] else 1
        paths.append([0] + sorted(rng.sample(range(low, n), k - 1)) + [-1] * (n - k))
    shape = (pool, case["kv_heads"], case["block"], case["dim"])
    st = dict(case=case, k=_cache(gen, shape, case), v=_cache(gen, shape, case), tables=tables,
              ctx=_i32(ctx), qs=_i32(_starts([n] * s)), accepted=_i32(paths),
              count=_i32([min(k, n) for k in keeps]), nodes=n, err=_i32([0]))
    if case["cache"] == "e4m3":
        st["ks"], st["vs"] = _scales(gen, case["kv_heads"]), _scales(gen, case["kv_heads"])
    return st


# ---- one pass --------------------------------------------------------------
def run(state):
    return {"tree": _run_tree, "verify": _run_verify,
            "compact": _run_compact}[state["case"]["op"]](state)


def _values(cache, scales, dtype):
    """The cached values in `dtype`: codes times their kv head's scale, or the elements."""
    if scales is None:
        return cache.to(dtype)
    return cache.view(torch.float8_e4m3fn).to(dtype) * scales.to(dtype)[:, None, None]


def _lib():
    from paged_kv_cache_394_b200 import pagedkv
    return pagedkv


def _run_tree(st):
    case = st["case"]
    if own:
        args = (st["out"], st["q"], st["k"], st["v"], st["tables"], st["ctx"], st["qs"],
                st["parents"], st["scale"])
        tail = (case["kv_heads"], case["block"], st["most_ctx"], st["most_nodes"])
        if case["cache"] == "e4m3":
            _lib().paged_attn_tree_fp8(*args, st["ks"], st["vs"], *tail, dev_err=st["err"])
        else:
            _lib().paged_attn_tree(*args, *tail, dev_err=st["err"])
        return st["out"]
    s, c, n = case["seqs"], st["most_ctx"], st["most_nodes"]
    kv, group, dim = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    dev = st["q"].device
    qs, ctx = st["qs"].long(), st["ctx"].long()
    count = qs[1:] - qs[:-1]
    # gather every sequence's tokens through its table: [S, kv heads, context, dim]
    pos = torch.arange(c, device=dev)
    there = pos[None] < ctx[:, None]
    block = torch.where(there, st["tables"].long().clamp(min=0)[:, pos // case["block"]], 0)
    take = lambda cache, scales: torch.where(  # noqa: E731
        there[:, None, :, None],
        _values(cache.permute(0, 2, 1, 3)[block, pos % case["block"]].transpose(1, 2), scales,
                torch.float32), 0.0)
    k, v = take(st["k"], st.get("ks")), take(st["v"], st.get("vs"))
    # each sequence's nodes, padded to the largest tree
    node = torch.arange(n, device=dev)
    real = node[None] < count[:, None]
    at = torch.where(real, qs[:-1, None] + node, 0)
    q = st["q"][at].float().reshape(s, n, kv, group, dim).permute(0, 2, 3, 1, 4)
    logits = torch.matmul(q.reshape(s, kv, group * n, dim), k.transpose(2, 3)) * st["scale"]
    # a node sees its ancestors and itself: the closure of the parent relation
    par = torch.where(real, st["parents"].long()[at], -1)
    step = (par[:, :, None] == node).double() + torch.eye(n, dtype=torch.float64, device=dev)
    sees = torch.linalg.matrix_power(step, n) > 0
    local = pos[None] - (ctx - count)[:, None]  # the key's node, below 0 in the history
    mask = torch.gather(sees, 2, local.clamp(0, n - 1)[:, None].expand(s, n, c))
    mask = (mask | (local < 0)[:, None]) & there[:, None]
    logits = logits.reshape(s, kv, group, n, c).masked_fill_(~mask[:, None, None], -math.inf)
    e = torch.exp(logits - logits.amax(dim=-1, keepdim=True))
    o = torch.matmul(e.reshape(s, kv, group * n, c), v) / e.sum(dim=-1).reshape(
        s, kv, group * n, 1)
    o = o.reshape(s, kv * group, n, dim).transpose(1, 2)
    return o[real].to(st["q"].dtype)


def _run_verify(st):
    if own:
        _lib().verify_draft(st["accepted"], st["count"], st["next"], st["target"], st["tokens"],
                            st["parents"], st["qs"], st["u"], st["u_next"], st["nodes"],
                            draft_probs=st["draft"], dev_err=st["err"])
        return [st["accepted"], st["count"], st["next"]]
    s, n = st["accepted"].shape
    each = torch.arange(s, device=st["qs"].device)
    cur, z = torch.zeros_like(each), torch.ones(s, dtype=torch.float64, device=each.device)
    r = st["target"][each * n].double().clamp_(min=0)
    kept = [torch.ones_like(each, dtype=torch.bool)]
    for j in range(1, n):  # nodes in order: each is tried if its parent is the last accepted
        at = each * n + j
        x = st["tokens"][at].long()
        tried = st["parents"][at] == cur
        q = st["draft"][each * n + cur].double() if st["draft"] is not None else (
            torch.zeros_like(r).scatter_(1, x[:, None], 1.0))
        qx, rx = q.gather(1, x[:, None])[:, 0], r.gather(1, x[:, None])[:, 0]
        taken = tried & (st["u"][at].double() * qx * z < rx)
        rejected = tried & ~taken
        if st["draft"] is not None:
            left = (r / z[:, None] - q).clamp_(min=0)
            z_left = left.sum(dim=1)
        else:  # a token sure to be drafted: nothing of it is left
            left = r * (1 - q)
            z_left = z - rx
        r = torch.where(taken[:, None], st["target"][at].double().clamp(min=0),
                        torch.where(rejected[:, None], left, r))
        z = torch.where(taken, 1.0, torch.where(rejected, z_left, z))
        cur = torch.where(taken, j, cur)
        kept.append(taken)
    full = st["target"][each * n + cur].double().clamp_(min=0)
    r = torch.where((r.sum(dim=1) > 0)[:, None], r, full)
    c = torch.cumsum(r, dim=1)
    nxt = (c <= st["u_next"].double()[:, None] * c[:, -1:]).sum(dim=1)
    last = r.shape[1] - 1 - (r > 0).flip(1).int().argmax(dim=1)
    kept = torch.stack(kept, dim=1)
    order = torch.where(kept, torch.arange(n, device=each.device), n).sort(dim=1)[0]
    return [torch.where(order < n, order, -1).int(), kept.sum(dim=1).int(),
            torch.minimum(nxt, last).int()]


def _run_compact(st):
    case = st["case"]
    if own:
        _lib().compact_accepted(st["k"], st["v"], st["tables"], st["ctx"], st["qs"],
                                st["accepted"], st["count"], dev_err=st["err"])
    else:
        s, n = st["accepted"].shape
        hist = (st["ctx"] - n).long()[:, None]
        d = torch.arange(n, device=hist.device)
        real = d < st["count"][:, None]
        src = (hist + st["accepted"].long())[real]
        dst = (hist + d)[real]
        seq = torch.arange(s, device=hist.device)[:, None].expand(s, n)[real]
        table = st["tables"].long()
        bs = case["block"]
        frm, to = table[seq, src // bs], table[seq, dst // bs]
        st["k"][to, :, dst % bs] = st["k"][frm, :, src % bs]
        st["v"][to, :, dst % bs] = st["v"][frm, :, src % bs]
    if case["cache"] == "e4m3":  # the values that the codes stand for
        return [st["k"].view(torch.float8_e4m3fn), st["v"].view(torch.float8_e4m3fn)]
    return [st["k"], st["v"]]


# ---- the definitions in 64 bits, one sequence after the other ---------------
def exact(case, seed):
    st = prepare(case, seed)
    return {"tree": _exact_tree, "verify": _exact_verify, "compact": _exact_compact}[case["op"]](
        case, st)


def _ancestors(parents, j):
    seen = []
    while j >= 0:
        seen.append(j)
        j = parents[j]
    return seen


def _exact_tree(case, st):
    qs, ctx, par = st["qs"].tolist(), st["ctx"].tolist(), st["parents"].tolist()
    kv, bs, group = case["kv_heads"], case["block"], case["heads"] // case["kv_heads"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for i in range(case["seqs"]):
        a, b, c = qs[i], qs[i + 1], ctx[i]
        if a == b:
            continue
        blocks = st["tables"][i, :-(-c // bs)].long()
        flat = lambda x: x.transpose(0, 1).reshape(kv, -1, case["dim"])[:, :c]  # noqa: E731
        k = flat(_values(st["k"][blocks], st.get("ks"), torch.float64))
        v = flat(_values(st["v"][blocks], st.get("vs"), torch.float64))
        hist = c - (b - a)
        bias = torch.full((b - a, c), -math.inf, dtype=torch.float64, device="cuda")
        bias[:, :hist] = 0
        for j in range(b - a):
            bias[j, [hist + t for t in _ancestors(par[a:b], j)]] = 0
        for h in range(kv):
            q = st["q"][a:b, h * group:(h + 1) * group].double()
            x = torch.einsum("tgd,cd->gtc", q, k[h]) * st["scale"] + bias
            out[a:b, h * group:(h + 1) * group] = torch.einsum(
                "gtc,cd->tgd", torch.softmax(x, dim=-1), v[h])
    return out


def _exact_verify(case, st):
    s, n = st["accepted"].shape
    par, tok, u = st["parents"].tolist(), st["tokens"].tolist(), st["u"].tolist()
    paths, counts, nexts = [], [], []
    for i in range(s):
        p = st["target"][i * n:(i + 1) * n]
        path, res = [0], p[0].double()
        z = 1.0
        while True:
            cur = path[-1]
            children = [j for j in range(cur + 1, n) if par[i * n + j] == cur]
            for j in children:
                x = tok[i * n + j]
                if st["draft"] is not None:
                    q = st["draft"][i * n + cur].double()
                    qx = q[x].item()
                else:
                    qx = 1.0
                if u[i * n + j] * qx * z < res[x].item():
                    path.append(j)
                    res, z = p[j].double(), 1.0
                    break
                if st["draft"] is not None:
                    res = torch.relu(res / z - q)
                    z = res.sum().item()
                else:
                    z -= res[x].item()
                    res = res.clone()
                    res[x] = 0.0
            if path[-1] == cur:
                break
        if not res.sum().item() > 0:
            res = p[path[-1]].double()
        c = res.cumsum(0)
        above = torch.nonzero(c > st["u_next"][i].double() * c[-1])
        nexts.append(int(above[0]) if len(above) else int(torch.nonzero(res)[-1]))
        paths.append(path + [-1] * (n - len(path)))
        counts.append(len(path))
    return [_i32(paths), _i32(counts), _i32(nexts)]


def _exact_compact(case, st):
    before = [x.clone() for x in (st["k"], st["v"])]
    tables, ctx, bs = st["tables"].tolist(), st["ctx"].tolist(), case["block"]
    for i, (path, count) in enumerate(zip(st["accepted"].tolist(), st["count"].tolist())):
        for d in range(count):
            a, b = ctx[i] - case["nodes"] + path[d], ctx[i] - case["nodes"] + d
            for old, new in zip(before, (st["k"], st["v"])):
                new[tables[i][b // bs], :, b % bs] = old[tables[i][a // bs], :, a % bs]
    if case["cache"] == "e4m3":
        return [x.view(torch.float8_e4m3fn).double() for x in (st["k"], st["v"])]
    return [st["k"].double(), st["v"].double()]
