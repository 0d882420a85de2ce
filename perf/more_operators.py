"""Cases for the operators of a step of speculative decoding over the paged
cache: the plan of drafted trees (positions and ancestor masks from parents),
attention of a tree's tokens over the cache, verification of the drafted tokens
against the target's probabilities, and the commit of the accepted path (rows
moved in every layer's pools, lengths, blocks given back).

``run`` computes a case in its plain form (elementary torch operations), or,
with ``own`` set, by the calls a user of this package makes.  ``exact`` states
the same operators in 64 bits.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _plan(seqs, nodes_lo, nodes_hi, width, ctx_hi, padding, shape_seed):
    return {"op": "plan", "seqs": seqs, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "width": width, "ctx_lo": 0,
            "ctx_hi": ctx_hi, "lens": "log", "padding": padding, "shape_seed": shape_seed}


def _attend(seqs, nodes_lo, nodes_hi, width, ctx_lo, ctx_hi, lens, heads, kv_heads, dim, dtype, block, shape_seed):
    return {"op": "attend", "seqs": seqs, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "width": width,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "lens": lens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "dtype": dtype, "block": block, "shape_seed": shape_seed}


def _verify(seqs, nodes_lo, nodes_hi, width, vocab, dtype, drafted, spread, shape_seed):
    return {"op": "verify", "seqs": seqs, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "width": width, "ctx_lo": 0,
            "ctx_hi": 64, "lens": "uniform", "vocab": vocab, "dtype": dtype, "drafted": drafted, "spread": spread,
            "shape_seed": shape_seed}


def _commit(seqs, nodes_lo, nodes_hi, width, ctx_lo, ctx_hi, layers, kv_heads, dim, dtype, block, ring, shape_seed):
    return {"op": "commit", "seqs": seqs, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "width": width,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "lens": "uniform", "layers": layers, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "block": block, "ring": ring, "shape_seed": shape_seed}


def listed():
    return [
        # the trees of a server's batch, 16 nodes each, three candidates wide
        {"name": "plan_batch", **_plan(64, 16, 16, 3, 8192, 0, 1)},
        # thousands of ragged trees of up to 61 nodes, padded to a captured size
        {"name": "plan_large", **_plan(2048, 1, 61, 5, 2048, 333, 2)},
        # one user of an idle server, a tree of 8 over a short context: latency of a single small call
        {"name": "attend_one", **_attend(1, 8, 8, 2, 700, 700, "uniform", 8, 2, 128, "bf16", 16, 3)},
        # the decode batch of this repository (Llama-8B-shaped heads, lognormal contexts), trees of 16
        {"name": "attend_batch", **_attend(64, 16, 16, 3, 16, 8192, "lognormal", 32, 8, 128, "bf16", 16, 4)},
        # wide trees of up to 64 nodes: 256 query rows for each KV head
        {"name": "attend_wide", **_attend(32, 40, 64, 6, 1024, 8192, "uniform", 32, 8, 128, "bf16", 16, 5)},
        # as many KV heads as heads (OPT-13B-shaped), ragged trees
        {"name": "attend_mha", **_attend(24, 1, 25, 3, 128, 2048, "uniform", 40, 40, 128, "f16", 16, 6)},
        # few long documents, the length of the long-context workload, narrow heads and large blocks
        {"name": "attend_long", **_attend(3, 31, 31, 4, 30001, 32768, "uniform", 16, 4, 64, "bf16", 32, 7)},
        # a chain of five drafted tokens of one user
        {"name": "verify_one", **_verify(1, 6, 6, 1, 32000, "f32", True, 0.5, 8)},
        # a batch of trees against a large vocabulary, probabilities of draft and target
        {"name": "verify_batch", **_verify(64, 12, 12, 3, 128256, "f32", True, 0.8, 9)},
        # many users, candidates without probabilities (a lookup in the prompt), an odd vocabulary, 16-bit rows
        {"name": "verify_lookup", **_verify(200, 1, 9, 2, 50021, "bf16", False, 0.5, 10)},
        # the accepted paths of one user's step, few layers
        {"name": "commit_one", **_commit(1, 16, 16, 3, 300, 300, 4, 8, 128, "bf16", 16, True, 11)},
        # a batch's accepted paths in every layer of a model of 32 layers
        {"name": "commit_batch", **_commit(96, 16, 24, 3, 20, 200, 32, 8, 128, "bf16", 16, True, 12)},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(8, 2), (32, 8), (40, 40), (16, 8), (4, 4), (16, 2), (8, 1), (12, 4)]


def draw(rng):
    op = rng.choice(["plan", "attend", "attend", "verify", "commit"])
    shape_seed = rng.randrange(1 << 20)
    hi = _log_int(rng, 1, 96)
    lo = rng.choice([1, max(1, hi // 2), hi])
    width = rng.choice([1, 2, 3, 6])
    if op == "plan":
        return _plan(_log_int(rng, 1, 2048), lo, hi, width, _log_int(rng, 16, 32768),
                     rng.choice([0, rng.randrange(1, 400)]), shape_seed)
    heads, kv_heads = rng.choice(_HEADS)
    dim, block = rng.choice([64, 128]), rng.choice([8, 16, 32])
    if op == "attend":
        ctx_hi = _log_int(rng, 16, 16384)
        room = min((1 << 27) // (ctx_hi * kv_heads * dim), (1 << 34) // (ctx_hi * heads * dim * hi))
        seqs = _log_int(rng, 1, max(1, min(128, room)))
        return _attend(seqs, lo, hi, width, rng.choice([0, ctx_hi // 2, ctx_hi]), ctx_hi,
                       rng.choice(["uniform", "log"]), heads, kv_heads, dim, rng.choice(["bf16", "f16"]), block,
                       shape_seed)
    if op == "verify":
        vocab = _log_int(rng, 500, 160000)
        hi = min(hi, 24)
        seqs = _log_int(rng, 1, max(1, min(256, (1 << 26) // (vocab * hi))))
        return _verify(seqs, min(lo, hi), hi, width, vocab, rng.choice(["f32", "f32", "bf16", "f16"]),
                       rng.random() < 0.7, rng.choice([0.2, 0.6, 1.5]), shape_seed)
    dtype = rng.choice(["bf16", "f16", "f32"])
    layers = _log_int(rng, 1, 24)
    seqs = _log_int(rng, 1, max(1, min(96, (1 << 27) // (layers * kv_heads * dim * (hi + 100)))))
    return _commit(seqs, lo, hi, width, rng.choice([0, 64]), 100, layers, kv_heads, dim, dtype, block,
                   rng.random() < 0.7, shape_seed)


def _shapes(case):
    """Of every sequence: tokens cached before the tree, parents of its nodes, an accepted path."""
    r = random.Random(case["shape_seed"])
    lo, hi, out = case["ctx_lo"], case["ctx_hi"], []
    for _ in range(case["seqs"]):
        n = r.randint(case["nodes_lo"], case["nodes_hi"])
        if case["lens"] == "uniform":
            ctx = r.randint(lo, hi)
        elif case["lens"] == "log":
            ctx = max(lo, _log_int(r, 1, max(1, hi)))
        else:
            ctx = min(hi, max(lo, int(round(r.lognormvariate(math.log(1024), 1.0)))))
        parents = [-1] + [r.randrange(max(0, i - case["width"]), i) for i in range(1, n)]
        children = [[] for _ in range(n)]
        for i in range(1, n):
            children[parents[i]].append(i)
        path = [0]
        while children[path[-1]] and r.random() < 0.75:
            path.append(r.choice(children[path[-1]]))
        out.append((ctx, parents, path))
    return out


def _ceil(a, b):
    return -(-a // b)


def _words(case):
    return _ceil(case["nodes_hi"], 64)


def work(case):
    shapes = _shapes(case)
    tokens = sum(len(parents) for _, parents, _ in shapes)
    seqs = len(shapes)
    if case["op"] == "plan":
        total = tokens + case["padding"]
        return {"bytes": 4 * tokens + 8 * seqs + (4 + 8 * _words(case)) * total, "flops": tokens}
    if case["op"] == "attend":
        h, hkv, d, e = case["heads"], case["kv_heads"], case["dim"], SIZE[case["dtype"]]
        cached = sum(ctx + len(parents) for ctx, parents, _ in shapes)
        pairs = sum(ctx * len(parents) + sum(len(a) for a in _ancestors(parents)) for ctx, parents, _ in shapes)
        return {"bytes": 2 * cached * hkv * d * e + 2 * tokens * h * d * e + 8 * tokens * _words(case)
                + 4 * sum(_ceil(ctx + len(parents), case["block"]) for ctx, parents, _ in shapes),
                "flops": 4 * d * h * pairs}
    if case["op"] == "verify":
        rows = 2 if case["drafted"] else 1  # of each sequence: the distribution that its last token is drawn from
        row_bytes = case["vocab"] * SIZE[case["dtype"]]
        return {"bytes": seqs * (rows * row_bytes + 8) + 16 * tokens, "flops": seqs * case["vocab"] * (rows + 1)}
    moved = sum(sum(at != i for i, at in enumerate(path)) for _, _, path in shapes)
    row = case["kv_heads"] * case["dim"] * SIZE[case["dtype"]]
    return {"bytes": 4 * moved * case["layers"] * row + 16 * seqs + 4 * tokens, "flops": moved}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _ancestors(parents):
    """Of every node: itself and the nodes above it."""
    out = []
    for i, p in enumerate(parents):
        out.append(([] if p < 0 else out[p]) + [i])
    return out


def _mask_words(parents, words):
    rows = []
    for nodes in _ancestors(parents):
        bits = sum(1 << j for j in nodes)
        row = [(bits >> (64 * w)) & (2 ** 64 - 1) for w in range(words)]
        rows.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in row])
    return rows


def _tables(lens, block, spare, seed):
    """Block tables of sequences of these lengths in a shuffled pool, and the ids left over."""
    g = torch.Generator()
    g.manual_seed(seed)
    held = [_ceil(n, block) for n in lens]
    total = sum(held) + spare
    order = torch.randperm(total, generator=g).int()
    rows = torch.full((len(lens), max(max(held), 1) + 2), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(held):
        rows[s, :n] = order[at:at + n]
        at += n
    return rows.cuda(), order[at:], total


def prepare(case, seed):
    st = dict(case)
    shapes = _shapes(case)
    lens = [len(parents) for _, parents, _ in shapes]
    n = sum(lens)
    total = n + case.get("padding", 0)
    start = [0]
    for x in lens:
        start.append(start[-1] + x)
    st["start"] = _i32(start)
    st["tokens"] = n
    g = _generator(seed)
    if case["op"] == "plan":
        # lengths and parents change from step to step: other ones for every seed
        r = random.Random(seed)
        ctx = [max(0, c + r.randrange(-3, 4)) for c, _, _ in shapes]
        parents = []
        for x in lens:
            parents += [-1] + [r.randrange(max(0, i - case["width"]), i) for i in range(1, x)]
        st["parents"] = _i32(parents + [-1] * (total - n))
        st["ctx"] = _i32([c + x for c, x in zip(ctx, lens)])
        st["deepest"] = max(lens)
        return st
    if case["op"] == "attend":
        h, hkv, d, dt, b = case["heads"], case["kv_heads"], case["dim"], DTYPE[case["dtype"]], case["block"]
        ctx = [c + x for (c, _, _), x in zip(shapes, lens)]
        st["tables"], _, blocks = _tables(ctx, b, 5, seed)
        st["ctx"] = _i32(ctx)
        st["q"] = torch.randn(n, h, d, generator=g, device="cuda").to(dt)
        st["k"] = torch.randn(blocks, hkv, b, d, generator=g, device="cuda").to(dt)
        st["v"] = torch.randn(blocks, hkv, b, d, generator=g, device="cuda").to(dt)
        st["mask"] = torch.tensor([w for _, parents, _ in shapes for w in _mask_words(parents, _words(case))],
                                  dtype=torch.int64, device="cuda")
        st |= {"scale": d ** -0.5, "ctx_list": ctx, "nodes": lens}
        return st
    if case["op"] == "verify":
        v, dt = case["vocab"], DTYPE[case["dtype"]]
        parents = [p for _, ps, _ in shapes for p in ps]
        st["parents"] = _i32(parents)
        logits = torch.randn(n, v, generator=g, device="cuda") * 2.5
        st["target"] = torch.softmax(logits, 1).to(dt)
        logits += torch.randn(n, v, generator=g, device="cuda") * case["spread"]
        draft = torch.softmax(logits, 1).to(dt)
        # every node's candidates were drawn from its row of the draft
        first = [a for a, x in zip(start, lens) for _ in range(x)]
        above = torch.tensor([a + max(p, 0) for a, p in zip(first, parents)], device="cuda")
        noise = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
        tokens = torch.empty(n, dtype=torch.int32, device="cuda")
        for r in range(0, n, 256):
            cum = draft[above[r:r + 256]].double().cumsum(1)
            at = noise[r:r + 256, None] * cum[:, -1:]
            tokens[r:r + 256] = torch.searchsorted(cum, at, right=True).clamp_(max=v - 1)[:, 0].int()
        st["ids"] = tokens
        st["draft"] = draft if case["drafted"] else None
        st["accept_u"] = torch.rand(n, generator=g, device="cuda")
        st["sample_u"] = torch.rand(case["seqs"], generator=g, device="cuda")
        st["longest"] = max(lens)
        return st
    hkv, d, dt, b = case["kv_heads"], case["dim"], DTYPE[case["dtype"]], case["block"]
    ctx = [c + x for (c, _, _), x in zip(shapes, lens)]
    st["tables"], left, blocks = _tables(ctx, b, 7, seed)
    st["ctx"] = _i32(ctx)
    # every layer's pools in one allocation, keys and then values
    st["pools"] = torch.randn(2, case["layers"], blocks, hkv, b, d, generator=g, device="cuda").to(dt)
    st["k"], st["v"] = list(st["pools"][0]), list(st["pools"][1])
    st["path"] = _i32([x for (_, ps, path) in shapes for x in path + [-1] * (len(ps) - len(path))])
    st["accepted"] = _i32([len(path) for _, _, path in shapes])
    st["ring"] = st["free"] = None
    if case["ring"]:
        head = int(torch.randint(blocks, (1,), generator=g, device="cuda"))  # the ring starts anywhere and wraps
        ring = torch.full((blocks,), -1, dtype=torch.int32)
        ring[(head + torch.arange(len(left))) % blocks] = left
        st["ring"], st["free"] = ring.cuda(), _i32([head, len(left)])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _sequence_of(start, rows):
    t = torch.arange(rows, device="cuda")
    return torch.searchsorted(start[1:], t, right=True).clamp_(max=start.numel() - 2), t


def _plain_plan(st):
    start, n = st["start"].long(), st["tokens"]
    total, words = st["parents"].numel(), _words(st)
    positions = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    mask = torch.zeros(total, words, dtype=torch.int64, device="cuda")
    seq, t = _sequence_of(start, n)
    base = start[seq]
    at = t - base
    depth = torch.zeros(n, dtype=torch.int64, device="cuda")
    parents = st["parents"][:n].long()
    one = torch.ones((), dtype=torch.int64, device="cuda")
    for step in range(st["deepest"]):
        alive = at >= 0
        here = at.clamp(min=0)
        bit = torch.where(alive, one << (here % 64), 0)
        mask[:n].scatter_add_(1, (here // 64)[:, None], bit[:, None])
        above = torch.where(alive, parents[base + here], -1)
        depth += above >= 0
        at = above
    grown = start[1:] - start[:-1]
    positions[:n] = ((st["ctx"].long() - grown)[seq] + depth).int()
    return {"positions": positions, "tree_mask": mask}


def _plain_attend(st):
    q, h, hkv, d, b = st["q"], st["heads"], st["kv_heads"], st["dim"], st["block"]
    g = h // hkv
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    start = st["start"].long()
    seqs, n = st["seqs"], max(st["nodes"])
    longest = max(st["ctx_list"])
    # as many sequences at a time as the scores and the gathered rows have room for
    few = max(1, (1 << 30) // max(h * n * longest, 2 * hkv * d * longest))
    for s0 in range(0, seqs, few):
        s1 = min(seqs, s0 + few)
        size = max(st["ctx_list"][s0:s1])
        pos = torch.arange(size, device="cuda")
        ctx = st["ctx"][s0:s1].long()
        there = pos < ctx[:, None]
        block = torch.where(there, st["tables"][s0:s1].long()[:, pos // b], 0)
        k = st["k"][block, :, pos % b].float()  # [sequences][positions][KV heads][d]
        v = st["v"][block, :, pos % b].float()
        nodes = (start[1:] - start[:-1])[s0:s1]
        i = torch.arange(n, device="cuda")
        row = torch.minimum(start[s0:s1, None] + i, start[-1] - 1)
        x = q[row].float().view(s1 - s0, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(s1 - s0, hkv, g * n, d)
        z = (x @ k.permute(0, 2, 3, 1)).view(s1 - s0, hkv, g, n, size) * st["scale"]
        # a row attends to every position before the tree and to the nodes of its mask
        node = pos - (ctx - nodes)[:, None]
        within = node.clamp(min=0, max=64 * st["mask"].shape[1] - 1)
        words = st["mask"][row].gather(2, (within // 64)[:, None].expand(-1, n, -1))
        attends = (node < 0)[:, None] | ((words >> (within % 64)[:, None]) & 1).bool()
        z.masked_fill_(~(attends & there[:, None])[:, None, None], float("-inf"))
        z -= z.amax(-1, keepdim=True)
        z.exp_()
        weight = z.sum(-1, keepdim=True)
        v = torch.where(there[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)
        o = (z.view(s1 - s0, hkv, g * n, size) @ v).view(s1 - s0, hkv, g, n, d) / weight
        real = i < nodes[:, None]
        out[row[real]] = o.permute(0, 3, 1, 2, 4).reshape(s1 - s0, n, h, d)[real]
    return out.to(q.dtype)


def _plain_verify(st):
    start, parents, ids, seqs = st["start"].long(), st["parents"].long(), st["ids"].long(), st["seqs"]
    target, draft = st["target"], st["draft"]
    f64 = torch.float64
    every = torch.arange(seqs, device="cuda")
    nodes = start[1:] - start[:-1]
    now = torch.zeros(seqs, dtype=torch.int64, device="cuda")  # last accepted node
    # weights max(p - c q, 0) of the candidates still possible, and their sum
    c = torch.zeros(seqs, dtype=f64, device="cuda")
    s = torch.ones(seqs, dtype=f64, device="cuda")
    # without a draft's rows: the tokens refused at this node, and whether nothing is left
    refused = torch.full((seqs, st["longest"]), -1, dtype=torch.int64, device="cuda")
    count = torch.ones(seqs, dtype=torch.int64, device="cuda")
    path = torch.full((ids.numel(),), -1, dtype=torch.int32, device="cuda")
    path[start[:-1]] = 0
    spent = torch.zeros(seqs, dtype=torch.bool, device="cuda")
    for i in range(1, st["longest"]):
        node = torch.minimum(start[:-1] + i, start[-1] - 1)
        tested = (i < nodes) & (parents[node] == now) & ~spent
        row, x = start[:-1] + now, ids[node]
        p = target[row, x].to(f64)
        u = st["accept_u"][node].to(f64)
        if draft is not None:
            q = draft[row, x].to(f64)
            accept = tested & (u * q * s < (p - c * q).clamp(min=0))
        else:
            p = torch.where((refused == x[:, None]).any(1), 0.0, p)
            accept = tested & (u * s < p)
        reject = tested & ~accept
        if draft is not None:
            c = torch.where(reject, c + s, c)
            left = torch.empty(seqs, dtype=f64, device="cuda")
            for r in range(0, seqs, 64):
                rows = row[r:r + 64]
                left[r:r + 64] = (target[rows].to(f64) - c[r:r + 64, None] * draft[rows].to(f64)).clamp_(min=0).sum(1)
            s = torch.where(reject, left, s)
        else:
            refused[:, i] = torch.where(reject, x, -1)
            s = torch.where(reject, (s - p).clamp(min=0), s)
        spent |= reject & (s == 0) if draft is not None else False
        # on the accepted node everything starts anew
        now = torch.where(accept, i, now)
        c = torch.where(accept, 0.0, c)
        s = torch.where(accept, 1.0, s)
        refused = torch.where(accept[:, None], -1, refused)
        at = start[:-1] + torch.minimum(count, nodes - 1)
        path[at] = torch.where(accept, i, path[at].long()).int()
        count += accept
    token = torch.empty(seqs, dtype=torch.int32, device="cuda")
    for r in range(0, seqs, 64):
        some = every[r:r + 64]
        row = start[some] + now[some]
        p = target[row].to(f64)
        w = p
        if draft is not None:
            w = (p - c[some, None] * draft[row].to(f64)).clamp_(min=0)
            w = torch.where(spent[some, None], p, w)
        else:
            gone = refused[some]
            w = p.scatter(1, gone.clamp(min=0), torch.where(gone < 0, p.gather(1, gone.clamp(min=0)), 0.0))
            # a token that stands for "none" must not bring back one that was refused
            zero = ((gone == 0).any(1, keepdim=True)) & (torch.arange(p.shape[1], device="cuda") == 0)
            w = torch.where(zero, 0.0, w)
            w = torch.where((w.sum(1, keepdim=True) == 0), p, w)
        cum = w.cumsum(1)
        at = st["sample_u"][some].to(f64)[:, None] * cum[:, -1:]
        last = (w > 0).to(torch.int64).cumsum(1).argmax(1)
        token[r:r + 64] = torch.minimum((cum <= at).sum(1), last).int()
    return {"accepted_lens": count.int(), "path": path, "next_tokens": token}


def _plain_commit(st):
    b, tables, start = st["block"], st["tables"].long(), st["start"].long()
    ctx, kept, path = st["ctx"].long(), st["accepted"].long(), st["path"].long()
    nodes = start[1:] - start[:-1]
    seq, t = _sequence_of(start, st["tokens"])
    base, i = (ctx - nodes)[seq], t - start[seq]
    moves = torch.nonzero((i < kept[seq]) & (path != i))[:, 0]
    seq, base, i = seq[moves], base[moves], i[moves]
    here, there = base + path[moves], base + i
    here_block, there_block = tables[seq, here // b], tables[seq, there // b]
    for pool in st["k"] + st["v"]:
        pool[there_block, :, there % b] = pool[here_block, :, here % b]
    after = ctx - nodes + kept
    out = {"pools": st["pools"], "context_lens": after.int()}
    if st["ring"] is not None:
        ring, (head, count) = st["ring"], st["free"].long()
        held, need = (ctx + b - 1) // b, (after + b - 1) // b
        given = held - need
        column = torch.arange(tables.shape[1], device="cuda")
        back = (column >= need[:, None]) & (column < held[:, None])
        order = (given.cumsum(0) - given - need)[:, None] + column
        ring[((head + count + order) % ring.numel())[back]] = tables[back].int()
        out |= {"free_state": torch.stack([head, count + given.sum()]).int(), "free_ring": ring}
    return out


def run(st):
    if not own:
        return {"plan": _plain_plan, "attend": _plain_attend, "verify": _plain_verify,
                "commit": _plain_commit}[st["op"]](st)
    from paged_kv_cache_132_gb300 import api

    if st["op"] == "plan":
        return api.plan_tree(st["parents"], st["start"], st["ctx"], st["nodes_hi"])._asdict()
    if st["op"] == "attend":
        return api.tree_attention(st["q"], st["start"], st["mask"], st["k"], st["v"], st["tables"], st["ctx"],
                                  st["scale"])
    if st["op"] == "verify":
        return api.verify_tree(st["ids"], st["parents"], st["start"], st["target"], st["draft"], st["accept_u"],
                               st["sample_u"])._asdict()
    done = api.commit_tree(st["k"], st["v"], st["start"], st["path"], st["accepted"], st["ctx"], st["tables"],
                           free_ring=st["ring"], free_state=st["free"])
    out = {"pools": st["pools"], "context_lens": done.context_lens}
    if st["ring"] is not None:
        out |= {"free_state": done.free_state, "free_ring": st["ring"]}
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _split(flat, start):
    return [flat[a:e] for a, e in zip(start, start[1:])]


def _exact_plan(case, seed):
    st = prepare(case, seed)
    start, words = st["start"].tolist(), _words(case)
    positions, mask = [], []
    for parents, ctx in zip(_split(st["parents"].tolist(), start), st["ctx"].tolist()):
        positions += [ctx - len(parents) + len(a) - 1 for a in _ancestors(parents)]
        mask += _mask_words(parents, words)
    positions += [-1] * case["padding"]
    mask += [[0] * words] * case["padding"]
    return {"positions": torch.tensor(positions, dtype=torch.int32),
            "tree_mask": torch.tensor(mask, dtype=torch.int64)}


def _exact_attend(case, seed):
    st = prepare(case, seed)
    g, b = case["heads"] // case["kv_heads"], case["block"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    begin = 0
    for s, (ctx, parents, _) in enumerate(_shapes(case)):
        n = len(parents)
        pos = torch.arange(ctx + n, device="cuda")
        block, offset = st["tables"][s].long()[pos // b], pos % b
        hidden = torch.ones(n, n, dtype=torch.bool)
        for i, nodes in enumerate(_ancestors(parents)):
            hidden[i, nodes] = False
        hidden = torch.cat([torch.zeros(n, ctx, dtype=torch.bool), hidden], 1).cuda()
        for h in range(case["heads"]):
            k = st["k"][block, h // g, offset].double()
            v = st["v"][block, h // g, offset].double()
            z = torch.mm(st["q"][begin:begin + n, h].double(), k.T) * st["scale"]
            out[begin:begin + n, h] = torch.softmax(z.masked_fill(hidden, -math.inf), dim=1) @ v
        begin += n
    return out


def _exact_verify(case, seed):
    st = prepare(case, seed)
    start, vocab = st["start"].tolist(), case["vocab"]
    ids, accept_u = st["ids"].tolist(), st["accept_u"].tolist()
    sample_u = st["sample_u"].tolist()
    counts, paths, tokens = [], [], []

    def row_of(probs, row):
        return probs[row].double().cpu().numpy()

    for s, parents in enumerate(_split(st["parents"].tolist(), start)):
        first, path = start[s], [0]
        going = True
        while going:
            row = first + path[-1]
            p = row_of(st["target"], row)
            left, scale = p, 1.0  # weights still possible, and what they are divided by
            used, going = 0.0, False
            q = row_of(st["draft"], row) if case["drafted"] else None
            for i in [j for j, above in enumerate(parents) if above == path[-1]]:
                x, u = ids[first + i], accept_u[first + i]
                if u * (q[x] if case["drafted"] else 1.0) * scale < left[x]:
                    path.append(i)
                    going = True
                    break
                if case["drafted"]:
                    used += scale
                    left = np.maximum(p - used * q, 0.0)
                    scale = math.fsum(left)
                    if scale == 0.0:
                        break
                else:
                    scale = max(scale - left[x], 0.0)
                    left = left.copy()
                    left[x] = 0.0
        if not left.any():
            left = p
        below = np.cumsum(left)
        at = int(np.searchsorted(below, sample_u[s] * below[-1], side="right"))
        tokens.append(min(at, int(np.flatnonzero(left)[-1]), vocab - 1))
        counts.append(len(path))
        paths += path + [-1] * (len(parents) - len(path))
    as_i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"accepted_lens": as_i32(counts), "path": as_i32(paths), "next_tokens": as_i32(tokens)}


def _exact_commit(case, seed):
    st = prepare(case, seed)
    b, tables = case["block"], st["tables"].tolist()
    src, dst, after, back = [], [], [], []
    for s, (ctx, parents, path) in enumerate(_shapes(case)):
        for i, node in enumerate(path):
            src.append(tables[s][(ctx + node) // b] * b + (ctx + node) % b)
            dst.append(tables[s][(ctx + i) // b] * b + (ctx + i) % b)
        after.append(ctx + len(path))
        back += tables[s][_ceil(after[-1], b):_ceil(ctx + len(parents), b)]
    src, dst = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
    for pool in st["k"] + st["v"]:
        flat = pool.transpose(1, 2).flatten(0, 1).clone()  # a row for each slot
        flat[dst] = flat[src]
        pool.copy_(flat.unflatten(0, (-1, b)).transpose(1, 2))
    out = {"pools": st["pools"], "context_lens": torch.tensor(after, dtype=torch.int32)}
    if case["ring"]:
        ring, (head, count) = st["ring"].tolist(), st["free"].tolist()
        for j, block in enumerate(back):
            ring[(head + count + j) % len(ring)] = block
        out |= {"free_state": torch.tensor([head, count + len(back)], dtype=torch.int32),
                "free_ring": torch.tensor(ring, dtype=torch.int32)}
    return out


def exact(case, seed):
    return {"plan": _exact_plan, "attend": _exact_attend, "verify": _exact_verify, "commit": _exact_commit}[
        case["op"]](case, seed)
