"""Cases for the operators around the paged cache's attention: the plan of a
step (block tables and slots from request lengths), the rotary embedding fused
with the cache write, and causal attention over whole packed prompts.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, rounded once), or, with ``own`` set, by the calls a user of this package
makes.  ``exact`` states the same operators in 64 bits.
"""
from __future__ import annotations

import math
import random
from collections import deque

import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
ROPE_BASE = 10000.0


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _prompt(seqs, lo, hi, heads, kv_heads, dim, dtype, fused, lens_seed, lens="uniform"):
    return {"op": "prompt", "seqs": seqs, "lo": lo, "hi": hi, "lens": lens, "lens_seed": lens_seed, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "fused": fused}


def _rotary(tokens, padding, heads, kv_heads, dim, rot, dtype, interleaved, keep_key, fused, block, far):
    return {"op": "rotary", "tokens": tokens, "padding": padding, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "dtype": dtype, "interleaved": interleaved, "keep_key": keep_key, "fused": fused,
            "block": block, "far": far}


def _plan(seqs, prompts, finished, idle, lo, hi, ctx_hi, block, padding, lens_seed):
    return {"op": "plan", "seqs": seqs, "prompts": prompts, "finished": finished, "idle": idle, "lo": lo, "hi": hi,
            "ctx_hi": ctx_hi, "block": block, "padding": padding, "lens_seed": lens_seed}


def listed():
    return [
        # one short question to an idle server: the latency of a single small call
        {"name": "prompt_one_short", **_prompt(1, 17, 17, 8, 2, 64, "bf16", False, 1)},
        # a prefill batch of chat requests, Llama-8B-shaped heads, sliced out of the fused projection
        {"name": "prompt_chat", **_prompt(32, 128, 1024, 32, 8, 128, "bf16", True, 2)},
        # a prefill batch with as many KV heads as heads, OPT-13B-shaped, separate projections
        {"name": "prompt_mha", **_prompt(16, 128, 1024, 40, 40, 128, "f16", False, 3)},
        # many short, ragged prompts (classification, search queries), narrow heads
        {"name": "prompt_many_short", **_prompt(256, 1, 130, 16, 8, 64, "f16", False, 4)},
        # prompts whose lengths spread lognormally, as the decode batches of this repository do
        {"name": "prompt_lognormal", **_prompt(16, 16, 4096, 32, 8, 128, "bf16", False, 5, "lognormal")},
        # one long document, the length of the long-context workload
        {"name": "prompt_long", **_prompt(1, 32768, 32768, 32, 8, 128, "bf16", False, 6)},
        # a decode step: every sequence grows by one token
        {"name": "plan_decode", **_plan(256, 0, 0, 0, 1, 1, 8192, 16, 0, 7)},
        # a mixed step: new prompts, running sequences, finished and idle ones, padded to a captured size
        {"name": "plan_mixed", **_plan(256, 32, 16, 16, 128, 1024, 8192, 16, 501, 8)},
        # a large server's step over thousands of sequences
        {"name": "plan_large", **_plan(4096, 128, 200, 96, 128, 1024, 2048, 16, 0, 9)},
        # a decode step's new tokens, Llama-8B-shaped
        {"name": "rotary_decode", **_rotary(256, 0, 32, 8, 128, 128, "bf16", False, False, True, 16, 8192)},
        # a prefill batch's new tokens; the rotated keys are kept for the prompt's attention
        {"name": "rotary_prompt", **_rotary(20588, 0, 32, 8, 128, 128, "bf16", False, True, True, 16, 32768)},
        # interleaved pairs over half of each head, 32-bit pools, an odd number of tokens and padded rows
        {"name": "rotary_partial_f32", **_rotary(333, 7, 8, 4, 64, 32, "f32", True, True, False, 8, 2048)},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(8, 2), (32, 8), (40, 40), (16, 8), (4, 4), (16, 2), (8, 1), (12, 4)]


def draw(rng):
    op = rng.choice(["prompt", "rotary", "plan"])
    heads, kv_heads = rng.choice(_HEADS)
    dim = rng.choice([64, 128])
    lens_seed = rng.randrange(1 << 20)
    if op == "prompt":
        hi = _log_int(rng, 1, 8192)
        seqs = _log_int(rng, 1, max(1, min(256, 32768 // hi)))
        kind = rng.choice(["uniform", "lognormal"])
        return _prompt(seqs, rng.choice([1, max(1, hi // 8), hi]), hi, heads, kv_heads, dim,
                       rng.choice(["bf16", "f16"]), rng.random() < 0.5, lens_seed, kind)
    if op == "rotary":
        dtype = rng.choice(["bf16", "f16", "f32"])
        tokens = _log_int(rng, 1, 8192 if dtype == "f32" else 16384)
        return _rotary(tokens, rng.choice([0, rng.randrange(1, 40)]), heads, kv_heads, dim,
                       rng.choice([dim, dim // 2, 32]), dtype, rng.random() < 0.5, rng.random() < 0.5,
                       rng.random() < 0.5, rng.choice([8, 16, 32]), _log_int(rng, max(tokens // 64, 256), 131072))
    seqs = _log_int(rng, 1, 4096)
    prompts = min(seqs, rng.choice([0, 1, seqs // 16, seqs // 4, 128]))
    left = seqs - prompts
    finished = left // rng.choice([1000, 16, 4])
    hi = _log_int(rng, 1, 1024)
    return _plan(seqs, prompts, finished, (left - finished) // rng.choice([1000, 8]), rng.choice([1, max(1, hi // 8)]),
                 hi, _log_int(rng, 16, 4096), rng.choice([8, 16, 32]), rng.choice([0, rng.randrange(1, 700)]),
                 lens_seed)


def _lengths(case):
    r = random.Random(case["lens_seed"])
    lo, hi, n = case["lo"], case["hi"], case["seqs"]
    if case["lens"] == "uniform":
        return [r.randint(lo, hi) for _ in range(n)]
    mu = math.log(max(1.0, hi / 4))
    return [min(hi, max(lo, int(round(r.lognormvariate(mu, 1.0))))) for _ in range(n)]


def _roles(case):
    """(context, new) of every sequence of a plan; new = -1: finished, 0: idle."""
    r = random.Random(case["lens_seed"])
    kinds = ["prompt"] * case["prompts"] + ["finished"] * case["finished"] + ["idle"] * case["idle"]
    kinds += ["decode"] * (case["seqs"] - len(kinds))
    r.shuffle(kinds)
    out = []
    for k in kinds:
        ctx = 0 if k == "prompt" else _log_int(r, 1, case["ctx_hi"])
        out.append((ctx, {"prompt": r.randint(case["lo"], case["hi"]), "finished": -1, "idle": 0, "decode": 1}[k]))
    return out


def _ceil(a, b):
    return -(-a // b)


def work(case):
    if case["op"] == "prompt":
        lens = _lengths(case)
        t, h, hkv, d = sum(lens), case["heads"], case["kv_heads"], case["dim"]
        return {"bytes": 2 * t * (h + hkv) * d * SIZE[case["dtype"]] + 4 * (len(lens) + 1),
                "flops": 4 * d * h * sum(n * (n + 1) // 2 for n in lens)}
    if case["op"] == "rotary":
        t, h, hkv, d, e = case["tokens"], case["heads"], case["kv_heads"], case["dim"], SIZE[case["dtype"]]
        rows = 2 * h + (5 if case["keep_key"] else 4) * hkv  # read and written head rows of a token
        tables = 4 * case["rot"] * min(t, case["far"])
        return {"bytes": t * (rows * d * e + 12) + tables, "flops": 3 * t * (h + hkv) * case["rot"]}
    b, roles = case["block"], _roles(case)
    s, tokens = len(roles), sum(max(0, n) for _, n in roles)
    taken = sum(_ceil(c + n, b) - _ceil(c, b) for c, n in roles if n > 0)
    given = sum(_ceil(c, b) for c, n in roles if n < 0)
    return {"bytes": 16 * s + 8 * taken + 8 * given + 12 * (tokens + case["padding"]), "flops": tokens}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _qkv(case, tokens, seed):
    """q, k, v of every token; with "fused" they are slices of one projection's rows."""
    h, hkv, d, dt = case["heads"], case["kv_heads"], case["dim"], DTYPE[case["dtype"]]
    rows = torch.randn(tokens, (h + 2 * hkv) * d, generator=_generator(seed), device="cuda").to(dt)
    q, k, v = (x.unflatten(1, (-1, d)) for x in rows.split([h * d, hkv * d, hkv * d], dim=1))
    return (q, k, v) if case["fused"] else (q.contiguous(), k.contiguous(), v.contiguous())


def _cos_sin(positions, rot):
    """The table a model keeps: row p holds cos and then sin of its rot/2 angles, made in 64 bits."""
    inv = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _prepare_plan(case, seed):
    b, roles = case["block"], _roles(case)
    g = torch.Generator()
    g.manual_seed(seed)
    ctx = torch.tensor([c for c, _ in roles], dtype=torch.int32)
    new = torch.tensor([n for _, n in roles], dtype=torch.int32)
    held = (ctx.long() + b - 1) // b
    after = (ctx.long() + new.clamp(min=0) + b - 1) // b
    used, taken = int(held.sum()), int((after - held).sum())
    total = used + taken + taken // 8 + 8
    order = torch.randperm(total, generator=g).int()
    width = int(after.max()) + 3
    tables = torch.full((len(roles), width), -1, dtype=torch.int32)
    tables[torch.arange(width) < held[:, None]] = order[:used]
    head = int(torch.randint(total, (1,), generator=g))  # the ring starts anywhere and wraps
    ring = torch.full((total,), -1, dtype=torch.int32)
    ring[(head + torch.arange(total - used)) % total] = order[used:]
    tokens = int(new.clamp(min=0).sum()) + case["padding"]
    return {"new": new.cuda(), "ctx": ctx.cuda(), "ring": ring.cuda(), "tables": tables.cuda(),
            "free": torch.tensor([head, total - used], dtype=torch.int32).cuda(), "tokens": tokens, "total": total}


def prepare(case, seed):
    st = dict(case)
    if case["op"] == "plan":
        st |= _prepare_plan(case, seed)
        return st
    if case["op"] == "prompt":
        lens = _lengths(case)
        start = torch.tensor([0] + lens).cumsum(0)
        st["q"], st["k"], st["v"] = _qkv(case, sum(lens), seed)
        st |= {"start": start.int().cuda(), "longest": max(lens), "scale": case["dim"] ** -0.5}
        # with the inputs, the plain form has each token's place in a padded batch
        seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens))
        st |= {"seq": seq.cuda(), "pos": (torch.arange(sum(lens)) - start[seq]).cuda()}
        return st
    n, total, b = case["tokens"], case["tokens"] + case["padding"], case["block"]
    g = _generator(seed + 1)
    st["q"], st["k"], st["v"] = _qkv(case, total, seed)
    st["cos_sin"] = _cos_sin(case["far"], case["rot"])
    st["positions"] = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    st["positions"][:n] = torch.randint(case["far"], (n,), generator=g, device="cuda").int()
    blocks = n // b + n // (8 * b) + 2
    st["slots"] = torch.full((total,), -1, dtype=torch.int64, device="cuda")
    st["slots"][:n] = torch.randperm(blocks * b, generator=g, device="cuda")[:n]
    pool = (blocks, case["kv_heads"], b, case["dim"])
    st["k_cache"] = torch.zeros(pool, dtype=st["q"].dtype, device="cuda")
    st["v_cache"] = torch.zeros(pool, dtype=st["q"].dtype, device="cuda")
    st["q_out"] = torch.zeros(st["q"].shape, dtype=st["q"].dtype, device="cuda")
    st["k_out"] = torch.zeros(st["k"].shape, dtype=st["q"].dtype, device="cuda") if case["keep_key"] else None
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_prompt(st):
    q, k, v, seq, pos = st["q"], st["k"], st["v"], st["seq"], st["pos"]
    h, hkv, d, s, n = st["heads"], st["kv_heads"], st["dim"], st["seqs"], st["longest"]
    g = h // hkv

    def padded(x, heads):
        y = torch.zeros(s, n, heads, d, dtype=torch.float32, device="cuda")
        y[seq, pos] = x.float()
        return y.transpose(1, 2)

    qp = padded(q, h).reshape(s, hkv, g, n, d)
    kt, vp = padded(k, hkv).transpose(2, 3), padded(v, hkv)
    out = torch.empty(s, hkv, g, n, d, dtype=torch.float32, device="cuda")
    at = torch.arange(n, device="cuda")
    # the scores of all queries of a long prompt do not fit the card at once: as many rows at a time as do
    rows = max(1, min(n, (1 << 31) // (s * h * n)))
    for r in range(0, n, rows):
        part = qp[:, :, :, r:r + rows]
        m = part.shape[3]
        z = (part.reshape(s, hkv, g * m, d) @ kt).view(s, hkv, g, m, n) * st["scale"]
        z.masked_fill_(at > at[r:r + rows, None], float("-inf"))
        z -= z.amax(-1, keepdim=True)
        z.exp_()
        total = z.sum(-1, keepdim=True)
        o = (z.view(s, hkv, g * m, n) @ vp).view(s, hkv, g, m, d)
        out[:, :, :, r:r + rows] = o / total
    return out.reshape(s, h, n, d).transpose(1, 2)[seq, pos].to(q.dtype)


def _rotate(x, cos, sin, rot, interleaved):
    """x [T][heads][d] in its computing type, cos and sin [T][rot / 2]."""
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_rotary(st):
    n, b, rot, dt = st["tokens"], st["block"], st["rot"], st["q"].dtype
    at = st["positions"][:n].long()
    cos, sin = st["cos_sin"][at].split(rot // 2, dim=1)
    st["q_out"][:n] = _rotate(st["q"][:n].float(), cos, sin, rot, st["interleaved"]).to(dt)
    key = _rotate(st["k"][:n].float(), cos, sin, rot, st["interleaved"]).to(dt)
    if st["k_out"] is not None:
        st["k_out"][:n] = key
    slots = st["slots"][:n]
    block = torch.div(slots, b, rounding_mode="floor")
    st["k_cache"][block, :, slots - block * b] = key
    st["v_cache"][block, :, slots - block * b] = st["v"][:n]


def _plain_plan(st):
    b, ring, tables, tokens = st["block"], st["ring"], st["tables"], st["tokens"]
    ctx, new, cap = st["ctx"].long(), st["new"].long(), st["ring"].numel()
    head, count = st["free"].long()
    held = (ctx + b - 1) // b
    grown = new.clamp(min=0)
    after = (ctx + grown + b - 1) // b
    column = torch.arange(tables.shape[1], device="cuda")
    # blocks of finished sequences go behind the ring's last entry, in order
    given = torch.where(new < 0, held, 0)
    there = column < given[:, None]
    back = given.cumsum(0)[:, None] - given[:, None] + column
    ring[((head + count + back) % cap)[there]] = tables[there]
    # growing sequences take theirs from its first ones
    taken = torch.where(new < 0, 0, after - held)
    there = (column >= held[:, None]) & (column < (held + taken)[:, None])
    nth = (taken.cumsum(0) - taken - held)[:, None] + column
    tables[there] = ring[(head + nth) % cap][there]
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), grown.cumsum(0)])
    t = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(start, t, right=True) - 1
    real = t < start[-1]
    seq = torch.where(real, seq, 0)
    pos = torch.where(real, ctx[seq] + t - start[seq], 0)
    slot = tables[seq, pos // b].long() * b + pos % b
    free = torch.stack([(head + taken.sum()) % cap, count + given.sum() - taken.sum()])
    return {"context_lens": torch.where(new < 0, 0, ctx + grown).int(), "free_state": free.int(),
            "query_start_loc": start.int(), "slot_mapping": torch.where(real, slot, -1),
            "positions": torch.where(real, pos, -1).int(), "block_tables": tables, "free_ring": ring}


def run(st):
    if own:
        from paged_kv_cache_132_gb300 import api
    if st["op"] == "prompt":
        if own:
            return api.prompt_attention(st["q"], st["k"], st["v"], st["start"], st["scale"])
        return _plain_prompt(st)
    if st["op"] == "rotary":
        if own:
            api.rotary_and_cache(st["q"], st["k"], st["v"], st["positions"], st["cos_sin"], st["slots"],
                                 st["k_cache"], st["v_cache"], interleaved=st["interleaved"],
                                 query_out=st["q_out"], key_out=st["k_out"])
        else:
            _plain_rotary(st)
        return {k: st[k] for k in ("q_out", "k_out", "k_cache", "v_cache")}
    if own:
        p = api.plan_step(st["new"], st["ctx"], st["ring"], st["free"], st["tables"], st["block"], st["tokens"],
                          st["total"])
        return {**p._asdict(), "block_tables": st["tables"], "free_ring": st["ring"]}
    return _plain_plan(st)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_prompt(case, seed):
    st = prepare(case, seed)
    g = case["heads"] // case["kv_heads"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    begin = 0
    for n in _lengths(case):
        for h in range(case["heads"]):
            k = st["k"][begin:begin + n, h // g].double()
            v = st["v"][begin:begin + n, h // g].double()
            for r in range(0, n, 4096):
                e = min(n, r + 4096)
                z = torch.mm(st["q"][begin + r:begin + e, h].double(), k[:e].T).mul_(st["scale"])
                z.masked_fill_(torch.ones(e - r, e, dtype=torch.bool, device="cuda").triu_(r + 1), -math.inf)
                w = torch.softmax(z, dim=1)
                out[begin + r:begin + e, h] = w @ v[:e]
        begin += n
    return out


def _exact_rotary(case, seed):
    st = prepare(case, seed)
    n, half, b = case["tokens"], case["rot"] // 2, case["block"]
    table = st["cos_sin"][st["positions"][:n].long()].double()
    turn = torch.complex(table[:, :half], table[:, half:])[:, None]  # a pair is a complex number

    def rotated(x):
        y = x[:n].double()
        if case["interleaved"]:
            first, second = torch.arange(0, 2 * half, 2), torch.arange(1, 2 * half, 2)
        else:
            first, second = torch.arange(half), torch.arange(half, 2 * half)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def rows(x, like):
        y = torch.zeros(like.shape, dtype=torch.float64, device="cuda")
        y[:n] = x
        return y

    def pool(x):
        y = torch.zeros(st["k_cache"].shape, dtype=torch.float64, device="cuda")
        flat = y.permute(0, 2, 1, 3)
        flat[st["slots"][:n] // b, st["slots"][:n] % b] = x
        return y

    key = rotated(st["k"])
    return {"q_out": rows(rotated(st["q"]), st["q"]), "k_out": rows(key, st["k"]) if case["keep_key"] else None,
            "k_cache": pool(key), "v_cache": pool(st["v"][:n].double())}


def _exact_plan(case, seed):
    st = prepare(case, seed)
    b, cap = case["block"], st["total"]
    new, ctx, tables, ring = (st[x].cpu().tolist() for x in ("new", "ctx", "tables", "ring"))
    head, count = st["free"].tolist()
    free = deque(ring[(head + i) % cap] for i in range(count))
    tail = (head + count) % cap
    for s, n in enumerate(new):
        if n < 0:
            for block in tables[s][:_ceil(ctx[s], b)]:
                free.append(block)
                ring[tail] = block
                tail = (tail + 1) % cap
    start, slots, positions, lens = [0], [], [], []
    for s, n in enumerate(new):
        for p in range(ctx[s], ctx[s] + max(0, n)):
            if p % b == 0:
                tables[s][p // b] = free.popleft()
                head = (head + 1) % cap
            slots.append(tables[s][p // b] * b + p % b)
            positions.append(p)
        start.append(len(slots))
        lens.append(0 if n < 0 else ctx[s] + n)
    pad = [-1] * (st["tokens"] - len(slots))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"context_lens": i32(lens), "free_state": i32([head, len(free)]), "query_start_loc": i32(start),
            "slot_mapping": torch.tensor(slots + pad, dtype=torch.int64), "positions": i32(positions + pad),
            "block_tables": i32(tables), "free_ring": i32(ring)}


def exact(case, seed):
    return {"prompt": _exact_prompt, "rotary": _exact_rotary, "plan": _exact_plan}[case["op"]](case, seed)
