"""The plan of a step on the GPU against the host block manager and a plain
restatement, exactly; and the operators of a step run together."""
from collections import deque

import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from paged_kv_cache_132_gb300.block_manager import BlockManager

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def plain(new, ctx, tables, ring, head, count, b, max_tokens):
    """One sequence after the other, on lists (updated in place)."""
    size = len(ring)
    free, tail = deque(ring[(head + i) % size] for i in range(count)), (head + count) % size
    for s, n in enumerate(new):
        if n < 0:
            for x in tables[s][:-(-ctx[s] // b)]:
                free.append(x)
                ring[tail] = x
                tail = (tail + 1) % size
    start, slots, pos, lens = [0], [], [], []
    for s, n in enumerate(new):
        for p in range(ctx[s], ctx[s] + max(n, 0)):
            if p % b == 0:
                tables[s][p // b] = free.popleft()
                head = (head + 1) % size
            slots.append(tables[s][p // b] * b + p % b)
            pos.append(p)
        start.append(len(slots))
        lens.append(0 if n < 0 else ctx[s] + n)
    pad = max_tokens - len(slots)
    return lens, [head, len(free)], start, slots + [-1] * pad, pos + [-1] * pad


def build(new, ctx, b, seed, spare=5):
    """Tables, ring and free state for given lengths, in a shuffled order."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-c // b) for c in ctx]
    after = [-(-(c + max(n, 0)) // b) for c, n in zip(ctx, new)]
    total = sum(after) + spare
    order = torch.randperm(total, generator=g).tolist()
    width = max(after + [1]) + 1
    tables, at = [], 0
    for h in held:
        tables.append(order[at:at + h] + [-7] * (width - h))
        at += h
    head = int(torch.randint(total, (1,), generator=g))
    ring = [-7] * total
    for i, x in enumerate(order[at:]):
        ring[(head + i) % total] = x
    return tables, ring, head, total - at, total


def check(new, ctx, b, seed=1, pad=0, in_place=False):
    tables, ring, head, count, total = build(new, ctx, b, seed)
    tokens = sum(max(n, 0) for n in new) + pad
    d = dict(new=i32(new), ctx=i32(ctx), ring=i32(ring), free=i32([head, count]), tables=i32(tables))
    out = None
    if in_place:
        out = api.StepPlan(d["ctx"], d["free"], i32([0] * (len(new) + 1)),
                           torch.zeros(tokens, dtype=torch.int64, device="cuda"), i32([0] * tokens))
    got = api.plan_step(d["new"], d["ctx"], d["ring"], d["free"], d["tables"], b, tokens, total, out=out)
    assert api.get_device_error() == (0, 0)
    want = plain(new, ctx, tables, ring, head, count, b, tokens)
    for name, x, y in zip(got._fields, got, want):
        assert x.tolist() == y, name
    assert d["tables"].tolist() == tables and d["ring"].tolist() == ring
    if not in_place:
        assert d["ctx"].tolist() == list(ctx) and d["free"].tolist() == [head, count]


def lengths(n, seed, hi_new, hi_ctx):
    g = torch.Generator().manual_seed(seed)
    kind = torch.randint(5, (n,), generator=g)
    new = torch.randint(1, hi_new + 1, (n,), generator=g)
    ctx = torch.randint(0, hi_ctx + 1, (n,), generator=g)
    new = torch.where(kind == 0, -1, torch.where(kind == 1, 0, torch.where(kind == 2, 1, new)))
    return new.tolist(), ctx.tolist()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,hi_new,hi_ctx,b", [(1, 1, 0, 16), (1, 40, 100, 8), (3, 70, 33, 16), (33, 1, 64, 16),
                                               (256, 9, 300, 32), (1023, 3, 40, 1), (1025, 5, 40, 7),
                                               (2500, 2, 20, 16)])
def test_random_steps(n, hi_new, hi_ctx, b, in_place):
    for seed in range(3):
        new, ctx = lengths(n, 100 * n + seed, hi_new, hi_ctx)
        check(new, ctx, b, seed, pad=(0, 3, 1500)[seed], in_place=in_place)


@pytest.mark.parametrize("tokens", [1, 4095, 4096, 4097, 9000, 40001])
def test_one_prompt(tokens):
    check([tokens], [0], 16)
    check([0, tokens, -1, 1], [5, 13, 64, 16], 16, pad=77)


def test_edges():
    check([1], [16], 16)       # a new block for the next token
    check([1], [15], 16)       # the last free slot of a block
    check([-1, -1], [0, 1], 16)
    check([0, 0, 0], [0, 16, 17], 16, pad=4)
    check([16, 17, 15, 1], [0, 0, 0, 0], 16)
    check([-1] * 700 + [3] * 700, [33] * 1400, 16, pad=9000)  # blocks given and taken in one step


def test_no_sequences():
    e = i32([])
    got = api.plan_step(e, e, i32([4, 5]), i32([1, 1]), torch.empty(0, 3, dtype=torch.int32, device="cuda"), 16, 6, 8)
    assert api.get_device_error() == (0, 0)
    assert got.query_start_loc.tolist() == [0] and got.free_state.tolist() == [1, 1]
    assert got.slot_mapping.tolist() == [-1] * 6 and got.positions.tolist() == [-1] * 6


def test_largest_batch():
    new, ctx = lengths(16384, 7, 2, 30)
    check(new, ctx, 16, 2, pad=100)


@pytest.mark.parametrize("what", ["blocks", "tokens", "ring", "head", "count"])
def test_a_step_that_does_not_fit_is_refused_whole(what):
    new, ctx, b = [40, -1, 1, 0], [0, 50, 32, 20], 16
    tables, ring, head, count, total = build(new, ctx, b, 3, spare=0)
    tokens = 41 if what != "tokens" else 40
    free = [head, count]
    if what == "blocks":  # 4 blocks are taken, 4 given back: none is free at first
        new = [200, -1, 1, 0]
        tokens = 201
        tables = [t + [-7] * 12 for t in tables]
    if what == "ring":
        ring = ring[:count + 3]
        free = [0, count]
    if what == "head":
        free = [len(ring), count]
    if what == "count":
        free = [head, -1]
    d = dict(new=i32(new), ctx=i32(ctx), ring=i32(ring), free=i32(free), tables=i32(tables))
    got = api.plan_step(d["new"], d["ctx"], d["ring"], d["free"], d["tables"], b, tokens, total)
    assert api.get_device_error() == (-5, native.DEVERR_STEP)
    assert got.context_lens.tolist() == ctx and got.free_state.tolist() == free
    assert got.query_start_loc.tolist() == [0] * 5
    assert got.slot_mapping.tolist() == [-1] * tokens and got.positions.tolist() == [-1] * tokens
    assert d["tables"].tolist() == tables and d["ring"].tolist() == ring


def test_bad_lengths_leave_their_sequence_alone():
    b = 16
    new, ctx = [3, 5, -2, 1, 2 ** 31 - 1, 4], [10, -1, 20, 80, 30, 0]
    tables = [[i * 10 + j for j in range(5)] for i in range(6)]
    ring = list(range(100, 110))
    d = dict(new=i32(new), ctx=i32(ctx), ring=i32(ring), free=i32([0, 10]), tables=i32(tables))
    got = api.plan_step(d["new"], d["ctx"], d["ring"], d["free"], d["tables"], b, 7, 200)
    assert api.get_device_error() == (-5, native.DEVERR_CONTEXT_LEN)
    assert got.context_lens.tolist() == [13, -1, 20, 80, 30, 4]
    assert got.query_start_loc.tolist() == [0, 3, 3, 3, 3, 3, 7]
    assert got.slot_mapping.tolist() == [10, 11, 12, 1600, 1601, 1602, 1603]
    assert got.free_state.tolist() == [1, 9]


def test_bad_block_ids_are_reported():
    d = dict(new=i32([1, 1, 1]), ctx=i32([16, 3, 5]), ring=i32([50, 60]), free=i32([0, 1]),
             tables=i32([[1, -7], [2, -7], [-3, -7]]))
    got = api.plan_step(d["new"], d["ctx"], d["ring"], d["free"], d["tables"], 16, 3, 50)
    assert api.get_device_error() == (-5, native.DEVERR_BLOCK_ID)
    assert got.slot_mapping.tolist() == [-1, 35, -1]


def test_many_steps_follow_the_host_manager():
    """A captured step that advances in place, against BlockManager, over steps
    that add, grow and finish sequences."""
    b, seats, nb, width, tokens = 16, 24, 400, 20, 600
    g = torch.Generator().manual_seed(11)
    bm = BlockManager(nb, b, free_order=torch.randperm(nb, generator=g).tolist())
    ring, state = i32(list(bm.free)), i32([0, nb])
    new, ctx, tables = i32([0] * seats), i32([0] * seats), i32([[-1] * width] * seats)
    out = api.StepPlan(ctx, state, i32([0] * (seats + 1)), torch.zeros(tokens, dtype=torch.int64, device="cuda"),
                       i32([0] * tokens))
    graph = torch.cuda.CUDAGraph()
    api.plan_step(new, ctx, ring, state, tables, b, tokens, nb, out=out)  # all idle: changes nothing
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        api.plan_step(new, ctx, ring, state, tables, b, tokens, nb, out=out)
    live = {}
    for step in range(40):
        want, done = [0] * seats, []
        for s in range(seats):
            r = float(torch.rand(1, generator=g))
            if s in live and (r < 0.1 or live[s] > 250):
                want[s] = -1
                done.append(s)
            elif s in live:
                want[s] = 1 if r < 0.9 else 0
            elif r < 0.3:
                want[s] = int(torch.randint(1, 60, (1,), generator=g))
        new.copy_(i32(want))
        graph.replay()
        for s in done:
            bm.free_sequence(s)
            del live[s]
        slots = []
        for s, n in enumerate(want):
            if n <= 0:
                continue
            if s not in live:
                bm.add_sequence(s, 0)
                live[s] = 0
            for _ in range(n):
                slots.append(bm.append_token(s))
            live[s] += n
        assert api.get_device_error() == (0, 0)
        assert out.slot_mapping.tolist() == slots + [-1] * (tokens - len(slots))
        assert ctx.tolist() == [live.get(s, 0) for s in range(seats)]
        assert int(state[1]) == bm.num_free()
        for s in live:
            assert tables[s, :len(bm.table(s))].tolist() == bm.table(s)


def test_refusals():
    d = dict(new_lens=i32([1]), context_lens=i32([0]), free_ring=i32([0, 1]), free_state=i32([0, 2]),
             block_tables=i32([[0, 0]]), block_size=16, max_tokens=4, num_blocks=2)
    for bad in (dict(new_lens=i32([1]).long()), dict(context_lens=i32([0, 0])), dict(free_state=i32([0])),
                dict(free_ring=i32([[0, 1]])), dict(block_tables=i32([[0], [0]])), dict(max_tokens=-1),
                dict(new_lens=i32([1]).cpu()), dict(out=api.StepPlan(*[i32([0])] * 5))):
        with pytest.raises(ValueError):
            api.plan_step(**{**d, **bad})
    for bad in (dict(block_size=0), dict(num_blocks=0)):
        with pytest.raises(native.PaError):
            api.plan_step(**{**d, **bad})


def attention(q, k, v, scale):
    """float64 causal attention of the last len(q) tokens of one sequence."""
    n, m, g = q.shape[0], k.shape[0], q.shape[1] // k.shape[1]
    z = q.double().transpose(0, 1) @ k.double().transpose(0, 1).repeat_interleave(g, 0).transpose(1, 2) * scale
    z = z.masked_fill(torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1), float("-inf"))
    return (torch.softmax(z, -1) @ v.double().transpose(0, 1).repeat_interleave(g, 0)).transpose(0, 1)


@pytest.mark.parametrize("dtype,h,hkv,d,b", [(torch.bfloat16, 8, 2, 128, 16), (torch.float16, 4, 4, 64, 8)])
def test_a_serving_loop(dtype, h, hkv, d, b):
    """Plan, rotary embedding with cache write, attention over the prompts, then
    decode steps over the pools that these filled, all from device state; against
    attention in 64 bits over the rotated rows that a plain list keeps.  Bounds:
    weights and outputs rounded to the type, each half a step, of values that the
    largest |v| bounds; the decode's 2e-3."""
    seats, nb, width, scale, far = 5, 120, 40, d ** -0.5, 512
    g = torch.Generator(device="cuda").manual_seed(5)
    lens = [70, 1, 0, 133, 16]
    kc, vc = (torch.full((nb, hkv, b, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    a = torch.arange(far, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    cs = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    ring, free = i32(list(range(nb))[::-1]), i32([0, nb])
    ctx, tables = i32([0] * seats), i32([[-1] * width] * seats)
    keys, values = [[] for _ in lens], [[] for _ in lens]
    u = torch.finfo(dtype).eps / 2
    for step in range(6):
        new = lens if step == 0 else [1, 1, 20 if step == 3 else (1 if step > 3 else 0), 1, -1 if step == 2 else (1 if step < 2 else 0)]
        total = sum(max(n, 0) for n in new)
        room = total + 3  # rows of a padded batch
        plan = api.plan_step(i32(new), ctx, ring, free, tables, b, room, nb)
        ctx, free = plan.context_lens, plan.free_state
        rows = torch.randn(room, (h + 2 * hkv) * d, generator=g, device="cuda").to(dtype)
        q, k, v = (x.unflatten(1, (-1, d)) for x in rows.split([h * d, hkv * d, hkv * d], 1))
        ko = torch.empty(room, hkv, d, dtype=dtype, device="cuda")
        q = api.rotary_and_cache(q, k, v, plan.positions, cs, plan.slot_mapping, kc, vc, key_out=ko)
        start = plan.query_start_loc.tolist()
        for s, n in enumerate(new):
            if n < 0:
                keys[s], values[s] = [], []
            keys[s].append(ko[start[s]:start[s + 1]].clone())
            values[s].append(v[start[s]:start[s + 1]].clone())
        if step == 0 or step == 3:
            if step == 0:
                out = api.prompt_attention(q, ko, v, plan.query_start_loc, scale)
            else:  # prompts next to running sequences: over the pools
                out = api.prefill(q, plan.query_start_loc, kc, vc, tables, ctx, scale, 20, out_dtype=dtype)
            for s, n in enumerate(new):
                if n > 0:
                    ref = attention(q[start[s]:start[s + 1]], torch.cat(keys[s]), torch.cat(values[s]), scale)
                    bound = 2 * u * float(torch.cat(values[s]).abs().max()) + 2e-3
                    assert float((out[start[s]:start[s + 1]].double() - ref).abs().max()) <= bound
        else:
            seqs = [s for s, n in enumerate(new) if n == 1]
            at = torch.tensor(seqs, device="cuda")
            out = api.decode(q[plan.query_start_loc[at].long()], kc, vc, tables[at], ctx[at], scale)
            for i, s in enumerate(seqs):
                ref = attention(q[start[s]:start[s] + 1], torch.cat(keys[s]), torch.cat(values[s]), scale)
                assert float((out[i].double() - ref[0]).abs().max()) <= 2e-3
        assert api.get_device_error() == (0, 0)
