"""The plan of drafted trees and the commit of accepted paths against lists, bit for
bit, and a whole step: plan, rotary embedding and cache write, attention, verification,
commit, and the next step on what they leave."""
import random

import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from trees import Cache, ancestors, attention, i32, parents_of, random_trees, starts, words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


# ---------------------------------------------------------------------------
# plan_tree
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("lens,width,bound", [
    ([1], 1, 1), ([5, 0, 64, 1], 3, 64), ([64] * 5, 1, 64), ([65, 3], 2, 65), ([128, 200, 7], 5, 256),
    ([1024], 1, 1024), ([1000, 30], 400, 1024), ([16] * 700, 3, 16), ([0, 0], 1, 4)])
@pytest.mark.parametrize("first,extra", [(0, 0), (3, 40)])
def test_plan(lens, width, bound, first, extra):
    trees = random_trees(lens, width, len(lens))
    ctx = [n + 11 * s for s, n in enumerate(lens)]
    total, count = first + sum(lens) + extra, -(-bound // 64)
    parents = i32([5] * first + [p for t in trees for p in t] + [99] * extra)
    got = api.plan_tree(parents, starts(lens, first), i32(ctx), bound)
    assert api.get_device_error() == (0, 0)
    pos = [-1] * first + [c - n + len(a) - 1 for t, c, n in zip(trees, ctx, lens) for a in ancestors(t)] + [-1] * extra
    assert got.positions.tolist() == pos
    mask = torch.zeros(total, count, dtype=torch.int64)
    mask[first:first + sum(lens)] = words([a for t in trees for a in ancestors(t)], count)
    assert torch.equal(got.tree_mask.cpu(), mask)


def test_plan_of_bad_parents_and_lengths():
    parents = i32([-1, 0, 1, 2] * 4)
    parents[2], parents[7], parents[9] = 2, 5, -3
    got = api.plan_tree(parents, starts([4] * 4), i32([4, 9, 20, 3]), 64)
    assert api.get_device_error() == (-5, native.DEVERR_TREE | native.DEVERR_CONTEXT_LEN)
    assert got.positions.tolist() == [0, 1, 0, 1, 5, 6, 7, 5, 16, 16, 17, 18, -1, -1, -1, -1]
    assert got.tree_mask[:, 0].tolist() == [1, 3, 4, 12, 1, 3, 7, 8, 1, 2, 6, 14, 0, 0, 0, 0]
    got = api.plan_tree(i32([-1] + list(range(69))), starts([70]), i32([70]), 64)  # more nodes than bits
    assert api.get_device_error() == (-5, native.DEVERR_CONTEXT_LEN)
    assert (got.positions == -1).all() and (got.tree_mask == 0).all()


def test_plan_captured():
    parents, start, ctx = i32([-1, 0, 0, 1, -1, 0, -1, -1]), starts([4, 2]), i32([10, 2])
    out = api.plan_tree(parents, start, ctx, 8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.plan_tree(parents, start, ctx, 8, out=out)
    parents.copy_(i32([-1, 0, -1, 0, 1, 2, 3, 4]))
    start.copy_(i32([0, 2, 8]))
    ctx.copy_(i32([2, 106]))
    graph.replay()
    torch.cuda.synchronize()
    assert out.positions.tolist() == [0, 1, 100, 101, 102, 103, 104, 105]
    assert out.tree_mask[:, 0].tolist() == [1, 3, 1, 3, 7, 15, 31, 63]


def test_plan_refusals():
    parents, start, ctx = i32([-1, 0]), starts([2]), i32([2])
    for args in ((parents.long(), start, ctx, 2), (parents, start.long(), ctx, 2), (parents, start, ctx.repeat(2), 2),
                 (parents, start, ctx, 0), (parents.cpu(), start, ctx, 2)):
        with pytest.raises(ValueError):
            api.plan_tree(*args)
    with pytest.raises(native.PaError):
        api.plan_tree(parents, start, ctx, 1025)


# ---------------------------------------------------------------------------
# commit_tree
# ---------------------------------------------------------------------------
class Commit:
    def __init__(self, before, nodes, keep, layers, hkv, d, block, dtype, seed=1, ring=True, paths=None):
        r = random.Random(seed)
        self.ctx = [b + n for b, n in zip(before, nodes)]
        self.before, self.nodes, self.keep, self.block = before, nodes, keep, block
        c = Cache(self.ctx, hkv, d, block, dtype, seed, spare=4)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.tables, self.num_blocks = c.tables, c.num_blocks
        shape = (c.num_blocks, hkv, block, d)
        self.k = [torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(layers)]
        self.v = [torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(layers)]
        self.paths = paths or [sorted(r.sample(range(n), k)) for n, k in zip(nodes, keep)]
        self.start, self.lens = starts(nodes), i32(keep)
        self.path = i32([x for p, n in zip(self.paths, nodes) for x in p + [-1] * (n - len(p))])
        self.ring = self.free = None
        if ring:
            size, head = c.num_blocks, c.num_blocks - 2
            ids = torch.full((size,), -1, dtype=torch.int32)
            for j, b in enumerate(c.left):
                ids[(head + j) % size] = b
            self.ring, self.free = ids.cuda(), i32([head, len(c.left)])

    def expected(self, bad=()):
        k, v = [x.clone() for x in self.k], [x.clone() for x in self.v]
        ctx, back = list(self.ctx), []
        tables = self.tables.tolist()
        for s, (b, n, path) in enumerate(zip(self.before, self.nodes, self.paths)):
            if s in bad:
                continue

            def at(i):
                return tables[s][(b + i) // self.block], (b + i) % self.block

            for x in k + v:
                rows = [x[at(i)[0], :, at(i)[1]].clone() for i in path]
                for i, row in enumerate(rows):
                    x[at(i)[0], :, at(i)[1]] = row
            ctx[s] = b + len(path)
            back += tables[s][-(-ctx[s] // self.block):-(-(b + n) // self.block)]
        ring = free = None
        if self.ring is not None:
            ring, (head, count) = self.ring.tolist(), self.free.tolist()
            for j, x in enumerate(back):
                ring[(head + count + j) % len(ring)] = x
            free = [head, count + len(back)]
        return k, v, ctx, ring, free

    def call(self, **kw):
        return api.commit_tree(self.k, self.v, self.start, self.path, self.lens, i32(self.ctx), self.tables,
                               free_ring=self.ring, free_state=self.free, **kw)

    def check(self, want, got):
        k, v, ctx, ring, free = want
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(k + v, self.k + self.v))
        assert got.context_lens.tolist() == ctx
        if ring is not None:
            assert self.ring.tolist() == ring and got.free_state.tolist() == free
        else:
            assert got.free_state is None


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64), (torch.float32, 128), (torch.float32, 36),
                                     (torch.float16, 24)])
@pytest.mark.parametrize("block", [8, 16, 5])
@pytest.mark.parametrize("ring", [True, False])
def test_commit(dtype, d, block, ring):
    before, nodes = [0, 7, 30, 64, 1, 12], [1, 9, 40, 0, 16, 5]
    keep = [1, 3, 20, 0, 16, 0]
    c = Commit(before, nodes, keep, 3, 3, d, block, dtype, ring=ring)
    want = c.expected()
    got = c.call()
    assert api.get_device_error() == (0, 0)
    c.check(want, got)


@pytest.mark.parametrize("seqs,layers", [(1, 1), (1, 256), (200, 5), (3000, 1), (16384, 1)])
def test_commit_of_batches(seqs, layers):
    r = random.Random(seqs)
    nodes = [r.randrange(0, 12) for _ in range(seqs)]
    keep = [r.randint(0, n) for n in nodes]
    c = Commit([r.randrange(0, 20) for _ in nodes], nodes, keep, layers, 1, 64, 8, torch.bfloat16)
    want = c.expected()
    got = c.call()
    assert api.get_device_error() == (0, 0)
    c.check(want, got)


def test_commit_of_long_paths():
    """More than the 32 entries that are looked up at once; every other row moves onto a
    place that an earlier one left."""
    n = 1000
    paths = [list(range(1, n, 2)), list(range(n - 300, n)), list(range(n))]
    c = Commit([3, 100, 0], [n] * 3, [len(p) for p in paths], 2, 2, 64, 16, torch.bfloat16, paths=paths)
    want = c.expected()
    got = c.call()
    assert api.get_device_error() == (0, 0)
    c.check(want, got)


@pytest.mark.parametrize("seqs", [5, 3000])
def test_commit_in_place_and_captured(seqs):
    """Lengths and free blocks overwritten, as a captured step does."""
    r = random.Random(seqs)
    nodes = [r.randrange(1, 12) for _ in range(seqs)]
    c = Commit([r.randrange(0, 20) for _ in nodes], nodes, [r.randint(1, n) for n in nodes], 2, 2, 64, 8, torch.float16)
    want = c.expected()
    ctx = i32(c.ctx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = api.commit_tree(c.k, c.v, c.start, c.path, c.lens, ctx, c.tables, free_ring=c.ring, free_state=c.free,
                              out=api.TreeCommit(ctx, c.free))
    graph.replay()
    torch.cuda.synchronize()
    assert api.get_device_error() == (0, 0)
    c.check(want, got)


def test_bad_paths_and_lengths_leave_a_sequence_as_it_is():
    before, nodes = [10] * 7, [8] * 7
    paths = [[0, 2, 5], [0, 2, 2], [0, 8], [3, 1], [-1, 2], [0, 4], [0, 6]]
    c = Commit(before, nodes, [len(p) for p in paths], 2, 2, 64, 4, torch.bfloat16, paths=paths)
    c.lens[5] = 9
    want = c.expected(bad=(1, 2, 3, 4, 5))
    got = c.call()
    assert api.get_device_error() == (-5, native.DEVERR_TREE | native.DEVERR_CONTEXT_LEN)
    c.check(want, got)


def test_commit_with_a_full_ring_or_a_bad_block():
    c = Commit([10, 3], [30, 30], [2, 3], 1, 2, 64, 8, torch.bfloat16)
    want = c.expected()
    before = c.ring.clone()
    c.free[1] = c.ring.numel() - 1
    got = c.call()
    assert api.get_device_error() == (-5, native.DEVERR_STEP)
    assert torch.equal(c.ring, before) and got.free_state.tolist() == c.free.tolist()
    assert got.context_lens.tolist() == want[2]
    c = Commit([8, 3], [8, 30], [2, 3], 1, 2, 64, 8, torch.bfloat16, paths=[[0, 7], [0, 1, 2]], ring=False)
    c.tables[0, 1] = c.num_blocks
    old = c.k[0].clone()
    c.call()
    assert api.get_device_error() == (-5, native.DEVERR_BLOCK_ID)
    assert torch.equal(c.k[0], old)


def test_commit_refusals():
    c = Commit([10, 3], [3, 4], [2, 3], 2, 2, 64, 8, torch.bfloat16)
    ctx = i32(c.ctx)
    args = dict(k_caches=c.k, v_caches=c.v, query_start_loc=c.start, path=c.path, accepted_lens=c.lens, context_lens=ctx,
                block_tables=c.tables, free_ring=c.ring, free_state=c.free)
    for over in (dict(k_caches=c.k[:1]), dict(k_caches=[], v_caches=[]), dict(k_caches=[c.k[0], c.k[1].half()]),
                 dict(path=c.path.long()), dict(accepted_lens=c.lens[:1]), dict(context_lens=ctx.long()),
                 dict(block_tables=c.tables[:1]), dict(free_state=None), dict(free_ring=None), dict(free_state=c.free[:1]),
                 dict(query_start_loc=c.start[:2]), dict(v_caches=[x.cpu() for x in c.v]),
                 dict(out=api.TreeCommit(ctx, None))):
        with pytest.raises(ValueError):
            api.commit_tree(**{**args, **over})
    assert api.get_device_error() == (0, 0)


# ---------------------------------------------------------------------------
# a run of them together
# ---------------------------------------------------------------------------
def test_steps_of_a_draft_together():
    """Several sequences through several steps: what the pools hold at the end is the keys
    and values of the accepted tokens alone, at their positions, and no block is lost."""
    layers, h, hkv, d, b, vocab, nb, seqs, room = 2, 8, 2, 64, 8, 97, 60, 4, 40
    r = random.Random(1)
    g = torch.Generator(device="cuda").manual_seed(1)
    cos_sin = torch.cat([torch.ones(256, d // 2), torch.zeros(256, d // 2)], 1).cuda()  # keys stay as they are
    pools = [[torch.full((nb, hkv, b, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
             for _ in range(2)]
    # the key and value of a token at a position, the same whenever it is computed
    embed = torch.randn(layers, 2, vocab, hkv, d, generator=g, device="cuda").bfloat16()
    shift = torch.randn(256, 1, d, generator=g, device="cuda").bfloat16()
    tables, ring, free = i32([[-1] * 20] * seqs), i32(list(range(nb))), i32([0, nb])
    ctx, history, last = i32([0] * seqs), [[] for _ in range(seqs)], [r.randrange(vocab) for _ in range(seqs)]
    for step in range(6):
        nodes = [r.choice([1, 4, 9]) for _ in range(seqs)]
        trees = [parents_of(n, 3, r) for n in nodes]
        ids = [[last[s]] + [r.randrange(vocab) for _ in range(n - 1)] for s, n in enumerate(nodes)]
        total = sum(nodes)
        plan = api.plan_step(i32(nodes), ctx, ring, free, tables, b, room, nb)
        ctx, free, start = plan.context_lens, plan.free_state, plan.query_start_loc
        pad = room - total
        parents = i32([p for t in trees for p in t] + [-1] * pad)
        tree = api.plan_tree(parents, start, ctx, 9)
        tokens = i32([x for t in ids for x in t] + [0] * pad)
        at = tree.positions.clamp(min=0).long()
        q = torch.randn(room, h, d, generator=g, device="cuda").bfloat16()
        for l in range(layers):
            k, v = embed[l, 0, tokens.long()] + shift[at], embed[l, 1, tokens.long()] - shift[at]
            api.rotary_and_cache(q, k, v, tree.positions, cos_sin, plan.slot_mapping, pools[0][l], pools[1][l])
        outs = [api.tree_attention(q, start, tree.tree_mask, pools[0][l], pools[1][l], tables, ctx, d ** -0.5)
                for l in range(layers)]
        # each node: the accepted history, then its ancestors, at consecutive positions
        begin = 0
        for s, (t, n) in enumerate(zip(trees, nodes)):
            for i, above in enumerate(ancestors(t)):
                line = torch.tensor(history[s] + [ids[s][j] for j in above], device="cuda")
                place = torch.arange(len(line), device="cuda")
                for l in range(layers):
                    k, v = embed[l, 0, line] + shift[place], embed[l, 1, line] - shift[place]
                    ref, tol = attention(q[begin + i:begin + i + 1], k, v, len(line) - 1, torch.ones(1, 1, dtype=torch.bool),
                                         d ** -0.5)
                    assert ((outs[l][begin + i:begin + i + 1].double() - ref).abs() <= tol).all(), (step, s, i)
            begin += n
        target = torch.softmax(torch.randn(room, vocab, generator=g, device="cuda"), 1)
        draft = torch.softmax(target.log() + torch.randn(room, vocab, generator=g, device="cuda") * 0.3, 1)
        verdict = api.verify_tree(tokens, parents, start, target, draft, torch.rand(room, generator=g, device="cuda") * 0.5,
                                  torch.rand(seqs, generator=g, device="cuda"))
        done = api.commit_tree(pools[0], pools[1], start, verdict.path, verdict.accepted_lens, ctx, tables,
                               free_ring=ring, free_state=free)
        ctx, free = done.context_lens, done.free_state
        assert api.get_device_error() == (0, 0)
        begin = 0
        for s, n in enumerate(nodes):
            kept = verdict.accepted_lens[s].item()
            history[s] += [ids[s][j] for j in verdict.path[begin:begin + kept].tolist()]
            last[s] = verdict.next_tokens[s].item()
            begin += n
    assert ctx.tolist() == [len(x) for x in history]
    for s, line in enumerate(history):
        place = torch.arange(len(line), device="cuda")
        slots = tables[s].long()[place // b] * b + place % b
        line = torch.tensor(line, device="cuda")
        for l in range(layers):
            assert torch.equal(pools[0][l][slots // b, :, slots % b], embed[l, 0, line] + shift[place])
            assert torch.equal(pools[1][l][slots // b, :, slots % b], embed[l, 1, line] - shift[place])
    held = [x for s, line in enumerate(history) for x in tables[s, :-(-len(line) // b)].tolist()]
    head, count = free.tolist()
    idle = [ring[(head + j) % nb].item() for j in range(count)]
    assert sorted(held + idle) == list(range(nb))
