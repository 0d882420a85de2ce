"""Calls of drafted trees on several streams at once, behind other calls without a wait of
the host, and steps without any node or sequence."""
import random

import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from trees import Cache, i32, parents_of, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


class Job:
    """The three calls behind the model's layers, their inputs and a chain of calls over them."""
    def __init__(self, lens, before, h, hkv, d, dtype, vocab, seed):
        r, g = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
        ctx = [a + n for a, n in zip(before, lens)]
        c = Cache(ctx, hkv, d, 16, dtype, seed)
        self.k, self.v, self.tables, self.ctx = c.k, c.v, c.tables, i32(ctx)
        t = sum(lens)
        self.start, self.bound, self.scale = starts(lens), max(lens), d ** -0.5
        self.parents = i32([p for n in lens for p in parents_of(n, 3, r)])
        self.tokens = torch.randint(vocab, (t,), generator=g, device="cuda", dtype=torch.int32)
        self.q = rand(t, h, d).to(dtype)
        self.p = torch.softmax(rand(t, vocab), 1)
        self.d = torch.softmax(self.p.log() + rand(t, vocab) * 0.5, 1)
        self.u, self.w = torch.rand(t, generator=g, device="cuda"), torch.rand(len(lens), generator=g, device="cuda")

    def run(self, stream):
        tree = api.plan_tree(self.parents, self.start, self.ctx, self.bound, stream=stream)
        out = api.tree_attention(self.q, self.start, tree.tree_mask, self.k, self.v, self.tables, self.ctx, self.scale,
                                 stream=stream)
        return [tree.positions, out, *api.verify_tree(self.tokens, self.parents, self.start, self.p, self.d, self.u, self.w,
                                                      stream=stream)]


def test_streams_at_once():
    jobs = [Job([16] * 40, [900 + 13 * s for s in range(40)], 32, 8, 128, torch.bfloat16, 5003, 1),
            Job([3, 64, 1, 40], [4000, 77, 0, 2500], 8, 2, 128, torch.float16, 30011, 2),
            Job([31] * 3, [9000, 5, 700], 16, 4, 64, torch.bfloat16, 1009, 3)]
    torch.cuda.synchronize()
    want = [j.run(None) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for _ in range(20):
        for n, (j, s) in enumerate(zip(jobs, streams)):
            got[n].append(j.run(s))
    torch.cuda.synchronize()
    assert api.get_device_error() == (0, 0)
    for w, runs in zip(want, got):
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, run))


def test_steps_without_nodes_or_sequences():
    e32, f32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")  # noqa: E731
    k = torch.ones(4, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    for seqs in (0, 3):
        start, ctx, tables = i32([0] * (seqs + 1)), i32([8] * seqs), i32([[1]] * seqs).reshape(seqs, 1)
        tree = api.plan_tree(e32(0), start, ctx, 8)
        assert tree.positions.shape == (0,) and tree.tree_mask.shape == (0, 1)
        q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
        assert api.tree_attention(q, start, tree.tree_mask, k, k, tables, ctx, 0.125).shape == (0, 4, 64)
        verdict = api.verify_tree(e32(0), e32(0), start, torch.empty(0, 10, device="cuda"), None, f32,
                                  torch.zeros(seqs, device="cuda"))
        assert verdict.accepted_lens.tolist() == [0] * seqs and verdict.next_tokens.tolist() == [-1] * seqs
        ring, free = i32([0, 2, 3, -1]), i32([0, 3])
        left = api.commit_tree([k], [k.clone()], start, verdict.path, verdict.accepted_lens, ctx, tables, free_ring=ring,
                               free_state=free)
        assert left.context_lens.tolist() == [8] * seqs and left.free_state.tolist() == [0, 3]
        assert ring.tolist() == [0, 2, 3, -1] and (k == 1).all()
    # padding alone: rows of no sequence
    tree = api.plan_tree(i32([5] * 70), i32([0]), e32(0), 65)
    assert (tree.positions == -1).all() and (tree.tree_mask == 0).all() and tree.tree_mask.shape == (70, 2)
    assert api.get_device_error() == (0, 0)
