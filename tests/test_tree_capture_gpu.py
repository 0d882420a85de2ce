"""A whole step of drafted trees captured in a graph, on a stream of its own, and replayed
with other trees, lengths and probabilities: what the same calls make one by one."""
import random

import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from trees import i32, parents_of

pytestmark = pytest.mark.gpu

H, HKV, D, B, NB, SEQS, ROOM, VOCAB, LAYERS, NODES = 8, 2, 128, 16, 96, 5, 80, 331, 2, 16


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


def inputs(seed):
    r, g = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
    nodes = [r.choice([0, 1, 7, NODES]) for _ in range(SEQS)]
    cached = [r.randrange(0, 150) for _ in range(SEQS)]
    parents = [p for n in nodes for p in parents_of(n, 3, r)]
    blocks = [-(-c // B) for c in cached]
    ids = r.sample(range(NB), NB)
    tables = torch.full((SEQS, 16), -1, dtype=torch.int32)
    for s, n in enumerate(blocks):
        tables[s, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
    ring = torch.full((NB,), -1, dtype=torch.int32)
    ring[:len(ids)] = torch.tensor(ids, dtype=torch.int32)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    target = torch.softmax(rand(ROOM, VOCAB), 1)
    return dict(lens=i32(nodes), ctx=i32(cached), tables=tables.cuda(), ring=ring.cuda(), free=i32([0, len(ids)]),
                parents=i32(parents + [-1] * (ROOM - len(parents))),
                tokens=torch.randint(VOCAB, (ROOM,), generator=g, device="cuda", dtype=torch.int32),
                qkv=rand(ROOM, (H + 2 * HKV) * D).bfloat16(), pools=rand(2, LAYERS, NB, HKV, B, D).bfloat16(),
                target=target, draft=torch.softmax(target.log() + 0.5 * rand(ROOM, VOCAB), 1),
                accept=torch.rand(ROOM, generator=g, device="cuda"), sample=torch.rand(SEQS, generator=g, device="cuda"))


def step(x, cos_sin):
    plan = api.plan_step(x["lens"], x["ctx"], x["ring"], x["free"], x["tables"], B, ROOM, NB)
    start, ctx = plan.query_start_loc, plan.context_lens
    tree = api.plan_tree(x["parents"], start, ctx, NODES)
    q, k, v = (y.unflatten(1, (-1, D)) for y in x["qkv"].split([H * D, HKV * D, HKV * D], dim=1))
    outs = []
    for kc, vc in zip(*x["pools"]):
        rotated = api.rotary_and_cache(q, k, v, tree.positions, cos_sin, plan.slot_mapping, kc, vc)
        outs.append(api.tree_attention(rotated, start, tree.tree_mask, kc, vc, x["tables"], ctx, D ** -0.5,
                                       out=torch.zeros(ROOM, H, D, dtype=torch.bfloat16, device="cuda")))
    verdict = api.verify_tree(x["tokens"], x["parents"], start, x["target"], x["draft"], x["accept"], x["sample"],
                              out=api.TreeVerdict(*(torch.full((n,), -7, dtype=torch.int32, device="cuda")
                                                    for n in (SEQS, ROOM, SEQS))))
    left = api.commit_tree(list(x["pools"][0]), list(x["pools"][1]), start, verdict.path, verdict.accepted_lens, ctx,
                           x["tables"], free_ring=x["ring"], free_state=plan.free_state)
    return [tree.positions, tree.tree_mask, *outs, *verdict, *left, x["pools"], x["tables"], x["ring"]]


def test_captured_step():
    a = torch.arange(256, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    cos_sin = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    held = inputs(1)
    step({k: v.clone() for k, v in held.items()}, cos_sin)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        got = step(held, cos_sin)
    for seed in (1, 2, 3, 4):
        fresh = inputs(seed)
        for name, x in held.items():
            x.copy_(fresh[name])
        want = step(fresh, cos_sin)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()
        assert api.get_device_error() == (0, 0)
        for i, (w, g) in enumerate(zip(want, got)):
            assert torch.equal(w.view(torch.uint8), g.view(torch.uint8)), (seed, i)
