"""Guard regions around every buffer that the calls of drafted trees read and write: the
margins still hold their pattern afterwards, and the results equal those on plain buffers
bit for bit.  And pools whose rows lie beyond 32-bit element numbers."""
import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from test_guards_gpu import Guarded, same_bits
from test_tree_attention_gpu import Case
from test_tree_step_gpu import Commit
from test_tree_verify_gpu import Case as Verdicts
from trees import attention, i32, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


def boxed(x):
    return Guarded(x.shape, x.dtype, init=x)


@pytest.mark.parametrize("before,nodes", [([5], [1]), ([900, 0, 33], [17, 64, 3]), ([100] * 90, [12] * 90)])
@pytest.mark.parametrize("h,hkv,d", [(8, 2, 128), (6, 2, 64), (5, 5, 128)])
def test_attention(before, nodes, h, hkv, d):
    c = Case(before, nodes, h, hkv, d, 16, torch.bfloat16)
    want = c.call()
    ins = [boxed(x) for x in (c.q, c.start, c.mask, c.cache.k, c.cache.v, c.cache.tables, c.ctx)]
    out = Guarded(c.q.shape, torch.bfloat16)
    ws = Guarded((api.tree_attention_workspace_size(c.q.shape[0], c.mask.shape[1], h, hkv, d),), torch.uint8)
    api.tree_attention(*(x.t for x in ins), c.scale, out=out.t, workspace=ws.t)
    assert api.get_device_error() == (0, 0)
    assert out.intact() and ws.intact() and all(x.intact() for x in ins)
    assert same_bits(out.t, want)


@pytest.mark.parametrize("lens", [[1], [70, 0, 3], [16] * 300])
def test_plan(lens):
    start, ctx = starts(lens), i32([n + 4 for n in lens])
    parents = i32([x for n in lens for x in [-1] + [i // 2 for i in range(n - 1)]][:sum(lens)])
    want = api.plan_tree(parents, start, ctx, 128)
    ins, outs = [boxed(x) for x in (parents, start, ctx)], [Guarded(x.shape, x.dtype) for x in want]
    api.plan_tree(*(x.t for x in ins), 128, out=api.TreePlan(*(x.t for x in outs)))
    assert api.get_device_error() == (0, 0)
    assert all(x.intact() for x in ins + outs) and all(same_bits(x.t, y) for x, y in zip(outs, want))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("vocab,lens", [(1, [3]), (4099, [6, 0, 9]), (70001, [5] * 9)])
def test_verify(vocab, lens, dtype):
    c = Verdicts(lens, vocab, dtype)
    want = c.call()
    ins = [boxed(x.contiguous()) for x in (c.ids, c.up, c.start, c.p, c.q, c.accept, c.sample)]
    outs = [Guarded(x.shape, x.dtype) for x in want]
    api.verify_tree(*(x.t for x in ins), out=api.TreeVerdict(*(x.t for x in outs)))
    assert api.get_device_error() == (0, 0)
    assert all(x.intact() for x in ins + outs) and all(same_bits(x.t, y) for x, y in zip(outs, want))


def test_commit():
    c = Commit([10, 3, 0], [30, 8, 5], [12, 3, 5], 2, 3, 64, 8, torch.bfloat16)
    want = c.expected()
    k, v = [boxed(x) for x in c.k], [boxed(x) for x in c.v]
    ins = [boxed(x) for x in (c.start, c.path, c.lens, i32(c.ctx), c.tables)]
    ring, free, lens, state = boxed(c.ring), boxed(c.free), Guarded((3,), torch.int32), Guarded((2,), torch.int32)
    c.k, c.v, c.ring = [x.t for x in k], [x.t for x in v], ring.t
    got = api.commit_tree(c.k, c.v, *(x.t for x in ins), free_ring=ring.t, free_state=free.t,
                          out=api.TreeCommit(lens.t, state.t))
    assert api.get_device_error() == (0, 0)
    assert all(x.intact() for x in k + v + ins + [ring, free, lens, state])
    c.check(want, got)


def test_pools_beyond_32_bits():
    """Rows of blocks behind element 2^32: attended to, and moved."""
    h, hkv, d, b, dt = 8, 4, 128, 16, torch.bfloat16
    blocks = (1 << 32) // (hkv * b * d) + 64
    k = torch.zeros(blocks, hkv, b, d, dtype=dt, device="cuda")
    v = torch.zeros(blocks, hkv, b, d, dtype=dt, device="cuda")
    ids = torch.arange(blocks - 8, blocks, device="cuda", dtype=torch.int32)
    g = torch.Generator(device="cuda").manual_seed(1)
    k[-8:], v[-8:] = (torch.randn(8, hkv, b, d, generator=g, device="cuda").to(dt) for _ in range(2))
    n, ctx = 6, 8 * b - 3
    q = torch.randn(n, h, d, generator=g, device="cuda").to(dt)
    mask = torch.tensor([[1], [3], [5], [9], [17], [35]], device="cuda")
    start, lens = starts([n]), i32([ctx])
    out = api.tree_attention(q, start, mask, k, v, ids[None], lens, d ** -0.5)
    rows = [x[-8:].transpose(1, 2).flatten(0, 1)[:ctx] for x in (k, v)]
    allowed = ((mask >> torch.arange(n, device="cuda")) & 1).bool()
    ref, tol = attention(q, *rows, ctx - n, allowed, d ** -0.5)
    assert ((out.double() - ref).abs() <= tol).all()
    path = i32([0, 1, 5, -1, -1, -1])
    api.commit_tree([k], [v], start, path, i32([3]), lens, ids[None])
    assert api.get_device_error() == (0, 0)
    for x, old in zip((k, v), rows):
        old = old.clone()
        old[ctx - n + 2] = old[ctx - 1]
        assert torch.equal(x[-8:].transpose(1, 2).flatten(0, 1)[:ctx], old)
