"""Attention of drafted trees over the paged cache against its definition in 64 bits
(the tolerance is derived in trees.attention)."""
import random

import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from trees import Cache, ancestors, attention, i32, random_trees, starts, words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


class Case:
    """Sequences of `before` cached tokens and `nodes` of a tree behind them."""

    def __init__(self, before, nodes, h, hkv, d, block, dtype, width=3, seed=1, rows=None, count=None, extra=0, first=0,
                 fused=False):
        self.before, self.nodes, self.scale = before, nodes, d ** -0.5
        self.cache = Cache([b + n for b, n in zip(before, nodes)], hkv, d, block, dtype, seed)
        self.first, total = first, first + sum(nodes) + extra
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        wide = torch.randn(total, (h + 2 * hkv) * d, generator=g, device="cuda").to(dtype)
        self.q = wide[:, :h * d].unflatten(1, (h, d))
        if not fused:
            self.q = self.q.contiguous()
        count = count or max(1, -(-max(nodes + [1]) // 64))
        # rows of node numbers, sequence by sequence
        self.attends = rows if rows is not None else [ancestors(p) for p in random_trees(nodes, width, seed)]
        # a mask's bits past a tree's nodes, and rows of no sequence, count for nothing
        self.mask = torch.full((total, count), -1, dtype=torch.int64)
        at = first
        for s, seq in enumerate(self.attends):
            for i, row in enumerate(seq):
                past = range(len(seq), 64 * count) if (s + i) % 2 else ()
                self.mask[at] = words([list(row) + list(past)], count)[0]
                at += 1
        self.mask = self.mask.cuda()
        self.start = starts(nodes, first)
        self.ctx = i32([b + n for b, n in zip(before, nodes)])

    def call(self, **kw):
        return api.tree_attention(self.q, self.start, self.mask, self.cache.k, self.cache.v, self.cache.tables, self.ctx,
                                  self.scale, **kw)

    def check(self, out, skip=()):
        at = self.first
        for s, (b, n) in enumerate(zip(self.before, self.nodes)):
            if n and s not in skip:
                k, v = self.cache.rows(s, b + n)
                allowed = torch.zeros(n, n, dtype=torch.bool)
                for i, row in enumerate(self.attends[s]):
                    allowed[i, list(row)] = True
                ref, tol = attention(self.q[at:at + n], k, v, b, allowed, self.scale)
                got = out[at:at + n]
                assert not torch.isnan(got).any(), f"NaN in sequence {s} ({b} + {n})"
                off = (got.double() - ref).abs() - tol
                assert float(off.max()) <= 0, f"sequence {s} ({b} + {n}): {float(off.max())} over its tolerance"
            at += n


def run(*args, **kw):
    c = Case(*args, **kw)
    out = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda")
    assert c.call(out=out) is out
    assert api.get_device_error() == (0, 0)
    c.check(out)
    end = c.first + sum(c.nodes)
    assert (out[:c.first] == 7).all() and (out[end:] == 7).all(), "rows of no sequence were written"
    return c, out


BF16, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("before,n", [(0, 1), (5, 1), (7, 3), (127, 1), (128, 5), (120, 8), (100, 60), (300, 64)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
def test_one_sequence(before, n, dtype, d):
    run([before], [n], 8, 2, d, 16, dtype)


@pytest.mark.parametrize("block", [8, 16, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_block_sizes(block, d):
    run([0, 3, 500, 129, 31], [9, 1, 17, 40, 64], 8, 4, d, block, BF16)


@pytest.mark.parametrize("h,hkv", [(4, 4), (8, 1), (12, 4), (5, 1), (7, 7), (32, 2), (128, 1), (130, 2)])
def test_heads(h, hkv):
    run([200, 0, 61, 1000], [7, 13, 1, 30], h, hkv, 64, 16, F16)


@pytest.mark.parametrize("nodes", [[31], [32], [33], [64], [65], [127], [128], [129], [200, 1, 70], [600], [1024]])
def test_more_rows_than_a_tile(nodes):
    """Group 4: 32 nodes to a query tile, 64 to a pair of them."""
    run([150 + 7 * i for i in range(len(nodes))], nodes, 8, 2, 128, 16, BF16, width=9)


@pytest.mark.parametrize("seed", range(4))
def test_many_ragged_sequences(seed):
    r = random.Random(seed)
    s = r.choice([40, 150, 700])
    before = [r.choice([0, 1, 15, 16, 127, 128, r.randrange(1500)]) for _ in range(s)]
    nodes = [r.choice([0, 1, 2, 16, 33, 40]) for _ in range(s)]
    run(before, nodes, 8, 2, r.choice([64, 128]), r.choice([8, 16, 32]), r.choice([BF16, F16]), seed=seed)


def test_many_sequences_of_several_pairs():
    r = random.Random(3)
    nodes = [r.choice([0, 20, 70, 150]) for _ in range(600)]
    run([r.randrange(200) for _ in nodes], nodes, 4, 1, 64, 16, BF16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [2, 8])
def test_short_sequences_in_a_row(d, hkv):
    """Items of one K/V tile, which one chain computes alone, among items of both chains."""
    r = random.Random(hkv)
    before = [r.choice([1, 20, 90, 100, 100, 300]) for _ in range(600)]
    c, want = run(before, [r.choice([1, 16, 16, 40]) for _ in before], 4 * hkv, hkv, d, 16, BF16)
    for _ in range(20):
        out = c.call()
    assert torch.equal(out, want)
    # one long sequence first: the short ones' items follow in the same CTA
    run([4000] + [40] * 300, [8] * 301, 4 * hkv, hkv, d, 16, BF16)


def test_one_long_sequence_is_shared_by_every_cta():
    run([32768 - 5], [17], 8, 2, 128, 16, BF16)
    run([40000], [1], 1, 1, 64, 32, F16)


def test_rows_that_attend_to_nothing_are_zero():
    rows = [[[], [0], [0, 1], []], [[], [], []], [[1], [0]]]
    c, out = run([0, 0, 20], [4, 3, 2], 8, 2, 64, 16, BF16, rows=rows)
    assert (out[0] == 0).all() and (out[3:7] == 0).all()


def test_any_mask():
    """Not a tree: later nodes, and without itself."""
    r = random.Random(5)
    nodes = [90, 64, 3]
    rows = [[[j for j in range(n) if r.random() < 0.3] for _ in range(n)] for n in nodes]
    run([0, 77, 256], nodes, 8, 2, 128, 8, F16, rows=rows)


def test_chain_equals_causal_prefill():
    c, out = run([700, 33, 0], [16, 5, 64], 8, 2, 128, 16, BF16, width=1)
    ref = api.prefill(c.q, c.start, c.cache.k, c.cache.v, c.cache.tables, c.ctx, c.scale, 64, out_dtype=torch.float32)
    assert api.get_device_error() == (0, 0)
    assert float((out.float() - ref).abs().max()) < 0.05


def test_rows_of_a_fused_projection_and_padding():
    run([90, 300], [10, 40], 8, 2, 128, 16, BF16, fused=True, extra=13, first=5, count=3)


def test_masked_values_of_any_kind():
    """NaN and infinite values of nodes that a row does not attend to change nothing;
    those that it does make their columns so."""
    for dtype in (BF16, F16):
        for before in (0, 100, 1000):
            nodes = [40]
            c = Case([before], nodes, 8, 2, 128, 16, dtype, width=40, seed=before + 2)
            at = c.cache.slots(0, before + 40)
            clean = c.call()
            for node, column, bad in ((7, 3, float("nan")), (11, 100, float("inf")), (11, 64, float("-inf"))):
                c.cache.v[at[before + node] // 16, 1, at[before + node] % 16, column] = bad
            c.cache.k[at[before + 7] // 16, 0, at[before + 7] % 16] = float("nan")
            out = c.call()
            assert api.get_device_error() == (0, 0)
            for i, row in enumerate(c.attends[0]):
                for h in range(8):
                    want = clean[i, h].clone()
                    if 7 in row and h < 4:
                        want[:] = float("nan")
                    if h >= 4:
                        if 7 in row:
                            want[3] = float("nan")
                        if 11 in row:
                            want[100], want[64] = float("inf"), float("-inf")
                    assert torch.allclose(out[i, h], want, rtol=0, atol=0, equal_nan=True), (dtype, before, i, h)


def test_non_finite_values_before_the_tree_stay_in_their_columns():
    c = Case([300], [5], 8, 2, 64, 16, BF16)
    clean = c.call()
    at = c.cache.slots(0, 305)
    c.cache.v[at[17] // 16, 0, at[17] % 16, 9] = float("nan")
    out = c.call()
    assert out[:, :4, 9].isnan().all()
    out[:, :4, 9] = clean[:, :4, 9]
    assert torch.equal(out, clean)


def test_f16_means_next_to_the_types_end():
    c = Case([500], [8], 8, 2, 64, 16, F16)
    c.cache.v[~c.cache.v.isnan()] = 65504.0
    out = c.call()
    assert (out == 65504.0).all()
    at = c.cache.slots(0, 508)
    c.cache.v[at[20] // 16, 0, at[20] % 16, 5] = float("inf")
    out = c.call()
    assert not torch.isfinite(out[:, :4, 5].float()).any() and (out[:, 4:] == 65504.0).all()


def test_large_scores():
    """Differences of hundreds between scores: the running maximum is moved often."""
    c = Case([900, 10], [30, 64], 8, 2, 128, 16, BF16)
    c.q *= 40
    out = c.call()
    c.check(out)


def test_deterministic_and_workspaces_apart():
    c = Case([5000, 3, 400], [20, 9, 64], 8, 2, 128, 16, BF16)
    want = c.call()
    assert all(torch.equal(c.call(), want) for _ in range(5))
    need = api.tree_attention_workspace_size(c.q.shape[0], 1, 8, 2, 128)
    a, b = (torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for st, ws in zip(streams, (a, b)):
            out = torch.zeros_like(want)
            torch.cuda.synchronize()
            c.call(out=out, workspace=ws, stream=st)
            outs.append(out)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_captured_and_replayed_with_other_lengths():
    c = Case([3000, 70, 0], [20, 9, 33], 8, 2, 128, 16, BF16)
    out, ws = torch.zeros_like(c.q), torch.zeros(api.tree_attention_workspace_size(c.q.shape[0], 1, 8, 2, 128),
                                                 dtype=torch.uint8, device="cuda")
    c.call(out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(out=out, workspace=ws)
    for before, nodes in (([3000, 70, 0], [20, 9, 33]), ([1, 500, 2222], [3, 40, 2]), ([64, 64, 64], [0, 0, 7])):
        n = Case(before, nodes, 8, 2, 128, 16, BF16, seed=sum(nodes))
        want = n.call()
        for dst, src in ((c.ctx, n.ctx), (c.start, n.start)):
            dst.copy_(src)
        rows = n.q.shape[0]
        c.q[:rows], c.mask[:rows] = n.q, n.mask
        # the replayed call reads the captured pools: the new sequences' rows go there
        for s, (b, m) in enumerate(zip(before, nodes)):
            k, v = n.cache.rows(s, b + m)
            used = -(-(b + m) // 16)
            assert used <= c.cache.tables.shape[1]
            ids = torch.arange(used, dtype=torch.int32, device="cuda") + sum(
                -(-(x + y) // 16) for x, y in zip(before[:s], nodes[:s]))
            assert used == 0 or int(ids.max()) < c.cache.num_blocks
            c.cache.tables[s, :used] = ids
            at = c.cache.slots(s, b + m)
            c.cache.k[at // 16, :, at % 16], c.cache.v[at // 16, :, at % 16] = k, v
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert api.get_device_error() == (0, 0)
        assert torch.equal(out[:rows], want) and (out[rows:] == 7).all()


def test_bad_lengths_and_blocks_are_reported():
    nodes = [5, 6, 7, 8]
    c = Case([100, 200, 300, 40], nodes, 8, 2, 64, 16, BF16)
    want = c.call()
    c.ctx[1] = 3                     # fewer tokens than nodes
    c.ctx[3] = 16 * c.cache.tables.shape[1] + 1  # past the table
    out = torch.full_like(want, 7.0)
    c.call(out=out)
    assert api.get_device_error() == (-5, native.DEVERR_CONTEXT_LEN)
    assert (out[5:11] == 7).all() and (out[18:] == 7).all()
    u = 2.0 ** -7  # other borders of the work: sums in another order, then one rounding
    for rows in (slice(0, 5), slice(11, 18)):
        assert torch.allclose(out[rows].float(), want[rows].float(), rtol=u, atol=1e-3)
    c = Case([100, 200, 300, 40], nodes, 8, 2, 64, 16, BF16)
    c.cache.tables[2, 4] = c.cache.num_blocks
    c.call(out=out)
    assert api.get_device_error() == (-5, native.DEVERR_BLOCK_ID)
    assert torch.equal(out[:11], want[:11]) and torch.equal(out[18:], want[18:])


def test_refusals():
    c = Case([100], [5], 8, 2, 64, 16, BF16)
    args = [c.q, c.start, c.mask, c.cache.k, c.cache.v, c.cache.tables, c.ctx, c.scale]

    def refused(error, **over):
        names = ["q", "start", "mask", "k", "v", "tables", "ctx", "scale"]
        call = [over.pop(n, a) for n, a in zip(names, args)]
        with pytest.raises(error):
            api.tree_attention(*call, **over)

    refused(ValueError, q=c.q[:, :, :32])
    refused(ValueError, q=c.q.half())
    refused(ValueError, q=c.q.cpu())
    refused(ValueError, mask=c.mask[:4])
    refused(ValueError, mask=c.mask.int())
    refused(ValueError, start=c.start.long())
    refused(ValueError, tables=c.cache.tables.long())
    refused(ValueError, ctx=c.ctx.repeat(2))
    refused(ValueError, out=torch.empty(5, 8, 64, device="cuda"))
    refused(native.PaError, scale=0.0)
    refused(native.PaError, scale=float("nan"))
    refused(native.PaError, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    refused(native.PaError, mask=c.mask.repeat(1, 17))
    with pytest.raises(native.PaError):  # 32-bit pools
        api.tree_attention(c.q.float(), c.start, c.mask, c.cache.k.float(), c.cache.v.float(), c.cache.tables, c.ctx, 1.0)
    assert api.get_device_error() == (0, 0)


def test_nothing_to_do():
    c = Case([100, 5], [0, 0], 8, 2, 64, 16, BF16, extra=3)
    out = torch.full_like(c.q, 7.0)
    c.call(out=out)
    assert api.get_device_error() == (0, 0) and (out == 7).all()
    empty = api.tree_attention(c.q[:0], c.start, c.mask[:0], c.cache.k, c.cache.v, c.cache.tables, c.ctx, 1.0)
    assert empty.shape == (0, 8, 64)
