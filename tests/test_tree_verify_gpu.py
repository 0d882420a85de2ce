"""Verification of drafted trees against its rules in 64 bits, token for token: the
sums of weights are exact to 2^-52 a weight and better, so a token differs only where a random
number falls that close to a border."""
import math
import random

import numpy as np
import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from trees import i32, parents_of, random_trees, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


def weight(x):
    """A probability as the call reads it."""
    return np.clip(np.nan_to_num(x.double().cpu().numpy(), nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)


def expected(ids, parents, p, q, accept_u, sample_u):
    """One sequence: (path, token); p and q are [n][V] arrays of weights, q None without a draft."""
    path = [0]
    while True:
        row = p[path[-1]]
        left, s, c, taken = row, 1.0, 0.0, None
        for i in [j for j in range(1, len(parents)) if parents[j] == path[-1]]:
            x = ids[i]
            if accept_u[i] * (1.0 if q is None else q[path[-1]][x]) * s < left[x]:
                taken = i
                break
            if q is None:
                s = max(s - left[x], 0.0)
                left = left.copy()
                left[x] = 0.0
            else:
                c += s
                left = np.maximum(row - c * q[path[-1]], 0.0)
                s = math.fsum(left)
                if s == 0.0:
                    break
        if taken is None:
            break
        path.append(taken)
    if not left.any():
        left = row
    if not left.any():
        return path, -1
    below = np.cumsum(left)
    at = int(np.searchsorted(below, sample_u * below[-1], side="right"))
    return path, min(at, int(np.flatnonzero(left)[-1]))


class Case:
    def __init__(self, lens, vocab, dtype=torch.float32, drafted=True, width=3, spread=0.6, seed=1, pad=0, extra=0,
                 sharp=2.5):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = sum(lens) + extra
        self.lens, self.vocab = lens, vocab
        self.parents = random_trees(lens, width, seed)

        def probs(logits):
            wide = torch.full((n, vocab + pad), float("nan"), dtype=dtype, device="cuda")
            wide[:, :vocab] = torch.softmax(logits, 1).to(dtype)
            return wide[:, :vocab]

        logits = torch.randn(n, vocab, generator=g, device="cuda") * sharp
        self.p = probs(logits)
        draft = probs(logits + torch.randn(n, vocab, generator=g, device="cuda") * spread)
        first = [a for a, x in zip(starts(lens).tolist(), lens) for _ in range(x)]
        above = torch.tensor([a + max(u, 0) for a, u in zip(first, [u for ps in self.parents for u in ps])] + [0] * extra,
                             device="cuda")
        u = torch.rand(n, 1, generator=g, device="cuda", dtype=torch.float64)
        cum = draft.double().cumsum(1)[above]
        self.ids = torch.searchsorted(cum, u * cum[:, -1:], right=True).clamp_(max=vocab - 1)[:, 0].int()
        self.q = draft if drafted else None
        self.accept = torch.rand(n, generator=g, device="cuda")
        self.sample = torch.rand(len(lens), generator=g, device="cuda")
        self.start = starts(lens)
        self.up = i32([u for ps in self.parents for u in ps] + [-1] * extra)

    def call(self, **kw):
        return api.verify_tree(self.ids, self.up, self.start, self.p, self.q, self.accept, self.sample, **kw)

    def check(self, got, some=None):
        lens, path, tokens = (x.tolist() for x in got)
        at = 0
        for s, n in enumerate(self.lens):
            if n == 0:
                assert lens[s] == 0 and tokens[s] == -1
            elif some is None or s in some:
                rows = slice(at, at + n)
                want, token = expected(self.ids[rows].tolist(), self.up[rows].tolist(), weight(self.p[rows]),
                                       None if self.q is None else weight(self.q[rows]), self.accept[rows].tolist(),
                                       self.sample[s].item())
                assert path[rows] == want + [-1] * (n - len(want)), s
                assert lens[s] == len(want) and tokens[s] == token, (s, want, token, tokens[s])
            at += n


def run(*args, **kw):
    c = Case(*args, **kw)
    got = c.call()
    assert api.get_device_error() == (0, 0)
    c.check(got)
    return c, got


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("vocab", [1, 2, 5, 511, 512, 513, 4096, 5003, 32000])
def test_vocabularies(vocab, drafted, dtype):
    run([1, 2, 9, 0, 6], vocab, dtype, drafted, seed=vocab)


@pytest.mark.parametrize("vocab,seqs", [(131072, 1), (128256, 3), (50021, 40), (100003, 20)])
@pytest.mark.parametrize("drafted", [True, False])
def test_large_vocabularies(vocab, seqs, drafted):
    run([5] * seqs, vocab, drafted=drafted, seed=seqs)


@pytest.mark.parametrize("seqs", [1, 37, 38, 76, 77, 152, 153, 305, 700])
def test_batches(seqs):
    """Eight, four, two CTAs to a sequence, and one."""
    r = random.Random(seqs)
    run([r.randrange(0, 8) for _ in range(seqs)], 33000, width=2, seed=seqs)


@pytest.mark.parametrize("spread", [0.0, 0.1, 3.0])
@pytest.mark.parametrize("width", [1, 2, 30])
def test_wide_and_deep_trees(spread, width):
    """Width 30: most nodes are children of the first few, and are refused one after the other."""
    run([40, 64, 33] * 3, 1009, width=width, spread=spread, seed=width)


def test_the_largest_tree():
    run([1024, 3], 700, width=200, spread=2.0)
    c = Case([1025, 4], 64)
    got = c.call()
    assert api.get_device_error() == (-5, native.DEVERR_CONTEXT_LEN)
    assert got.accepted_lens.tolist()[0] == 0 and got.next_tokens.tolist()[0] == -1
    c.lens[0] = 0
    rows = c.call()
    api.get_device_error()
    assert torch.equal(rows.next_tokens, got.next_tokens)


def test_equal_distributions_accept_everything():
    """u < 1, so a child whose q is its p is never refused; a chain is kept whole."""
    c = Case([9, 5], 900, width=1, spread=0.0)
    c.q = c.p.clone()
    got = c.call()
    assert got.accepted_lens.tolist() == [9, 5]
    c.check(got)


def test_same_token_twice():
    for drafted in (True, False):
        c = Case([6, 6, 6, 6], 50, drafted=drafted, width=6, spread=2.0, sharp=0.5)
        c.up = i32([-1, 0, 0, 0, 0, 0] * 4)
        c.ids[1:4], c.ids[7:12] = 17, 3
        c.accept[:] = 0.999
        c.check(c.call())


def test_residual_without_weight_falls_back_to_the_row():
    """q covers p everywhere (no distribution): a refusal leaves nothing."""
    c = Case([4, 4], 300, width=1)
    c.q = torch.ones_like(c.p)
    c.accept[:] = 0.9999
    got = c.call()
    assert got.accepted_lens.tolist() == [1, 1]
    c.check(got)
    c = Case([3], 2, drafted=False, width=3)   # every token refused
    c.up, c.ids = i32([-1, 0, 0]), i32([0, 0, 1])
    c.p[:] = torch.tensor([0.4, 0.3], device="cuda")
    c.accept[:] = 1.0
    got = c.call()
    assert got.accepted_lens.tolist() == [1]
    c.check(got)


def test_strange_probabilities():
    """NaN and negative entries count as 0, those above 1 as 1; a row of zeros has no token."""
    c = Case([5, 5, 5], 2000, width=2)
    c.p[:, 5::7], c.p[:, 6::7], c.q[:, 3::5] = float("nan"), -1.0, float("nan")
    c.p[2, 8] = float("inf")
    got = c.call()
    assert api.get_device_error() == (0, 0)
    c.check(got)
    c.p[5:10] = 0.0
    got = c.call()
    assert api.get_device_error() == (-5, native.DEVERR_PROBS)
    assert got.next_tokens.tolist()[1] == -1 and got.accepted_lens.tolist()[1] == 1
    c.check(got)


@pytest.mark.parametrize("u", [0.0, 0.99999994, 1.0, 2.0, -1.0, float("nan")])
def test_ends_of_the_random_numbers(u):
    """1 and more: as the largest number below 1; negative and NaN: as 0."""
    c = Case([4, 3], 777, sharp=0.1)
    c.sample[:] = u
    got = c.call()
    c.sample[:] = 0.0 if not u >= 0 else min(u, 0.99999994)
    c.check(got)


def test_borders_of_the_cumulative_weights():
    """Equal weights of 2^-9: the k-th border is k 2^-9 exactly, and belongs to the next token;
    the next smaller binary32 number (2^-26 and less is no step above 1/4, where they are 2^-25
    apart) to the one before."""
    n = 64
    c = Case([1] * n, 512)
    c.p[:] = 2.0 ** -9
    c.sample[:] = torch.arange(n, device="cuda") * 2.0 ** -9 * 8
    assert c.call().next_tokens.tolist() == [8 * k for k in range(n)]
    c.sample[1:] = torch.nextafter(c.sample[1:], torch.zeros(n - 1, device="cuda"))
    assert c.call().next_tokens.tolist()[1:] == [8 * k - 1 for k in range(1, n)]


@pytest.mark.parametrize("pad", [1, 3, 4, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_padded_rows(pad, dtype):
    """Strides of any size; the rows of the draft begin elsewhere than the target's."""
    c, got = run([6, 2, 7], 3001, dtype, pad=pad, extra=4)
    tight = torch.empty(c.p.shape[0], c.vocab + pad + 5, dtype=dtype, device="cuda")[:, 2:2 + c.vocab]
    tight.copy_(c.q)
    c.q = tight
    again = c.call()
    assert all(torch.equal(a[:15], b[:15]) for a, b in zip(again, got))


def test_bad_parents_and_tokens():
    c = Case([6, 6, 6], 100, width=2)
    c.up[2], c.up[4], c.ids[9], c.ids[14] = 2, -7, 100, -1
    got = c.call()
    assert api.get_device_error() == (-5, native.DEVERR_TREE)
    c.up[2] = c.up[4] = c.up[9] = c.up[14] = -1   # tried by none
    assert all(torch.equal(a, b) for a, b in zip(got, c.call()))
    assert api.get_device_error() == (-5, native.DEVERR_TREE)
    c.ids[9] = c.ids[14] = 0
    c.check(c.call())
    assert api.get_device_error() == (0, 0)


def test_bad_start_rows():
    c = Case([6, 6, 6], 100)
    want = c.call()
    c.start[1] = 30   # sequences 0 and 1 break the rules
    got = c.call()
    assert api.get_device_error() == (-5, native.DEVERR_CONTEXT_LEN)
    assert got.accepted_lens.tolist()[:2] == [0, 0] and got.next_tokens.tolist()[:2] == [-1, -1]
    assert torch.equal(got.path[12:], want.path[12:]) and got.next_tokens[2] == want.next_tokens[2]


def test_streams_capture_and_repeats():
    c = Case([7] * 30, 20011)
    want = c.call()
    assert all(all(torch.equal(a, b) for a, b in zip(c.call(), want)) for _ in range(5))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = api.TreeVerdict(*(torch.empty_like(x) for x in want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(out=out)
    other = Case([7] * 30, 20011, seed=9)
    for name in ("ids", "up", "p", "q", "accept", "sample"):
        getattr(c, name).copy_(getattr(other, name))
    graph.replay()
    torch.cuda.synchronize()
    other.check(out)


def test_tokens_are_distributed_as_the_targets():
    """First tokens behind the root over 40 000 draws of two children each: frequencies
    within 5 standard deviations of p, sqrt(p (1 - p) / n) each."""
    n, vocab = 40000, 8
    g = torch.Generator(device="cuda").manual_seed(4)
    p = torch.tensor([.3, .25, .2, .1, .05, .05, .03, .02], device="cuda")
    q = torch.tensor([.05, .1, .2, .3, .05, .1, .1, .1], device="cuda")
    rows_p, rows_q = p.repeat(3 * n, 1), q.repeat(3 * n, 1)
    ids = torch.multinomial(q, 3 * n, replacement=True, generator=g).int()
    up = i32([-1, 0, 0]).repeat(n)
    got = api.verify_tree(ids, up, starts([3] * n), rows_p, rows_q, torch.rand(3 * n, generator=g, device="cuda"),
                          torch.rand(n, generator=g, device="cuda"))
    second = got.path.view(n, 3)[:, 1].long()
    drawn = torch.where(second >= 0, ids.view(n, 3).gather(1, second.clamp(min=0)[:, None])[:, 0], got.next_tokens)
    freq = torch.bincount(drawn.long(), minlength=vocab).double() / n
    assert ((freq - p.double()).abs() <= 5 * (p * (1 - p) / n).double().sqrt()).all()


def test_refusals():
    c = Case([4, 3], 100)
    args = dict(tokens=c.ids, parents=c.up, query_start_loc=c.start, target_probs=c.p, draft_probs=c.q,
                accept_uniforms=c.accept, sample_uniforms=c.sample)
    for over in (dict(tokens=c.ids.long()), dict(parents=c.up[:6]), dict(query_start_loc=c.start.long()),
                 dict(target_probs=c.p[:6]), dict(target_probs=c.p.double()), dict(draft_probs=c.q.half()),
                 dict(draft_probs=c.q[:, :50]), dict(accept_uniforms=c.accept[:3]), dict(sample_uniforms=c.sample.double()),
                 dict(sample_uniforms=c.sample.cpu()), dict(target_probs=c.p.cpu(), draft_probs=None),
                 dict(target_probs=c.p.t().contiguous().t()), dict(out=(c.up, c.up, c.up))):
        with pytest.raises(ValueError):
            api.verify_tree(**{**args, **over})
    assert api.get_device_error() == (0, 0)
