"""Verification of drafted trees, further: long rows of refused children without a draft, and
sequences beside one that breaks the rules, each against the rules in 64 bits."""
import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from test_tree_verify_gpu import Case, expected, weight
from trees import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


@pytest.mark.parametrize("vocab", [40, 3001])
def test_many_looked_up_children(vocab):
    """Up to 300 children of a node, refused one after the other: each token out of the row once,
    those that come again with weight 0.  Node 150 is tried with a number that accepts it, so the
    list begins anew under it."""
    lens = [301, 64, 2, 300, 33]
    c = Case(lens, vocab, drafted=False, sharp=0.5)
    up, at = [], 0
    for n in lens:
        up += [-1] + [0 if i <= 150 else 150 for i in range(1, n)]
        if n > 150:
            c.accept[at + 150] = 0.0
        at += n
    c.up = i32(up)
    hard = torch.ones_like(c.accept, dtype=torch.bool)
    hard[c.accept == 0] = False
    c.accept[hard] = 1.0 - c.accept[hard] * 2.0 ** -12
    for _ in range(3):
        got = c.call()
        assert api.get_device_error() == (0, 0)
        c.check(got)
    assert max(got.accepted_lens.tolist()) > 1


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("lens", [[1025, 4], [4, 1025, 6, 1200, 3], [1100]])
def test_beside_a_sequence_of_too_many_nodes(lens, drafted):
    """The sequences beside it get their own verdicts; its rows of the path are not written."""
    c = Case(lens, 64, drafted=drafted, seed=len(lens))
    out = api.TreeVerdict(*(torch.full((n,), -7, dtype=torch.int32, device="cuda")
                            for n in (len(lens), sum(lens), len(lens))))
    got = c.call(out=out)
    assert api.get_device_error() == (-5, native.DEVERR_CONTEXT_LEN)
    at = 0
    for s, n in enumerate(lens):
        rows = slice(at, at + n)
        at += n
        if n > native.MAX_TREE_NODES:
            assert got.accepted_lens[s] == 0 and got.next_tokens[s] == -1 and (got.path[rows] == -7).all()
            continue
        want, token = expected(c.ids[rows].tolist(), c.up[rows].tolist(), weight(c.p[rows]),
                               weight(c.q[rows]) if drafted else None, c.accept[rows].tolist(), c.sample[s].item())
        assert got.path[rows].tolist() == want + [-1] * (n - len(want))
        assert got.accepted_lens[s] == len(want) and got.next_tokens[s] == token
