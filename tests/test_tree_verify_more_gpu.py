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
