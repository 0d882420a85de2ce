"""Infinite and NaN values of the prompt attention: where they end up, exactly.

A value's element (token j, KV head, column) may change that column of the rows that
attend it -- tokens j and later of its sequence, the heads of its group -- and those it
makes infinite or NaN.  Everything else equals the same call without it, bit for bit.
"""
import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from test_prompt_gpu import rows, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


def check(q, k, v, lens, scale, spots):
    """spots: (sequence, token, KV head, column, value)."""
    loc, g = starts(lens), q.shape[1] // k.shape[1]
    clean = api.prompt_attention(q, k, v, loc, scale)
    assert bool(clean.isfinite().all())
    v2, finite = v.clone(), torch.ones_like(q, dtype=torch.bool)
    first = [0] + torch.tensor(lens).cumsum(0).tolist()
    for s, j, h, c, x in spots:
        v2[first[s] + j, h, c] = x
        finite[first[s] + j:first[s + 1], h * g:(h + 1) * g, c] = False
    out = api.prompt_attention(q, k, v2, loc, scale)
    assert api.get_device_error() == (0, 0)
    assert torch.equal(out.isfinite(), finite)
    assert torch.equal(out[finite], clean[finite])
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("gap", [0.0, 19.0, 30.0, 120.0])
@pytest.mark.parametrize("h,hkv,d", [(8, 2, 64), (3, 3, 128)])
def test_a_peaked_row(h, hkv, d, gap, dtype):
    """Weights far below the row's largest, down to those that round to 0, on values in
    every place of an item and before it."""
    n = 700
    q, k, v = rows(n, h, hkv, d, dtype, 41)
    q, k = torch.zeros_like(q), torch.zeros_like(k)
    q[..., 0], k[0, :, 0] = 1, gap
    inf = float("inf")
    spots = [(0, j, j % hkv, c, x) for c, (j, x) in
             enumerate([(1, inf), (63, -inf), (64, inf), (128, float("nan")), (255, inf), (256, -inf), (333, inf),
                        (511, inf), (512, float("nan")), (640, inf), (699, -inf)])]
    check(q, k, v, [n], 1.0, spots)


@pytest.mark.parametrize("h,hkv,d,dtype", [(16, 8, 64, torch.float16), (32, 8, 128, torch.bfloat16),
                                           (8, 8, 128, torch.float16)])
def test_many_items_of_a_cta(h, hkv, d, dtype):
    """Ragged prompts, several items for each CTA, one sequence in three with such
    values: the marks of one item do not reach another."""
    g = torch.Generator().manual_seed(h)
    lens = torch.randint(1, 600, (100,), generator=g).tolist()
    q, k, v = rows(sum(lens), h, hkv, d, dtype, 42)
    values = [float("inf"), float("-inf"), float("nan")]
    pick = lambda n: int(torch.randint(n, (1,), generator=g))  # noqa: E731
    spots = [(s, pick(lens[s]), pick(hkv), pick(d), values[pick(3)]) for s in range(0, 100, 3) for _ in range(pick(3) + 1)]
    out = check(q, k, v, lens, d ** -0.5, spots)
    # over and over: the same answer, whichever CTA takes which item
    loc, first = starts(lens), [0] + torch.tensor(lens).cumsum(0).tolist()
    for s, j, hk, c, x in spots:
        v[first[s] + j, hk, c] = x
    for _ in range(10):
        again = api.prompt_attention(q, k, v, loc, d ** -0.5)
        assert torch.equal(again.isnan(), out.isnan()) and torch.equal(again[~out.isnan()], out[~out.isnan()])
