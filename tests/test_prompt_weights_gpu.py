"""Small weights of the prompt attention in f16: long rows whose many small weights
add up, against the definition in 64 bits.

Tolerance: that of test_prompt_gpu.py, but for the weights' subnormal steps.  A weight
is held in f16 as 2^7 times its share of the row's reference or more, so one below
2^-14 there is off by up to 2^-25, which is 2^-32 of the reference; n of them by
n 2^-32 max|v|.
"""
import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from test_prompt_gpu import exact, rows, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


def check(q, k, v, scale):
    n = q.shape[0]
    out = api.prompt_attention(q, k, v, starts([n]), scale)
    assert api.get_device_error() == (0, 0)
    ref, tol = exact(q, k, v, scale)
    tol = tol - n * (2.0 ** -25 - 2.0 ** -32) * v.double().abs().amax()
    assert float(((out.double() - ref).abs() - tol).max()) <= 0


@pytest.mark.parametrize("gap", [14.0, 17.675, 21.0])   # 2^-20, 2^-25.5, 2^-30
@pytest.mark.parametrize("where", [0, 1000, 6143])
@pytest.mark.parametrize("h,hkv,d", [(2, 1, 64), (1, 1, 128)])
def test_one_large_score_among_many_small_ones(h, hkv, d, gap, where):
    n = 6144
    q, k, v = (torch.zeros(n, x, d, dtype=torch.float16, device="cuda") for x in (h, hkv, hkv))
    q[..., 0] = 1
    k[where, :, 0] = gap
    v += 1
    v[where] = 0
    check(q, k, v, 1.0)


@pytest.mark.parametrize("spread", [1.0, 3.0, 8.0])
def test_random_scores(spread):
    q, k, v = rows(3000, 4, 2, 64, torch.float16, 31)
    check(q, k, v.abs(), spread * 0.125)


def test_largest_values():
    """Weights of 2^15 and values at the type's end: the sums stay in binary32."""
    q, k, v = rows(700, 4, 4, 64, torch.float16, 32)
    check(q, k, v.sign() * torch.finfo(torch.float16).max, 1.0)


def test_infinite_values_stay():
    """Only finite sums end at the largest value: an infinite one decides its column."""
    n, big = 300, torch.finfo(torch.float16).max
    q, k, v = rows(n, 2, 2, 64, torch.float16, 33)
    v = v.sign() * big
    v[0, 0, 3] = float("inf")
    v[290, 1, 5] = float("-inf")
    v[10, 1, 7] = float("nan")
    out = api.prompt_attention(q, k, v, starts([n]), 0.125)
    assert api.get_device_error() == (0, 0)
    want = torch.ones_like(out, dtype=torch.bool)
    want[:, 0, 3], want[290:, 1, 5], want[10:, 1, 7] = False, False, False
    assert torch.equal(out.isfinite(), want)
    assert bool((out[:, 0, 3] == float("inf")).all()) and bool((out[290:, 1, 5] == float("-inf")).all())
